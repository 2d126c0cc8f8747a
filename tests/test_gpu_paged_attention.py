"""Attention of new tokens over a paged cache against the 64-bit definition
(attention_ref) on the oracle's products: single tokens and chunks, grouped
heads, pages that end inside a tile of keys, ragged and empty sequences,
missing pages, special values in masked places, large offsets, streams and
graphs."""
import numpy as np
import pytest

import attention_ref as ref
import oracle
from datagen import normal
from test_gpu_attention import dev, load

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def am():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import approximate_multiplier_dnn_amd as m
    yield m
    m.approx_exponent_bits_set(8)
    m.approx_lut_load(oracle.lut_generate(7, "mitchell"), 7)


def cache(seed, k_len, page, K, D, spare=2, width=None):
    """Pages in a shuffled order; (k_pages, v_pages, table)."""
    count = [-(-n // page) for n in k_len]
    total = sum(count) + spare
    order = np.random.RandomState(seed).permutation(total).astype(np.int32)
    table = np.full((len(k_len), width or max(count + [1])), -1, np.int32)
    at = 0
    for b, c in enumerate(count):
        table[b, :c] = order[at:at + c]
        at += c
    return normal(seed + 1, (total, page, K, D)), normal(seed + 2, (total, page, K, D)), table


def reference(q, kp, vp, table, new, k_len, causal, scale, lut, M, E=8):
    H, K, D = q.shape[1], kp.shape[2], q.shape[2]
    o, lse, mag = np.zeros(q.shape), np.zeros(q.shape[:2]), np.zeros(q.shape)
    at = 0
    for b, n in enumerate(new):
        m = k_len[b]
        pages = table[b][: -(-m // kp.shape[1])]
        there = (pages >= 0) & (pages < kp.shape[0])
        rows = np.repeat(there, kp.shape[1])[:m]
        k, v = (x[np.where(there, pages, 0)].reshape(-1, K, D)[:m] for x in (kp, vp))
        seen = ref.causal_mask(n, m, causal) & rows[None]
        for h in range(H):
            g = h // (H // K)
            o[at:at + n, h], lse[at:at + n, h], mag[at:at + n, h] = ref.attention(q[at:at + n, h], k[:, g], v[:, g], seen, scale, lut, M, E)
        at += n
    return o, lse, mag


def check(am, mul, q, kp, vp, table, new, k_len, causal=True, scale=None, E=8, what=""):
    lut, M = mul
    lse = torch.full(q.shape[:2], 5.0, device="cuda")
    o = am.attention_paged(dev(q), dev(kp), dev(vp), dev(table), dev(ref.packed(new)), dev(np.array(k_len, np.int32)), causal=causal,
                           scale=scale, lse=lse)
    torch.cuda.synchronize()
    o, lse = o.cpu().numpy(), lse.cpu().numpy()
    scale = q.shape[2] ** -0.5 if scale is None else scale
    want, want_lse, mag = reference(q, kp, vp, table, new, k_len, causal, scale, lut, M, E)
    extra = 2.0 ** -23 * (1 + 8 * scale * q.shape[2]) if lut is None else 0.0
    ref.near(o, want, np.where(np.isfinite(mag), mag, 0.0), max(k_len, default=0), what, extra)
    fin = np.isfinite(want_lse)
    assert np.array_equal(np.isnan(lse), np.isnan(want_lse)) and np.array_equal(np.isinf(lse), np.isinf(want_lse)), what
    assert (np.abs(lse[fin] - want_lse[fin]) <= (2.0 ** -23 + extra) * (1 + np.abs(want_lse[fin]))).all(), what
    return o, lse


CASES = [
    # multiplier, new tokens, cached keys, page, heads, kv heads, dim
    ("mitchell07", [1], [1], 16, 1, 1, 64),
    ("mitchell07", [1, 1, 1], [300, 17, 64], 16, 8, 2, 64),
    ("mitchell07", [1, 1], [130, 700], 100, 12, 4, 128),
    ("mitchell07", [1, 0, 1], [65, 9, 0], 8, 4, 4, 32),           # no new token; no cached key
    ("mitchell07", [40, 3, 1], [100, 3, 257], 16, 4, 2, 64),      # chunks
    ("skew07", [17], [200], 24, 6, 2, 40),
    ("skew07", [9, 30], [9, 64], 1, 2, 1, 80),                    # pages of one key
    ("mitchell07", [5], [70], 7, 3, 1, 33),                       # odd dimension and page
    ("mitchell07", [6], [4], 16, 2, 2, 64),                       # more tokens than keys
    ("exact01", [1], [20], 16, 2, 1, 3),
    ("perturbed08", [1, 20], [150, 90], 16, 8, 2, 64),
    ("perturbed08", [3], [100], 64, 8, 1, 128),
    ("exact09", [1, 9], [70, 40], 16, 4, 1, 64),
    ("native", [1, 20], [90, 50], 16, 8, 2, 96),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}-p{c[3]}-{c[4]}x{c[5]}x{c[6]}")
def test_against_definition(am, case):
    name, new, k_len, page, H, K, D = case
    mul = load(am, name)
    kp, vp, table = cache(8000 + 13 * D + H, k_len, page, K, D)
    q = normal(8001 + D, (sum(new), H, D))
    check(am, mul, q, kp, vp, table, new, k_len, what=str(case))
    if max(new) > 1:
        check(am, mul, q, kp, vp, table, new, k_len, causal=False, what=str(case))


def test_more_sequences_than_a_wave(am):
    mul = load(am, "mitchell07")
    k_len = [int(n) for n in np.random.RandomState(8).randint(0, 40, 70)]
    new = [min(1, n) for n in k_len]
    kp, vp, table = cache(8050, k_len, 16, 1, 32)
    check(am, mul, normal(8051, (sum(new), 2, 32)), kp, vp, table, new, k_len, what="many")


def test_same_result_as_packed(am):
    """The whole prompt as one chunk over the cache is the packed call."""
    mul = load(am, "mitchell07")
    k_len, page, H, K, D = [90, 33], 16, 4, 2, 64
    kp, vp, table = cache(8100, k_len, page, K, D)
    q = normal(8101, (sum(k_len), H, D))
    o, lse = check(am, mul, q, kp, vp, table, k_len, k_len)
    k, v = (np.concatenate([x[table[b][: -(-n // page)]].reshape(-1, K, D)[:n] for b, n in enumerate(k_len)]) for x in (kp, vp))
    cu = dev(ref.packed(k_len))
    o2, lse2 = am.attention_fwd(dev(q), dev(k), dev(v), cu, cu)
    torch.cuda.synchronize()
    assert np.array_equal(lse.view(np.uint32), lse2.cpu().numpy().view(np.uint32))
    want, _, mag = reference(q, kp, vp, table, k_len, k_len, True, D ** -0.5, *mul)
    ref.near(o2.cpu().numpy(), want, mag, max(k_len))


@pytest.mark.parametrize("name,H,new", [("mitchell07", 4, [1, 1]), ("native", 8, [3, 1]), ("exact09", 2, [9, 2]), ("perturbed08", 8, [12, 1])])
def test_missing_pages_and_special_values(am, name, H, new):
    """Pages that the table does not name are seen by no row; NaN and Inf in
    them, behind a sequence's length or behind a chunk's mask have no part;
    a NaN key that is seen makes its rows NaN, and only those."""
    mul = load(am, name)
    k_len, page, K, D = [100, 40], 16, 1, 64
    kp, vp, table = cache(8200, k_len, page, K, D, spare=4)
    q = normal(8201, (sum(new), H, D))
    used = set(table[table >= 0].tolist())
    for x in set(range(kp.shape[0])) - used:
        kp[x], vp[x] = np.nan, np.inf                       # pages of nobody
    kp[table[0, 6], 100 % page:] = np.nan                   # behind the length
    vp[table[0, 6], 100 % page:] = np.inf
    check(am, mul, q, kp, vp, table, new, k_len, what="pages of nobody")
    for wrong in (-1, -(1 << 31), kp.shape[0], (1 << 31) - 1):
        t = table.copy()
        t[0, 2] = wrong
        t[1, 0] = wrong
        check(am, mul, q, kp, vp, t, new, k_len, what=f"page {wrong}")
    t = np.full_like(table, -1)
    o, lse = check(am, mul, q, kp, vp, t, new, k_len, what="no page")
    assert (o == 0).all() and np.isneginf(lse).all()
    last = new[0] > 1
    kp[table[0, 6], 99 % page] = np.nan                     # seen by the first sequence's last token only
    vp[table[0, 6], 99 % page] = np.inf
    o, lse = check(am, mul, q, kp, vp, table, new, k_len, what="NaN key")
    assert np.isnan(o[new[0] - 1]).all() and (not last or np.isfinite(o[: new[0] - 1]).all())


@pytest.mark.parametrize("E", [5, 8])
def test_checked_path(am, E, monkeypatch):
    mul = load(am, "perturbed08")
    am.approx_exponent_bits_set(E)
    try:
        new, k_len = [1, 11], [200, 90]
        kp, vp, table = cache(8300, k_len, 16, 2, 48)
        q = normal(8301, (sum(new), 4, 48))
        monkeypatch.setenv("APPROX_FORCE_CHECKED", "1")
        o, lse = check(am, mul, q, kp, vp, table, new, k_len, E=E, what="checked")
        monkeypatch.delenv("APPROX_FORCE_CHECKED")
        o2, lse2 = check(am, mul, q, kp, vp, table, new, k_len, E=E, what="fast")
        assert np.array_equal(lse.view(np.uint32), lse2.view(np.uint32))
    finally:
        am.approx_exponent_bits_set(8)


def test_tiny_and_huge_values(am):
    """Operands outside the fast range in the cache alone, in part of it."""
    mul = load(am, "mitchell07")
    new, k_len = [1, 2], [300, 70]
    kp, vp, table = cache(8400, k_len, 16, 2, 64)
    q = normal(8401, (sum(new), 4, 64))
    vp[table[0, 3]] *= np.float32(2.0 ** -110)
    vp[table[0, 4]] *= np.float32(2.0 ** 70)
    kp[table[1, 1]] *= np.float32(2.0 ** -90)
    check(am, mul, q, kp, vp, table, new, k_len, what="ranges")


def test_wrong_lengths_stay_inside(am):
    """Lengths beyond the table's row or below zero are clamped."""
    mul = load(am, "mitchell07")
    kp, vp, table = cache(8500, [64, 64], 16, 1, 64, spare=0)
    q = normal(8501, (2, 2, 64))
    out = am.attention_paged(dev(q), dev(kp), dev(vp), dev(table), dev(np.array([0, 1, 2], np.int32)), dev(np.array([1 << 30, -7], np.int32)))
    torch.cuda.synchronize()
    want, _, mag = reference(q, kp, vp, table, [1, 1], [64, 0], True, 0.125, *mul)
    ref.near(out.cpu().numpy(), want, mag, 64)


def test_offsets_beyond_32_bits(am):
    """A cache of more than 2^31 elements (and 2^32 bytes): the last pages."""
    mul = load(am, "mitchell07")
    page, K, D = 64, 8, 128
    pages = (1 << 31) // (page * K * D) + 3
    kp = torch.zeros((pages, page, K, D), device="cuda")
    vp = torch.zeros((pages, page, K, D), device="cuda")
    small_k, small_v, _ = cache(8600, [100], page, K, D, spare=0)
    q = normal(8601, (1, 8, D))
    table = np.array([[pages - 1, pages - 2]], np.int32)
    for i, x in enumerate((pages - 1, pages - 2)):
        kp[x], vp[x] = dev(small_k[i]), dev(small_v[i])
    out = am.attention_paged(dev(q), kp, vp, dev(table), dev(np.array([0, 1], np.int32)), dev(np.array([100], np.int32)))
    torch.cuda.synchronize()
    want, _, mag = reference(q, small_k, small_v, np.array([[0, 1]], np.int32), [1], [100], True, D ** -0.5, *mul)
    ref.near(out.cpu().numpy(), want, mag, 100)


def test_untouched_rows_streams_and_graph(am):
    """Rows of no sequence keep what o holds; replays of a captured call, with
    new lengths and cache contents between them, give what calls give."""
    mul = load(am, "mitchell07")
    k_len, page, H, K, D = [200, 90], 16, 8, 2, 64
    kp, vp, table = cache(8700, [256, 256], page, K, D)
    q = normal(8701, (6, H, D))
    t = [dev(x) for x in (q, kp, vp, table, np.array([1, 2, 4], np.int32), np.array(k_len, np.int32))]
    out = torch.full(q.shape, 3.0, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        am.attention_paged(*t, out=out, stream=s)
    torch.cuda.synchronize()
    assert (out[0] == 3).all() and (out[4:] == 3).all()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        am.attention_paged(*t, out=out, stream=s)
    for rep, lens in enumerate(([200, 90], [201, 91], [256, 5])):
        t[5].copy_(dev(np.array(lens, np.int32)))
        t[0].copy_(dev(normal(8710 + rep, q.shape)))
        out.fill_(3.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        qq = t[0].cpu().numpy()[1:4]
        want, _, mag = reference(qq, kp, vp, table, [1, 2], lens, True, D ** -0.5, *mul)
        ref.near(out.cpu().numpy()[1:4], want, mag, max(lens), str(rep))
        with torch.cuda.stream(s):
            am.attention_paged(dev(q), *t[1:], stream=s)
        torch.cuda.synchronize()


def test_binding_refuses(am):
    load(am, "mitchell07")
    kp, vp, table = cache(8800, [20], 16, 2, 64)
    args = [dev(x) for x in (normal(8801, (1, 4, 64)), kp, vp, table, np.array([0, 1], np.int32), np.array([20], np.int32))]
    for i, bad in ((1, args[1][:, :, :, :32]), (2, args[2][:1]), (3, args[3].long()), (4, args[4][:1]), (5, args[5].float())):
        with pytest.raises(ValueError):
            am.attention_paged(*[bad if j == i else a for j, a in enumerate(args)])
