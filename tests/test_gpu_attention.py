"""Attention with approximate products over packed prompts, forward and
backward, against the 64-bit definition (attention_ref) on the oracle's
products: table widths in LDS and in global memory, the native multiplier,
narrow formats, head layouts, odd dimensions, ragged and empty sequences,
strided and unaligned tensors, special values in and behind the mask, wrong
offsets, streams and graphs."""
import numpy as np
import pytest

import attention_ref as ref
import oracle
from datagen import PERTURB_SEED, normal, pm_one

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def am():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import approximate_multiplier_dnn_amd as m
    yield m
    m.approx_exponent_bits_set(8)
    m.approx_lut_load(oracle.lut_generate(7, "mitchell"), 7)


def load(am, name):
    """Loads the named multiplier; (lut or None, M)."""
    if name == "native":
        am.approx_native_load()
        return None, 0
    model, M = name[:-2].rstrip("0"), int(name[-2:])
    if model == "perturbed":
        lut = oracle.lut_perturb(M, oracle.lut_generate(M, "exact"), pm_one(PERTURB_SEED, 1 << (2 * M)))
    elif model == "skew":                       # first and second operand not exchangeable
        lut = oracle.lut_generate(M, "exact")
        lut = lut.reshape(1 << M, 1 << M).copy()
        lut[: 1 << (M - 1)] ^= 1
        lut = lut.reshape(-1)
    else:
        lut = oracle.lut_generate(M, model)
    am.approx_lut_load(lut, M)
    return lut, M


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def inputs(seed, q_lens, k_lens, H, K, D):
    return (normal(seed, (sum(q_lens), H, D)), normal(seed + 1, (sum(k_lens), K, D)), normal(seed + 2, (sum(k_lens), K, D)),
            normal(seed + 3, (sum(q_lens), H, D)))


def forward_and_check(am, mul, q, k, v, cu_q, cu_k, causal, scale=None, E=8, what=""):
    lut, M = mul
    o, lse = am.attention_fwd(dev(q), dev(k), dev(v), dev(cu_q), dev(cu_k), causal=causal, scale=scale)
    torch.cuda.synchronize()
    o, lse = o.cpu().numpy(), lse.cpu().numpy()
    scale = q.shape[2] ** -0.5 if scale is None else scale
    want, want_lse, mag = ref.attention_packed(q, k, v, cu_q, cu_k, causal, scale, lut, M, E)
    n = int(np.diff(cu_k).max(initial=0))
    # native: a score may differ by one rounding from the reference's double one
    extra = 2.0 ** -23 * (1 + 8 * scale * q.shape[2]) if lut is None else 0.0
    ref.near(o, want, np.where(np.isnan(mag), 0.0, mag), n, what + " o", extra)
    fin = np.isfinite(want_lse)
    assert np.array_equal(np.isnan(lse), np.isnan(want_lse)) and np.array_equal(np.isinf(lse), np.isinf(want_lse)), what
    assert (np.abs(lse[fin] - want_lse[fin]) <= (2.0 ** -23 + extra) * (1 + np.abs(want_lse[fin]))).all(), what
    return o, lse


def backward_and_check(am, mul, q, k, v, dout, o, lse, cu_q, cu_k, causal, scale=None, E=8, what=""):
    lut, M = mul
    got = am.attention_bwd(dev(dout), dev(q), dev(k), dev(v), dev(o), dev(lse), dev(cu_q), dev(cu_k), causal=causal, scale=scale)
    torch.cuda.synchronize()
    scale = q.shape[2] ** -0.5 if scale is None else scale
    want, mags = ref.attention_packed_grad(q, k, v, o, lse, dout, cu_q, cu_k, causal, scale, lut, M, E)
    n = int(max(np.diff(cu_k).max(initial=0), np.diff(cu_q).max(initial=0))) * (q.shape[1] // k.shape[1])
    for x, w, m, name in zip(got, want, mags, ("dq", "dk", "dv")):
        # native: a one-rounding difference of a score or of dP (which cancels
        # against D) moves dS by up to that rounding of their magnitude
        if lut is None:
            m = m + np.abs(m).max(initial=0.0)
        ref.near(x.cpu().numpy(), w, m, n, f"{what} {name}", 2.0 ** -18 if lut is None else 0.0)
    return [x.cpu().numpy() for x in got]


CASES = [
    # multiplier, query lengths, key lengths, heads, kv heads, dim, causal
    ("mitchell07", [1], [1], 1, 1, 64, True),
    ("mitchell07", [5, 1, 70, 33], [5, 1, 70, 33], 4, 2, 64, True),
    ("mitchell07", [5, 0, 70, 33], [9, 3, 70, 0], 4, 4, 64, False),
    ("mitchell07", [130], [130], 3, 1, 40, True),
    ("mitchell07", [40, 3], [150, 20], 8, 2, 64, True),           # fewer queries than keys
    ("mitchell07", [50, 9], [20, 4], 2, 2, 32, True),             # rows that see no key
    ("skew07", [66, 31], [66, 31], 6, 2, 128, True),
    ("skew07", [37], [90], 2, 2, 33, False),                      # odd dimension
    ("exact03", [64, 64], [64, 64], 2, 1, 16, True),
    ("exact01", [20], [20], 2, 1, 1, True),
    ("perturbed08", [65, 17], [65, 17], 4, 2, 64, True),
    ("perturbed08", [40], [70], 4, 1, 96, True),
    ("exact09", [50], [50], 2, 1, 64, True),
    ("mitchell11", [30, 8], [30, 8], 2, 2, 80, True),
    ("native", [70, 12], [70, 12], 4, 2, 64, True),
    ("native", [33], [50], 2, 1, 100, False),
]


@pytest.mark.parametrize("columns", ["8", "16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}-{c[3]}x{c[4]}x{c[5]}-{'causal' if c[6] else 'full'}")
def test_forward_and_backward(am, case, columns, monkeypatch):
    """Both widths of a wave's share (the library takes 8 for small calls)."""
    monkeypatch.setenv("APPROX_ATTENTION_COLUMNS", columns)
    name, ql, kl, H, K, D, causal = case
    mul = load(am, name)
    q, k, v, dout = inputs(9000 + 17 * D + H, ql, kl, H, K, D)
    cu_q, cu_k = ref.packed(ql), ref.packed(kl)
    o, lse = forward_and_check(am, mul, q, k, v, cu_q, cu_k, causal, what=str(case))
    backward_and_check(am, mul, q, k, v, dout, o, lse, cu_q, cu_k, causal, what=str(case))


@pytest.mark.parametrize("columns", ["8", "16"])
def test_long_reduction_in_chunks(am, columns, monkeypatch):
    """Few rows over many keys (and many rows over few keys, backward): the
    ranges are split into chunks and joined."""
    monkeypatch.setenv("APPROX_ATTENTION_COLUMNS", columns)
    mul = load(am, "mitchell07")
    for ql, kl in (([3], [1500]), ([700], [5])):
        q, k, v, dout = inputs(9100 + ql[0], ql, kl, 2, 1, 64)
        cu_q, cu_k = ref.packed(ql), ref.packed(kl)
        o, lse = forward_and_check(am, mul, q, k, v, cu_q, cu_k, False, what="long")
        backward_and_check(am, mul, q, k, v, dout, o, lse, cu_q, cu_k, False, what="long")


@pytest.mark.parametrize("columns", ["8", "16"])
@pytest.mark.parametrize("dim", [24, 32])
def test_small_heads_with_a_wide_table(am, dim, columns, monkeypatch):
    """M = 8 and heads of up to 32: the backward pass takes either width."""
    monkeypatch.setenv("APPROX_ATTENTION_COLUMNS", columns)
    mul = load(am, "perturbed08")
    ql, kl = [70, 1, 33], [70, 20, 33]
    q, k, v, dout = inputs(9300 + dim, ql, kl, 4, 2, dim)
    cu_q, cu_k = ref.packed(ql), ref.packed(kl)
    o, lse = forward_and_check(am, mul, q, k, v, cu_q, cu_k, True, what="small heads")
    backward_and_check(am, mul, q, k, v, dout, o, lse, cu_q, cu_k, True, what="small heads")


@pytest.mark.parametrize("causal", [True, False])
def test_more_sequences_than_a_wave(am, causal):
    """Seventy-odd sequences, empty ones among them."""
    mul = load(am, "mitchell07")
    lens = [int(n) for n in np.random.RandomState(7).randint(0, 9, 75)]
    lens[3], lens[70] = 0, 70
    q, k, v, dout = inputs(9150, lens, lens, 2, 1, 32)
    cu = ref.packed(lens)
    o, lse = forward_and_check(am, mul, q, k, v, cu, cu, causal, what="many")
    backward_and_check(am, mul, q, k, v, dout, o, lse, cu, cu, causal, what="many")


def test_rising_scores_move_the_maximum(am):
    """Scores that rise by tens of powers of two along the keys: every block
    raises the running maximum, and the early weights vanish (below 2^-64)."""
    mul = load(am, "mitchell07")
    n, D = 200, 64
    q, k, v, dout = inputs(9200, [n], [n], 1, 1, D)
    q = np.abs(q)
    k = np.abs(k) * (1 + np.arange(n, dtype=np.float32)[:, None, None]) / 8
    cu = ref.packed([n])
    o, lse = forward_and_check(am, mul, q, k, v, cu, cu, False, what="rising")
    backward_and_check(am, mul, q, k, v, dout, o, lse, cu, cu, False, what="rising")


@pytest.mark.parametrize("E", [5, 8])
def test_checked_path(am, E, monkeypatch):
    """The checked path (forced; and a format with 5 exponent bits, whose
    weights below its range are zero) against the definition; where the fast
    path may run, both give the same bits."""
    mul = load(am, "perturbed08")
    am.approx_exponent_bits_set(E)
    try:
        q, k, v, dout = inputs(9300, [50, 21], [50, 21], 4, 2, 48)
        cu = ref.packed([50, 21])
        monkeypatch.setenv("APPROX_FORCE_CHECKED", "1")
        o, lse = forward_and_check(am, mul, q, k, v, cu, cu, True, E=E, what="checked")
        g = backward_and_check(am, mul, q, k, v, dout, o, lse, cu, cu, True, E=E, what="checked")
        monkeypatch.delenv("APPROX_FORCE_CHECKED")
        o2, lse2 = forward_and_check(am, mul, q, k, v, cu, cu, True, E=E, what="fast")
        g2 = backward_and_check(am, mul, q, k, v, dout, o, lse, cu, cu, True, E=E, what="fast")
        for a, b in zip([o, lse] + g, [o2, lse2] + g2):
            assert np.array_equal(a.view(np.uint32), b.view(np.uint32))
    finally:
        am.approx_exponent_bits_set(8)


@pytest.mark.parametrize("name", ["mitchell07", "perturbed08", "exact09", "native"])
def test_special_values_behind_the_mask(am, name):
    """NaN, infinities and the largest finite values in keys and values that a
    row does not see (later tokens, other sequences) have no part in its
    result, nor in the gradients."""
    mul = load(am, name)
    n = 24
    q, k, v, dout = inputs(9400, [n, 7], [n, 7], 2, 1, 64)
    k[n - 1, 0, :3] = [np.nan, np.inf, -np.inf]
    v[n - 1, 0, :4] = [np.nan, np.inf, -np.inf, np.finfo(np.float32).max]
    cu = ref.packed([n, 7])
    o, lse = forward_and_check(am, mul, q, k, v, cu, cu, True, what="masked specials")
    assert np.isfinite(o[: n - 1]).all() and np.isfinite(o[n:]).all() and np.isnan(o[n - 1]).all()
    # the row that sees them aside, the gradients are finite
    q2, d2, o2, l2 = (x.copy() for x in (q, dout, o, lse))
    o2[n - 1], l2[n - 1], d2[n - 1] = 0.0, 0.0, 0.0
    lut, M = mul
    got = am.attention_bwd(dev(d2), dev(q2), dev(k), dev(v), dev(o2), dev(l2), dev(cu), dev(cu), causal=True)
    torch.cuda.synchronize()
    dq = got[0].cpu().numpy()
    assert np.isfinite(dq[: n - 1]).all() and np.isfinite(dq[n:]).all()


def test_infinite_and_overflowing_scores(am):
    """A +Inf score (an overflowing sum among them) gives NaN; -Inf scores
    weigh nothing; a row of -Inf scores is an empty one."""
    mul = load(am, "mitchell07")
    D = 64
    q = np.ones((3, 1, D), np.float32)
    k = normal(9500, (6, 1, D))
    v = normal(9501, (6, 1, D))
    cu_q, cu_k = ref.packed([1, 1, 1]), ref.packed([2, 2, 2])
    k[0] = np.finfo(np.float32).max                      # sums to +Inf
    k[2] = -np.inf                                       # -Inf next to an ordinary score
    k[4:] = -np.inf                                      # nothing but -Inf
    o, lse = forward_and_check(am, mul, q, k, v, cu_q, cu_k, False, what="infinite scores")
    assert np.isnan(o[0]).all() and np.isfinite(o[1]).all() and (o[2] == 0).all() and np.isneginf(lse[2]).all()


def test_tiny_and_huge_operands(am):
    """Products below and above the normal range take the checked path."""
    mul = load(am, "mitchell07")
    q, k, v, dout = inputs(9600, [40], [40], 2, 2, 64)
    cu = ref.packed([40])
    v = v * np.float32(2.0 ** -100)
    o, lse = forward_and_check(am, mul, q, k, v, cu, cu, True, what="tiny values")
    v = v * np.float32(2.0 ** 100) * np.float32(2.0 ** 60)
    o, lse = forward_and_check(am, mul, q, k, v, cu, cu, True, what="huge values")
    backward_and_check(am, mul, q, k, v, dout, o, lse, cu, cu, True, what="huge values")


def test_views_and_untouched_rows(am):
    """Parts of one projection's output, at an address that is not 16-byte
    aligned, as inputs, and gradients into such parts; rows before the first
    and behind the last sequence keep what the outputs hold."""
    mul = load(am, "mitchell07")
    H, K, D, T = 4, 2, 64, 60
    row = (H + 2 * K) * D
    for shift, D2 in ((0, D), (1, 33)):
        row = (H + 2 * K) * D2 + 4
        flat = torch.zeros(T * row + 8, device="cuda")
        x = normal(9700 + D2, (T, row))
        flat[shift: shift + T * row] = dev(x).reshape(-1)
        both = flat[shift: shift + T * row].view(T, row)
        parts = [both[:, : H * D2].view(T, H, D2), both[:, H * D2: (H + K) * D2].view(T, K, D2),
                 both[:, (H + K) * D2: (H + 2 * K) * D2].view(T, K, D2)]
        cu = np.array([3, 20, 50], np.int32)
        out = torch.full((T, H, D2), 7.0, device="cuda")
        lse = torch.full((T, H), 7.0, device="cuda")
        am.attention_fwd(*parts, dev(cu), dev(cu), causal=True, out=out, lse=lse)
        torch.cuda.synchronize()
        q, k, v = (p.cpu().numpy() for p in parts)
        want, want_lse, mag = ref.attention_packed(q, k, v, cu, cu, True, D2 ** -0.5, *mul)
        ref.near(out.cpu().numpy()[3:50], want[3:50], mag[3:50], 30, "views")
        assert (out[:3] == 7).all() and (out[50:] == 7).all() and (lse[:3] == 7).all() and (lse[50:] == 7).all()
        dout = normal(9701, (T, H, D2))
        grads = torch.full((T, row), 7.0, device="cuda")
        gp = [grads[:, : H * D2].view(T, H, D2), grads[:, H * D2: (H + K) * D2].view(T, K, D2),
              grads[:, (H + K) * D2: (H + 2 * K) * D2].view(T, K, D2)]
        am.attention_bwd(dev(dout), *parts, out, lse, dev(cu), dev(cu), causal=True, dq=gp[0], dk=gp[1], dv=gp[2])
        torch.cuda.synchronize()
        wants, mags = ref.attention_packed_grad(q, k, v, out.cpu().numpy(), lse.cpu().numpy(), dout, cu, cu, True, D2 ** -0.5, *mul)
        for g, w, m in zip(gp, wants, mags):
            g = g.cpu().numpy()
            ref.near(g[3:50], w[3:50], m[3:50], 60, "views")
            assert (g[:3] == 7).all() and (g[50:] == 7).all()
        assert (grads[:, (H + 2 * K) * D2:] == 7).all()


def test_wrong_offsets_stay_inside(am):
    """Descending, negative and too large offsets are clamped: the call ends,
    and a well-formed prefix of sequences gets its result."""
    mul = load(am, "mitchell07")
    q, k, v, dout = inputs(9800, [40], [40], 2, 1, 64)
    for bad in ([0, 20, 10, 60], [-5, 20, 40, 40], [0, 20, 1 << 30, -(1 << 30)], [50, 60, 70, 80], [0, 20, 40, 0]):
        cu = np.array(bad, np.int32)
        out = torch.zeros((40, 2, 64), device="cuda")
        lse = torch.zeros((40, 2), device="cuda")
        am.attention_fwd(dev(q), dev(k), dev(v), dev(cu), dev(cu), out=out, lse=lse)
        am.attention_bwd(dev(dout), dev(q), dev(k), dev(v), out, lse, dev(cu), dev(cu))
        torch.cuda.synchronize()
        if bad[1] == 20 and bad[0] <= 0:
            want, _, mag = ref.attention_packed(q[:20], k[:20], v[:20], ref.packed([20]), ref.packed([20]), True, 0.125, *mul)
            ref.near(out[:20].cpu().numpy(), want, mag, 20, str(bad))


def test_gradient_against_differences(am):
    """Native multiplier: the gradients along random directions against
    central differences of the 64-bit forward pass."""
    am.approx_native_load()
    n, H, K, D, h = 30, 2, 1, 32, 1e-4
    q, k, v, dout = inputs(9900, [n], [n], H, K, D)
    cu = ref.packed([n])

    def loss(q, k, v):
        total = 0.0
        for i in range(H):
            s = np.where(ref.causal_mask(n, n), q[:, i] @ k[:, 0].T * D ** -0.5, -np.inf)
            p = np.exp(s - s.max(1, keepdims=True))
            total += (dout[:, i] * (p / p.sum(1, keepdims=True) @ v[:, 0])).sum()
        return total

    o, lse = am.attention_fwd(dev(q), dev(k), dev(v), dev(cu), dev(cu))
    grads = am.attention_bwd(dev(dout), dev(q), dev(k), dev(v), o, lse, dev(cu), dev(cu))
    base = [x.astype(np.float64) for x in (q, k, v)]
    for i in range(3):
        way = normal(9950 + i, base[i].shape).astype(np.float64)
        hi, lo = [x.copy() for x in base], [x.copy() for x in base]
        hi[i] += h * way
        lo[i] -= h * way
        slope = (loss(*hi) - loss(*lo)) / (2 * h)
        g = grads[i].cpu().numpy().astype(np.float64)
        # FP32 sums over n rows and D elements, and h^2 of the differences
        assert abs((g * way).sum() - slope) <= 2.0 ** -16 * np.abs(g * way).sum() + 1e-5, i


def test_same_bits_on_streams_and_in_graphs(am):
    """Calls on two streams at once, and replays of a captured forward and
    backward pass with other calls between, give the bits of a call alone."""
    load(am, "mitchell07")
    sets = []
    for seed, lens in ((9990, [70, 5, 130]), (9995, [200])):
        q, k, v, dout = inputs(seed, lens, lens, 4, 2, 64)
        sets.append([dev(x) for x in (q, k, v, dout, ref.packed(lens))])

    def step(t, outs=None):
        q, k, v, dout, cu = t
        if outs is None:
            outs = [torch.empty_like(q), torch.empty(q.shape[:2], device="cuda"), torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)]
        s = torch.cuda.current_stream()
        am.attention_fwd(q, k, v, cu, cu, out=outs[0], lse=outs[1], stream=s)
        am.attention_bwd(dout, q, k, v, outs[0], outs[1], cu, cu, dq=outs[2], dk=outs[3], dv=outs[4], stream=s)
        return outs

    alone = [[x.clone() for x in step(t)] for t in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for rep in range(3):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i].append(step(sets[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for outs in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(outs, alone[i]))
    outs = got[0][0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=streams[0]):
        step(sets[0], outs)
    for rep in range(3):
        for x in outs:
            x.fill_(-1.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, alone[0])), rep
        with torch.cuda.stream(streams[0]):
            step(sets[1])
        torch.cuda.synchronize()


def test_binding_refuses(am):
    load(am, "mitchell07")
    q, k, v, dout = (dev(x) for x in inputs(9001, [8], [8], 4, 2, 16))
    cu = dev(ref.packed([8]))
    with pytest.raises(ValueError):
        am.attention_fwd(q.transpose(0, 1), k, v, cu, cu)
    with pytest.raises(ValueError):
        am.attention_fwd(q, k, v[:4], cu, cu)
    with pytest.raises(ValueError):
        am.attention_fwd(q, k, v, cu.long(), cu)
    with pytest.raises(ValueError):
        am.attention_fwd(q, k, v, cu, cu[:1])
    with pytest.raises(ValueError):
        am.attention_fwd(q, k.cpu(), v, cu, cu)
    with pytest.raises(TypeError):
        am.attention_fwd(q.half(), k, v, cu, cu)
    with pytest.raises(am.ApproxError) as e:
        am.attention_fwd(q[:, :3], k, v, cu, cu)
    assert e.value.status == am.APPROX_EINVAL                   # 3 heads over 2 kv heads
    with pytest.raises(am.ApproxError) as e:
        am.attention_fwd(*(torch.zeros(4, 1, 130, device="cuda") for _ in range(3)), cu, cu)
    assert e.value.status == am.APPROX_EUNSUPPORTED
