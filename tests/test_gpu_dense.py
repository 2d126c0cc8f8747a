"""Dense layer with bias, activation and residual, forward and backward,
against 64-bit sums of the oracle's products; and a transformer block of the
layer calls, forward and backward and token by token."""
import math

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
    m.approx_lut_load(oracle.lut_generate(7, "mitchell"), 7)


erfc = np.vectorize(math.erfc, otypes=[float])


def act64(z, act):
    if act == "relu":
        return np.where(z < 0, 0.0, z)
    if act == "gelu":
        return 0.5 * z * erfc(-z / math.sqrt(2))
    return z / (1 + np.exp(-z)) if act == "silu" else z


def slope64(z, act):
    if act == "relu":
        return (z > 0).astype(float)
    if act == "gelu":
        return 0.5 * erfc(-z / math.sqrt(2)) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        s = 1 / (1 + np.exp(-z))
        return s * (1 + z * (1 - s))
    return np.ones_like(z)


def product(a, b, mul):
    """(sums, sums of magnitudes) of table products, float64."""
    lut, M = mul
    return oracle.gemm(np.ascontiguousarray(a), np.ascontiguousarray(b), lut, M)


CASES = [
    # multiplier, m, n, k, activation, bias, residual
    ("mitchell07", 1, 1024, 300, "gelu", True, False),
    ("mitchell07", 1, 5, 1, "silu", True, True),
    ("mitchell07", 33, 70, 130, "gelu", True, True),
    ("mitchell07", 300, 96, 200, "relu", True, True),
    ("mitchell07", 300, 201, 64, "none", True, False),
    ("mitchell07", 64, 64, 64, "silu", False, True),
    ("perturbed08", 130, 48, 500, "silu", True, True),
    ("exact09", 70, 40, 60, "gelu", False, False),
    ("native", 100, 64, 90, "gelu", True, True),
    ("mitchell07", 20, 8, 0, "gelu", True, True),                 # no reduction: the bias alone
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c))
def test_forward(am, case):
    name, m, n, k, act, with_bias, with_res = case
    mul = load(am, name)
    x, w = normal(7000 + m, (m, k)), normal(7001 + n, (k, n), std=1 / math.sqrt(max(k, 1)))
    bias = normal(7002, (n,)) if with_bias else None
    res = normal(7003, (m, n)) if with_res else None
    z, mag = product(x, w, mul) if k else (np.zeros((m, n)), np.zeros((m, n)))
    if bias is not None:
        z, mag = z + bias, mag + np.abs(bias)
    y = act64(z, act)
    args = dict(bias=None if bias is None else dev(bias), act=act, residual=None if res is None else dev(res))
    got, got_z = am.dense_fwd(dev(x), dev(w), keep_z=True, **args)
    alone = am.dense_fwd(dev(x), dev(w), **args)
    torch.cuda.synchronize()
    assert torch.equal(got, alone)
    # z: FP32 sums and the bias's addition; |act'| <= 1.13; FP32 erfc and exp
    # within 4 units of the last place, the residual's addition one more
    ref.near(got_z.cpu().numpy(), z, mag, k, "z")
    bound = 1.13 * (k + 40) * 2.0 ** -24 * mag + 8 * 2.0 ** -24 * (np.abs(y) + np.abs(z) * 0 + (np.abs(res) if with_res else 0))
    err = np.abs(got.cpu().numpy() - (y + (res if with_res else 0)))
    assert (err <= bound + 1e-30).all(), (err / np.maximum(bound, 1e-30)).max()


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c))
def test_backward(am, case):
    name, m, n, k, act, with_bias, _ = case
    mul = load(am, name)
    x, w = normal(7100 + m, (m, k)), normal(7101 + n, (k, n))
    dy, z = normal(7102, (m, n)), normal(7103, (m, n), std=2)
    z.flat[:4] = [0.0, -0.0, -9.0, 30.0][: z.size]
    dz = (dy.astype(np.float64) * slope64(z.astype(np.float64), act)).astype(np.float32)
    dx, dw, db = am.dense_bwd(dev(dy), dev(x), dev(w), z=dev(z), act=act, bias=with_bias)
    torch.cuda.synchronize()
    if k:
        for got, (want, mag), terms in ((dx, product(dz, w.T, mul), n), (dw, product(x.T, dz, mul), m)):
            ref.near(got.cpu().numpy(), want, mag, terms)
    if with_bias:
        want = dz.astype(np.float64).sum(0)
        assert (np.abs(db.cpu().numpy() - want) <= 2.0 ** -24 * np.abs(want) + 1e-12 * np.abs(dz).sum(0)).all()
    else:
        assert db is None


def test_special_values(am):
    """NaN and infinities of z pass the activations as the formulas have them."""
    load(am, "mitchell07")
    bias = np.array([np.nan, np.inf, -np.inf, 1.0, -0.0, 3e38, -3e38, -100.0], np.float32)
    x, w = torch.zeros(2, 4, device="cuda"), torch.zeros(4, 8, device="cuda")
    for act in ("none", "relu", "gelu", "silu"):
        y = am.dense_fwd(x, w, bias=dev(bias), act=act).cpu().numpy()[0]
        assert np.isnan(y[0]) and y[1] == np.inf and y[5] == np.float32(3e38)
        assert y[6] == (bias[6] if act == "none" else 0.0)
        # -Inf times Phi(-Inf) = 0, and -Inf / Inf, are NaN
        assert np.isnan(y[2]) if act in ("gelu", "silu") else y[2] == (-np.inf if act == "none" else 0.0)


def test_views_subsets_and_graph(am):
    """Leading dimensions and unaligned views; outputs left out; a captured
    backward pass replayed with other calls between."""
    mul = load(am, "mitchell07")
    m, n, k = 90, 35, 50
    x, w, dy, z, res = normal(7200, (m, k + 3)), normal(7201, (k, n + 2)), normal(7202, (m, n + 1)), normal(7203, (m, n)), normal(7204, (m, n + 5))
    dx_, dw_, ddy, dz_, dres = (dev(a) for a in (x, w, dy, z, res))
    y = am.dense_fwd(dx_[:, 1:k + 1], dw_[:, 2:], act="silu", residual=dres[:, 3:n + 3])
    torch.cuda.synchronize()
    zz, mag = product(x[:, 1:k + 1], w[:, 2:], mul)
    err = np.abs(y.cpu().numpy() - (act64(zz, "silu") + res[:, 3:n + 3]))
    assert (err <= 1.13 * (k + 40) * 2.0 ** -24 * mag + 16 * 2.0 ** -24 * (np.abs(zz) + np.abs(res[:, 3:n + 3]))).all()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [torch.empty(m, k, device="cuda"), torch.empty(k, n, device="cuda")]

    def back():
        return am.dense_bwd(ddy[:, 1:], dx_[:, 1:k + 1], dw_[:, 2:], z=dz_, act="gelu", bias=True, dx=outs[0], dw=outs[1], stream=s)

    with torch.cuda.stream(s):
        db = back()[2]
    torch.cuda.synchronize()
    eager = [t.clone() for t in outs] + [db.clone()]
    dz = (dy[:, 1:].astype(np.float64) * slope64(z.astype(np.float64), "gelu")).astype(np.float32)
    want, mag = product(dz, w[:, 2:].T, mul)
    ref.near(outs[0].cpu().numpy(), want, mag, n)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        db = back()[2]
    for rep in range(3):
        for t in outs + [db]:
            t.fill_(-1.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs + [db], eager)), rep
        with torch.cuda.stream(s):
            am.dense_bwd(ddy[:, 1:].contiguous() * 2, dx_[:, 1:k + 1], dw_[:, 2:], z=dz_, act="silu", bias=True, stream=s)
        torch.cuda.synchronize()
    # left out: db alone, dw alone
    L, st = am.lib(), torch.cuda.current_stream().cuda_stream
    only = torch.empty(n, device="cuda")
    assert L.approx_dense_bwd(m, n, k, None, k, None, n, dz_.data_ptr(), n, 2, ddy[:, 1:].data_ptr(), n + 1, None, k, None, n, only.data_ptr(), st) == 0
    torch.cuda.synchronize()
    assert torch.equal(only, eager[2])


def test_no_rows(am):
    """A batch without rows: nothing forward, zero gradients of w and the bias."""
    load(am, "mitchell07")
    x, w, e = torch.zeros(0, 5, device="cuda"), dev(normal(7290, (5, 6))), torch.zeros(0, 6, device="cuda")
    assert am.dense_fwd(x, w, act="gelu").shape == (0, 6)
    dx, dw, db = am.dense_bwd(e, x, w, z=e, act="gelu", bias=True)
    torch.cuda.synchronize()
    assert dx.shape == (0, 5) and (dw == 0).all() and (db == 0).all()


def test_gradient_against_differences(am):
    """Native multiplier: a layer's gradients along random directions against
    central differences of the 64-bit layer."""
    am.approx_native_load()
    m, n, k, h = 12, 9, 20, 1e-5
    x, w, b, dy = normal(7300, (m, k)), normal(7301, (k, n), std=0.3), normal(7302, (n,)), normal(7303, (m, n))
    for act in ("gelu", "silu", "none"):
        def loss(x, w, b):
            return (dy * act64(x @ w + b, act)).sum()

        _, z = am.dense_fwd(dev(x), dev(w), bias=dev(b), act=act, keep_z=True)
        grads = am.dense_bwd(dev(dy), dev(x), dev(w), z=z, act=act, bias=True)
        base = [t.astype(np.float64) for t in (x, w, b)]
        for i in range(3):
            way = normal(7310 + i, base[i].shape).astype(np.float64)
            hi, lo = [t.copy() for t in base], [t.copy() for t in base]
            hi[i] += h * way
            lo[i] -= h * way
            slope = (loss(*hi) - loss(*lo)) / (2 * h)
            g = grads[i].cpu().numpy().astype(np.float64)
            assert abs((g * way).sum() - slope) <= 2.0 ** -18 * np.abs(g * way).sum() + 1e-6, (act, i)


def test_block_trains_and_serves(am):
    """A transformer block of the layer calls (projection, attention, output
    projection with its residual, feed-forward): gradients by the chain of the
    layers' own backward calls against float64 with the native multiplier; and
    the last token's output computed over a paged cache is the prompt's."""
    am.approx_native_load()
    H, K, D, page = 4, 2, 16, 8
    d, lens = H * D, [19, 8]
    T, kvd = sum(lens), K * D
    cu = dev(ref.packed(lens))
    x = dev(normal(7400, (T, d)))
    W = {name: dev(normal(7401 + i, shape, std=0.15)) for i, (name, shape) in
         enumerate({"qkv": (d, d + 2 * kvd), "out": (d, d), "up": (d, 96), "down": (96, d)}.items())}
    bias = dev(normal(7410, (96,)))
    dy = dev(normal(7411, (T, d)))

    def split(t):
        return t[:, :d].view(-1, H, D), t[:, d:d + kvd].view(-1, K, D), t[:, d + kvd:].view(-1, K, D)

    qkv = am.dense_fwd(x, W["qkv"])
    o, lse = am.attention_fwd(*split(qkv), cu, cu)
    a = am.dense_fwd(o.view(T, d), W["out"], residual=x)
    u, z = am.dense_fwd(a, W["up"], bias=bias, act="gelu", keep_z=True)
    y = am.dense_fwd(u, W["down"], residual=a)

    du, g_down, _ = am.dense_bwd(dy, u, W["down"])
    da, g_up, g_bias = am.dense_bwd(du, a, W["up"], z=z, act="gelu", bias=True)
    da = da + dy
    do, g_out, _ = am.dense_bwd(da, o.view(T, d), W["out"])
    dqkv = torch.empty_like(qkv)
    dq, dk, dv = split(dqkv)
    am.attention_bwd(do.view(T, H, D), *split(qkv), o, lse, cu, cu, dq=dq, dk=dk, dv=dv)
    dx, g_qkv, _ = am.dense_bwd(dqkv, x, W["qkv"])
    dx = dx + da
    torch.cuda.synchronize()

    # the same block in float64 with torch's own gradients, on the CPU
    p = {n: t.detach().cpu().double().requires_grad_() for n, t in {**W, "x": x, "bias": bias}.items()}
    q64, k64, v64 = split(p["x"] @ p["qkv"])
    parts, at = [], 0
    for n in lens:
        s = slice(at, at + n)
        at += n
        kk, vv = (t[s].repeat_interleave(H // K, 1).transpose(0, 1).contiguous() for t in (k64, v64))
        sc = torch.matmul(q64[s].transpose(0, 1).contiguous(), kk.transpose(1, 2).contiguous()) * D ** -0.5
        sc = sc.masked_fill(~torch.ones(n, n, dtype=torch.bool).tril(), -math.inf)
        parts.append(torch.matmul(sc.softmax(-1), vv).transpose(0, 1))
    a64 = torch.cat(parts).reshape(T, d) @ p["out"] + p["x"]
    z64 = a64 @ p["up"] + p["bias"]
    y64 = (0.5 * z64 * torch.erfc(-z64 / math.sqrt(2))) @ p["down"] + a64
    y64.backward(dy.cpu().double())
    # chains of up to seven FP32 products of up to 128 terms each
    for got, want in ((y, y64), (dx, p["x"].grad), (g_qkv, p["qkv"].grad), (g_out, p["out"].grad), (g_up, p["up"].grad),
                      (g_bias, p["bias"].grad), (g_down, p["down"].grad)):
        want = want.detach()
        assert (got.cpu().double() - want).norm() <= 7 * 128 * 2.0 ** -24 * want.norm()

    # serving: the prompt's keys and values in a cache, the last tokens anew
    pages = -(-max(lens) // page)
    kp, vp = (torch.zeros(2 * pages, page, K, D, device="cuda") for _ in range(2))
    table = torch.arange(2 * pages, dtype=torch.int32, device="cuda").view(2, pages)
    ends = [sum(lens[: i + 1]) for i in range(2)]
    q, k, v = split(qkv)
    for b, n in enumerate(lens):
        s = slice(ends[b] - n, ends[b])
        kp.view(2, pages * page, K, D)[b, :n], vp.view(2, pages * page, K, D)[b, :n] = k[s], v[s]
    last = torch.tensor([e - 1 for e in ends], device="cuda")
    o1 = am.attention_paged(q[last].contiguous(), kp, vp, table, torch.arange(3, dtype=torch.int32, device="cuda"),
                            torch.tensor(lens, dtype=torch.int32, device="cuda"))
    a1 = am.dense_fwd(o1.view(2, d), W["out"], residual=x[last])
    y1 = am.dense_fwd(am.dense_fwd(a1, W["up"], bias=bias, act="gelu"), W["down"], residual=a1)
    torch.cuda.synchronize()
    want = y64.detach()[last.cpu()]
    assert (y1.cpu().double() - want).norm() <= 7 * 128 * 2.0 ** -24 * want.norm()


def test_binding_refuses(am):
    load(am, "mitchell07")
    x, w = torch.zeros(4, 5, device="cuda"), torch.zeros(5, 6, device="cuda")
    with pytest.raises(ValueError):
        am.dense_fwd(x, w, act="tanh")
    with pytest.raises(ValueError):
        am.dense_fwd(x, w.t())
    with pytest.raises(ValueError):
        am.dense_fwd(x, w, residual=torch.zeros(4, 5, device="cuda"))
    with pytest.raises(ValueError):
        am.dense_fwd(x, w, bias=torch.zeros(5, device="cuda"))
    with pytest.raises(ValueError):
        am.dense_bwd(torch.zeros(4, 6, device="cuda"), x, w, act="gelu")
    with pytest.raises(ValueError):
        am.dense_fwd(x, w.cpu())
