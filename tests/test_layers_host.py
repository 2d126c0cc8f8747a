"""Host-side checks of the attention and dense-layer calls that need no GPU:
arguments that are refused before any HIP call, calls with nothing to do, and
the reference of the GPU tests against plain float64 attention."""
import ctypes
import math

import numpy as np
import pytest

import attention_ref as ref
import oracle
from datagen import normal


@pytest.fixture(scope="module")
def am():
    import approximate_multiplier_dnn_amd as m
    return m


P = 4096            # never dereferenced: the checks fail first
ATTN = dict(nseq=2, heads=4, kv_heads=2, dim=64, total_q=10, total_k=12, cu_q=P, cu_k=P, causal=1, scale=0.125, q=P, ldq=256, k=P,
            ldk=128, v=P, ldv=128, o=P, ldo=256, lse=P, stream=None)
BWD = ["nseq", "heads", "kv_heads", "dim", "total_q", "total_k", "cu_q", "cu_k", "causal", "scale", "q", "ldq", "k", "ldk", "v",
       "ldv", "o", "ldo", "dout", "lddo", "lse", "dq", "lddq", "dk", "lddk", "dv", "lddv", "stream"]
PAGED = dict(nseq=2, heads=4, kv_heads=2, dim=64, total_q=3, cu_q=P, num_pages=5, page=16, kp=P, vp=P, table=P, table_ld=4, k_len=P,
             causal=1, scale=0.125, q=P, ldq=256, o=P, ldo=256, lse=None, stream=None)
WRONG = [dict(nseq=-1), dict(heads=0), dict(heads=3), dict(kv_heads=0), dict(dim=0), dict(total_q=-1), dict(causal=2),
         dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan), dict(scale=1e300), dict(scale=1e-300), dict(ldq=255), dict(ldo=255), dict(q=None),
         dict(o=None), dict(cu_q=None)]


@pytest.mark.parametrize("change", WRONG + [dict(total_k=-1), dict(ldk=127), dict(ldv=127), dict(k=None), dict(v=None), dict(cu_k=None)],
                         ids=str)
def test_attention_refusals(am, change):
    L = am.lib()
    args = {**ATTN, **change}
    assert L.approx_attention_fwd(*args.values()) == am.APPROX_EINVAL
    args = {**ATTN, "dout": P, "lddo": 256, "dq": P, "lddq": 256, "dk": P, "lddk": 128, "dv": P, "lddv": 128, **change}
    assert L.approx_attention_bwd(*(args[x] for x in BWD)) == am.APPROX_EINVAL


@pytest.mark.parametrize("change", [dict(dout=None), dict(lse=None), dict(dq=None), dict(dk=None), dict(dv=None), dict(lddo=1),
                                    dict(lddq=255), dict(lddk=127), dict(lddv=127)], ids=str)
def test_attention_gradient_refusals(am, change):
    args = {**ATTN, "dout": P, "lddo": 256, "dq": P, "lddq": 256, "dk": P, "lddk": 128, "dv": P, "lddv": 128, **change}
    assert am.lib().approx_attention_bwd(*(args[x] for x in BWD)) == am.APPROX_EINVAL


@pytest.mark.parametrize("change", WRONG + [dict(num_pages=-1), dict(page=0), dict(table_ld=-1), dict(kp=None), dict(vp=None),
                                            dict(table=None), dict(k_len=None)], ids=str)
def test_paged_refusals(am, change):
    assert am.lib().approx_attention_paged(*{**PAGED, **change}.values()) == am.APPROX_EINVAL


def test_sizes_beyond_the_limits(am):
    L = am.lib()
    for change in (dict(dim=129, ldq=1000, ldk=1000, ldv=1000, ldo=1000), dict(total_q=1 << 29), dict(total_k=1 << 30)):
        assert L.approx_attention_fwd(*{**ATTN, **change}.values()) == am.APPROX_EUNSUPPORTED
    for change in (dict(dim=129, ldq=1000, ldo=1000), dict(num_pages=1 << 27), dict(table_ld=1 << 27)):
        assert L.approx_attention_paged(*{**PAGED, **change}.values()) == am.APPROX_EUNSUPPORTED


def test_nothing_to_do(am):
    L = am.lib()
    assert L.approx_attention_fwd(*{**ATTN, "nseq": 0}.values()) == am.APPROX_OK
    assert L.approx_attention_fwd(*{**ATTN, "total_q": 0, "q": None, "o": None}.values()) == am.APPROX_OK
    assert L.approx_attention_paged(*{**PAGED, "total_q": 0}.values()) == am.APPROX_OK
    # m or n zero: no output
    assert L.approx_dense_fwd(0, 4, 4, None, 4, P, 4, None, 0, None, 4, None, 4, None, 4, None) == am.APPROX_OK


def test_dense_refusals(am):
    L = am.lib()
    ok = dict(m=4, n=6, k=5, X=P, ldx=5, W=P, ldw=6, bias=None, act=1, res=P, ldr=6, Y=P, ldy=6, Z=P, ldz=6, stream=None)
    for change in (dict(m=-1), dict(n=-1), dict(k=-1), dict(X=None), dict(W=None), dict(Y=None), dict(ldx=4), dict(ldw=5), dict(ldr=5),
                   dict(ldy=5), dict(ldz=5), dict(act=4), dict(act=-1)):
        assert L.approx_dense_fwd(*{**ok, **change}.values()) == am.APPROX_EINVAL, change
    ok = dict(m=4, n=6, k=5, X=P, ldx=5, W=P, ldw=6, Z=P, ldz=6, act=1, dY=P, lddy=6, dX=P, lddx=5, dW=P, lddw=6, db=None, stream=None)
    for change in (dict(m=-1), dict(n=-1), dict(k=-1), dict(X=None), dict(W=None), dict(Z=None), dict(dY=None), dict(ldx=4), dict(ldw=5),
                   dict(ldz=5), dict(lddy=5), dict(lddx=4), dict(lddw=5), dict(act=4)):
        assert L.approx_dense_bwd(*{**ok, **change}.values()) == am.APPROX_EINVAL, change


def test_reference_is_attention():
    """With exact products the reference is softmax attention and its gradient."""
    n, m, D = 9, 14, 8
    q, k, v, dout = normal(1, (n, D)), normal(2, (m, D)), normal(3, (m, D)), normal(4, (n, D))
    seen = ref.causal_mask(n, m)
    s = np.where(seen, q.astype(np.float64) @ k.T.astype(np.float64) / math.sqrt(D), -np.inf)
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    o, lse, _ = ref.attention(q, k, v, seen, D ** -0.5, None, 0)
    # FP32 scores: D roundings of 2^-24 each, and the weights' one
    assert np.allclose(o, p @ v, rtol=0, atol=1e-5)
    assert np.allclose(lse, s.max(1) + np.log(np.exp(s - s.max(1, keepdims=True)).sum(1)), rtol=0, atol=1e-5)
    dp = dout @ v.T
    ds = p * (dp - (dp * p).sum(1, keepdims=True))
    (dq, dk, dv), _ = ref.attention_grad(q, k, v, o.astype(np.float32), lse.astype(np.float32), dout, seen, D ** -0.5, None, 0)
    assert np.allclose(dq, ds @ k / math.sqrt(D), atol=1e-5)
    assert np.allclose(dk, ds.T @ q / math.sqrt(D), atol=1e-5)
    assert np.allclose(dv, p.T @ dout, atol=1e-5)


def test_reference_rounds_scores_as_the_oracle():
    """The reference's scores are the oracle's FP32 sums in one chunk."""
    M = 7
    lut = oracle.lut_generate(M, "mitchell")
    a, b = normal(5, (6, 40)), normal(6, (7, 40))
    want = oracle.gemm_f32(a, np.ascontiguousarray(b.T), lut, M, 40)
    assert np.array_equal(ref.dots32(a, b, lut, M).view(np.uint32), want.view(np.uint32))


def test_empty_rows_of_the_reference():
    lut = oracle.lut_generate(5, "exact")
    q, k, v = normal(7, (4, 8)), normal(8, (2, 8)), normal(9, (2, 8))
    o, lse, _ = ref.attention(q, k, v, ref.causal_mask(4, 2), 0.3, lut, 5)
    assert (o[:2] == 0).all() and np.isneginf(lse[:2]).all() and np.isfinite(lse[2:]).all()


def test_symbols_take_doubles(am):
    assert am.lib().approx_attention_fwd.argtypes[9] is ctypes.c_double
