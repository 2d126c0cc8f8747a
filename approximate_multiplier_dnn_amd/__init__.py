"""Python binding of the LUT-based approximate-multiplier library (libapproxmul.so).

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI declared in include/approx_mul.h. The names follow
that header. Tensors are torch tensors on the current HIP device (FP32,
contiguous unless a leading dimension is passed); the stream defaults to
torch's current stream.

There is no fallback: importing this package fails if the built library is
missing (run ``__graft_entry__.build()`` or ``approximate_multiplier_dnn_amd/build.py``).
"""
import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libapproxmul.so")

APPROX_OK = 0
APPROX_EINVAL = -1
APPROX_ENOLUT = -2
APPROX_EUNSUPPORTED = -3
APPROX_EHIP = -4
APPROX_ESCRATCH = -5
APPROX_MAX_GROUP = 4

CONV_PASSES = {"fwd": 0, "dgrad": 1, "wgrad": 2}

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}

MODEL_EXACT = 0
MODEL_MITCHELL = 1

#: every function the C header declares
EXPORTS = (
    "approx_lut_build", "approx_lut_build_from_model", "approx_lut_load", "approx_native_load", "approx_lut_bits",
    "approx_exponent_bits_set", "approx_exponent_bits",
    "approx_gemm", "approx_gemm_noalloc", "approx_gemm_noalloc_max_bytes", "approx_gemm_grouped",
    "approx_gemm_strided_batched", "approx_gemm_batched",
    "approx_conv2d_fwd", "approx_conv2d_dgrad", "approx_conv2d_wgrad",
    "approx_attention_fwd", "approx_attention_bwd", "approx_attention_paged",
    "approx_dense_fwd", "approx_dense_bwd",
    "approx_gemm_chunks", "approx_conv2d_chunks",
    "approx_profile_enable", "approx_profile_read",
    "approx_status_string", "approx_build_id", "approx_release",
)

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; the approximate-multiplier path has no fallback")

_lib = ctypes.CDLL(LIB_PATH)

_i, _ll, _vp = ctypes.c_int, ctypes.c_longlong, ctypes.c_void_p
MUL_FN = ctypes.CFUNCTYPE(ctypes.c_float, ctypes.c_float, ctypes.c_float)
_lib.approx_lut_build.argtypes = [_i, _i, _vp, _vp]
_lib.approx_lut_build_from_model.argtypes = [_i, MUL_FN, _vp]
_lib.approx_lut_load.argtypes = [_vp, _i]
_lib.approx_lut_bits.argtypes = []
_lib.approx_exponent_bits_set.argtypes = [_i]
_lib.approx_exponent_bits.argtypes = []
_lib.approx_gemm.argtypes = [_i] * 5 + [_vp, _i, _vp, _i, _vp, _i, _vp]
_lib.approx_gemm_noalloc.argtypes = [_i] * 5 + [_vp, _i, _vp, _i, _vp, _i, _vp]
_lib.approx_gemm_noalloc_max_bytes.argtypes = []
_lib.approx_gemm_strided_batched.argtypes = [_i] * 5 + [_vp, _i, _ll, _vp, _i, _ll, _vp, _i, _ll, _i, _vp]
_lib.approx_gemm_batched.argtypes = [_i] * 5 + [_vp, _i, _vp, _i, _vp, _i, _i, _vp]
_lib.approx_gemm_grouped.argtypes = [_i] + [_vp] * 12
for _n in ("approx_conv2d_fwd", "approx_conv2d_dgrad", "approx_conv2d_wgrad"):
    getattr(_lib, _n).argtypes = [_i] * 11 + [_vp, _vp, _vp, _vp]
_lib.approx_gemm_chunks.argtypes = [_i] * 6 + [_ll, _vp, _vp, _vp, _vp]
_lib.approx_conv2d_chunks.argtypes = [_i] * 12 + [_ll, _vp, _vp]
_d = ctypes.c_double
_lib.approx_attention_fwd.argtypes = [_i] * 6 + [_vp, _vp, _i, _d] + [_vp, _i] * 4 + [_vp, _vp]
_lib.approx_attention_bwd.argtypes = [_i] * 6 + [_vp, _vp, _i, _d] + [_vp, _i] * 5 + [_vp] + [_vp, _i] * 3 + [_vp]
_lib.approx_attention_paged.argtypes = [_i] * 5 + [_vp, _i, _i, _vp, _vp, _vp, _i, _vp, _i, _d] + [_vp, _i] * 2 + [_vp, _vp]
_lib.approx_dense_fwd.argtypes = [_i] * 3 + [_vp, _i, _vp, _i, _vp, _i, _vp, _i, _vp, _i, _vp, _i, _vp]
_lib.approx_dense_bwd.argtypes = [_i] * 3 + [_vp, _i, _vp, _i, _vp, _i, _i, _vp, _i, _vp, _i, _vp, _i, _vp, _vp]
_lib.approx_status_string.argtypes = [_i]
_lib.approx_status_string.restype = ctypes.c_char_p
_lib.approx_build_id.argtypes = []
_lib.approx_build_id.restype = ctypes.c_char_p
_lib.approx_release.argtypes = []
_lib.approx_profile_enable.argtypes = [_i]
_lib.approx_profile_read.argtypes = [_vp, _vp]
for _n in EXPORTS:
    if _n not in ("approx_status_string", "approx_build_id", "approx_gemm_noalloc_max_bytes"):
        getattr(_lib, _n).restype = ctypes.c_int
_lib.approx_gemm_noalloc_max_bytes.restype = ctypes.c_longlong


class ApproxError(RuntimeError):
    def __init__(self, status, what):
        super().__init__(f"{what}: {approx_status_string(status)} ({status})")
        self.status = status


def lib():
    return _lib


def _check(rc, what):
    if rc != APPROX_OK:
        raise ApproxError(rc, what)
    return rc


def approx_status_string(status):
    return _lib.approx_status_string(int(status)).decode()


def approx_build_id():
    """Stamp of the sources the loaded library was built from."""
    return _lib.approx_build_id().decode()


# ------------------------------------------------------------------ tables

def approx_lut_build(model, M, perturb=None):
    """Table of 4**M uint16 entries (Algorithm 1) for MODEL_EXACT or
    MODEL_MITCHELL, optionally moved by a +/-1 int8 perturbation."""
    out = np.zeros(1 << (2 * M), dtype=np.uint16)
    p = None
    if perturb is not None:
        p = np.ascontiguousarray(perturb, dtype=np.int8)
        if p.size != out.size:
            raise ValueError("perturbation must have 4**M entries")
    _check(_lib.approx_lut_build(int(model), int(M), p.ctypes.data if p is not None else None,
                                 out.ctypes.data), "approx_lut_build")
    return out


def approx_lut_build_from_model(M, mul):
    """Table from a Python model float(float, float) of the multiplier."""
    out = np.zeros(1 << (2 * M), dtype=np.uint16)
    cb = MUL_FN(lambda a, b: float(mul(a, b)))
    _check(_lib.approx_lut_build_from_model(int(M), cb, out.ctypes.data), "approx_lut_build_from_model")
    return out


def approx_lut_load(lut, M):
    t = np.ascontiguousarray(lut, dtype=np.uint16)
    if t.size != (1 << (2 * M)):
        raise ValueError("table must have 4**M entries")
    _check(_lib.approx_lut_load(t.ctypes.data, int(M)), "approx_lut_load")


def approx_native_load():
    """Select the native FP32 multiplier (fused multiply-add) on the current device."""
    _check(_lib.approx_native_load(), "approx_native_load")


def approx_lut_bits():
    return _lib.approx_lut_bits()


def approx_exponent_bits_set(E):
    """Exponent width E (1..8) of the multiplier's format (1, E, M) on the current device."""
    _check(_lib.approx_exponent_bits_set(int(E)), "approx_exponent_bits_set")


def approx_exponent_bits():
    return _lib.approx_exponent_bits()


def approx_release():
    _check(_lib.approx_release(), "approx_release")


def approx_profile_enable(on=True):
    _check(_lib.approx_profile_enable(1 if on else 0), "approx_profile_enable")


def approx_profile_read():
    """(launches, total_ms) of the GEMM kernel since the last read."""
    n = ctypes.c_int(0)
    ms = ctypes.c_double(0.0)
    _check(_lib.approx_profile_read(ctypes.byref(n), ctypes.byref(ms)), "approx_profile_read")
    return n.value, ms.value


# ------------------------------------------------------------------ compute

def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    import torch
    if t.dtype != torch.float32 or not t.is_cuda:
        raise TypeError("expected a float32 tensor on the GPU")
    return t.data_ptr()


def approx_gemm(transA, transB, m, n, k, A, lda, B, ldb, C, ldc, stream=None):
    """C (m x n, leading dimension ldc) = op(A) op(B) with approximate products."""
    return _check(_lib.approx_gemm(int(transA), int(transB), int(m), int(n), int(k), _ptr(A), int(lda),
                                   _ptr(B), int(ldb), _ptr(C), int(ldc), _stream(stream)), "approx_gemm")


def approx_gemm_grouped(calls, stream=None):
    """Independent GEMMs in one call: `calls` holds 1 .. APPROX_MAX_GROUP
    tuples (transA, transB, m, n, k, A, lda, B, ldb, C, ldc), approx_gemm's
    arguments; each C gets the bits approx_gemm would give it."""
    calls = list(calls)
    cnt = len(calls)
    if not 1 <= cnt <= APPROX_MAX_GROUP:
        return _check(APPROX_EINVAL, "approx_gemm_grouped")
    ints = [(ctypes.c_int * cnt)(*(int(c[f]) for c in calls)) for f in (0, 1, 2, 3, 4, 6, 8, 10)]
    ptrs = [(ctypes.c_void_p * cnt)(*(_ptr(c[f]) for c in calls)) for f in (5, 7, 9)]
    tA, tB, m, n, k, lda, ldb, ldc = ints
    A, B, C = ptrs
    return _check(_lib.approx_gemm_grouped(cnt, tA, tB, m, n, k, A, lda, B, ldb, C, ldc, _stream(stream)),
                  "approx_gemm_grouped")


def approx_gemm_chunks(transA, transB, m, n, k, batch, b, i, j):
    """Summation chunk length of each output (b[t], i[t], j[t]) of a GEMM
    call with these sizes on the current device (k: one chunk)."""
    bb = np.ascontiguousarray(np.broadcast_to(np.asarray(b, dtype=np.int32), np.shape(i)), dtype=np.int32).ravel()
    ii = np.ascontiguousarray(i, dtype=np.int32).ravel()
    jj = np.ascontiguousarray(j, dtype=np.int32).ravel()
    assert ii.shape == jj.shape == bb.shape
    out = np.zeros(ii.size, dtype=np.int64)
    _check(_lib.approx_gemm_chunks(int(transA), int(transB), int(m), int(n), int(k), int(batch), ii.size,
                                   bb.ctypes.data, ii.ctypes.data, jj.ctypes.data, out.ctypes.data),
           "approx_gemm_chunks")
    return out


def approx_conv2d_chunks(pass_name, N, H, W, C, K, R, S, stride, pad, idx):
    """Summation chunk length of the outputs at flat indices idx of a Conv2D
    pass ("fwd", "dgrad" or "wgrad") on the current device."""
    ix = np.ascontiguousarray(idx, dtype=np.int64).ravel()
    out = np.zeros(ix.size, dtype=np.int64)
    _check(_lib.approx_conv2d_chunks(CONV_PASSES[pass_name], int(N), int(H), int(W), int(C), int(K), int(R),
                                     int(S), int(stride[0]), int(stride[1]), int(pad[0]), int(pad[1]), ix.size,
                                     ix.ctypes.data, out.ctypes.data), "approx_conv2d_chunks")
    return out


def approx_gemm_noalloc(transA, transB, m, n, k, A, lda, B, ldb, C, ldc, stream=None):
    """approx_gemm without any allocation (fixed per-device scratch)."""
    return _check(_lib.approx_gemm_noalloc(int(transA), int(transB), int(m), int(n), int(k), _ptr(A), int(lda),
                                           _ptr(B), int(ldb), _ptr(C), int(ldc), _stream(stream)),
                  "approx_gemm_noalloc")


def approx_gemm_noalloc_max_bytes():
    return int(_lib.approx_gemm_noalloc_max_bytes())


def approx_gemm_strided_batched(transA, transB, m, n, k, A, lda, strideA, B, ldb, strideB, C, ldc, strideC,
                                batch, stream=None):
    return _check(_lib.approx_gemm_strided_batched(
        int(transA), int(transB), int(m), int(n), int(k), _ptr(A), int(lda), int(strideA), _ptr(B), int(ldb),
        int(strideB), _ptr(C), int(ldc), int(strideC), int(batch), _stream(stream)), "approx_gemm_strided_batched")


def approx_gemm_batched(transA, transB, m, n, k, A_ptrs, lda, B_ptrs, ldb, C_ptrs, ldc, batch, stream=None):
    """Batched GEMM by device pointer arrays (int64 tensors of data pointers on the GPU)."""
    def arr(t):
        if isinstance(t, int):
            return t
        import torch
        if t.dtype != torch.int64 or not t.is_cuda or t.numel() < batch:
            raise TypeError("pointer arrays must be int64 GPU tensors with one entry per batch")
        return t.data_ptr()
    return _check(_lib.approx_gemm_batched(int(transA), int(transB), int(m), int(n), int(k), arr(A_ptrs), int(lda),
                                           arr(B_ptrs), int(ldb), arr(C_ptrs), int(ldc), int(batch),
                                           _stream(stream)), "approx_gemm_batched")


def pointer_array(tensors_or_ptrs, device="cuda"):
    """int64 device tensor holding the data pointers of the given tensors."""
    import torch
    ptrs = [t if isinstance(t, int) else t.data_ptr() for t in tensors_or_ptrs]
    return torch.tensor(ptrs, dtype=torch.int64, device=device)


def _conv_call(name, N, H, W, C, K, R, S, stride, pad, t1, t2, out, stream):
    fn = getattr(_lib, name)
    return _check(fn(int(N), int(H), int(W), int(C), int(K), int(R), int(S), int(stride[0]), int(stride[1]),
                     int(pad[0]), int(pad[1]), _ptr(t1), _ptr(t2), _ptr(out), _stream(stream)), name)


def approx_conv2d_fwd(N, H, W, C, K, R, S, stride, pad, x, w, y, stream=None):
    return _conv_call("approx_conv2d_fwd", N, H, W, C, K, R, S, stride, pad, x, w, y, stream)


def approx_conv2d_dgrad(N, H, W, C, K, R, S, stride, pad, dy, w, dx, stream=None):
    return _conv_call("approx_conv2d_dgrad", N, H, W, C, K, R, S, stride, pad, dy, w, dx, stream)


def approx_conv2d_wgrad(N, H, W, C, K, R, S, stride, pad, x, dy, dw, stream=None):
    return _conv_call("approx_conv2d_wgrad", N, H, W, C, K, R, S, stride, pad, x, dy, dw, stream)


# ------------------------------------------------------------------ tensor helpers

def gemm(A, B, transA=False, transB=False, out=None, stream=None):
    """op(A) @ op(B) for contiguous 2-D tensors; allocates the output."""
    import torch
    m = A.shape[1] if transA else A.shape[0]
    k = A.shape[0] if transA else A.shape[1]
    n = B.shape[0] if transB else B.shape[1]
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=A.device)
    approx_gemm(transA, transB, m, n, k, A, A.stride(0), B, B.stride(0), out, out.stride(0), stream)
    return out


def _heads(t, what):
    """Leading dimension of a [tokens, heads, dim] tensor whose heads lie dim apart."""
    if t.dim() != 3 or (t.shape[2] > 1 and t.stride(2) != 1) or (t.shape[1] > 1 and t.stride(1) != t.shape[2]):
        raise ValueError(f"{what}: expected [tokens, heads, dim] with contiguous heads, got {tuple(t.shape)} "
                         f"strides {t.stride()}")
    least = t.shape[1] * t.shape[2]
    if t.shape[0] <= 1:
        return least
    if t.stride(0) < least:
        raise ValueError(f"{what}: tokens overlap (stride {t.stride(0)} below {least})")
    return t.stride(0)


def _int32(t, what, device, dims=1):
    import torch
    if t.dtype != torch.int32 or t.dim() != dims or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{what}: expected a contiguous {dims}-D int32 tensor on {device}")
    return t.data_ptr()


def _same_device(*tensors):
    """The tensors' device: one device, the current one (the library queues on it)."""
    import torch
    device = tensors[0].device
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError(f"tensors on {device} and {t.device}")
    if device.type != "cuda" or device.index != torch.cuda.current_device():
        raise ValueError(f"tensors on {device}: make it the current device")
    return device


def _packed_shapes(q, k, v, cu_q, cu_k):
    if k.shape != v.shape or k.shape[2] != q.shape[2]:
        raise ValueError(f"shapes of q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)} do not belong together")
    if cu_q.shape != cu_k.shape or cu_q.numel() < 1:
        raise ValueError("cu_q and cu_k hold one offset more than there are sequences")
    return cu_q.numel() - 1


def attention_fwd(q, k, v, cu_q, cu_k, causal=True, scale=None, out=None, lse=None, stream=None):
    """Attention of packed prompts with approximate products: q [tokens, heads, dim],
    k and v [tokens, kv_heads, dim] (views of one projection's output will do),
    cu_q and cu_k int32 offsets on the GPU. scale defaults to dim ** -0.5.
    Returns (o, lse); rows of no sequence keep what out and lse hold."""
    import torch
    device = _same_device(q, k, v, out, lse)
    ldq, ldk, ldv = _heads(q, "q"), _heads(k, "k"), _heads(v, "v")
    nseq = _packed_shapes(q, k, v, cu_q, cu_k)
    T, H, D = q.shape
    if out is None:
        out = torch.empty((T, H, D), dtype=torch.float32, device=device)
    if lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=device)
    if out.shape != q.shape or lse.shape != (T, H) or not lse.is_contiguous():
        raise ValueError("out has q's shape, lse is contiguous [tokens, heads]")
    _check(_lib.approx_attention_fwd(nseq, H, k.shape[1], D, T, k.shape[0], _int32(cu_q, "cu_q", device),
                                     _int32(cu_k, "cu_k", device), int(bool(causal)),
                                     D ** -0.5 if scale is None else float(scale), _ptr(q), ldq, _ptr(k), ldk,
                                     _ptr(v), ldv, _ptr(out), _heads(out, "out"), _ptr(lse), _stream(stream)),
           "approx_attention_fwd")
    return out, lse


def attention_bwd(dout, q, k, v, o, lse, cu_q, cu_k, causal=True, scale=None, dq=None, dk=None, dv=None, stream=None):
    """Gradients (dq, dk, dv) of attention_fwd's o, from its inputs and what it
    returned; rows of no sequence keep what dq, dk and dv hold."""
    import torch
    device = _same_device(q, k, v, o, dout, lse, dq, dk, dv)
    nseq = _packed_shapes(q, k, v, cu_q, cu_k)
    T, H, D = q.shape
    if o.shape != q.shape or dout.shape != q.shape or lse.shape != (T, H) or not lse.is_contiguous():
        raise ValueError("o and dout have q's shape, lse is contiguous [tokens, heads]")
    dq, dk, dv = (torch.empty(x.shape, dtype=torch.float32, device=device) if g is None else g
                  for g, x in ((dq, q), (dk, k), (dv, v)))
    if dq.shape != q.shape or dk.shape != k.shape or dv.shape != v.shape:
        raise ValueError("dq, dk and dv have the shapes of q, k and v")
    pairs = []
    for t, what in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout")):
        pairs += [_ptr(t), _heads(t, what)]
    grads = []
    for t, what in ((dq, "dq"), (dk, "dk"), (dv, "dv")):
        grads += [_ptr(t), _heads(t, what)]
    _check(_lib.approx_attention_bwd(nseq, H, k.shape[1], D, T, k.shape[0], _int32(cu_q, "cu_q", device),
                                     _int32(cu_k, "cu_k", device), int(bool(causal)),
                                     D ** -0.5 if scale is None else float(scale), *pairs, _ptr(lse), *grads,
                                     _stream(stream)), "approx_attention_bwd")
    return dq, dk, dv


def attention_paged(q, k_pages, v_pages, block_table, cu_q, k_len, causal=True, scale=None, out=None, lse=None, stream=None):
    """Attention of new tokens q [tokens, heads, dim] over a paged cache:
    k_pages and v_pages [pages, page, kv_heads, dim], block_table [sequences,
    pages per sequence] int32, cu_q offsets of the sequences' new tokens, k_len
    their cached keys (the new ones included). Returns o; lse ([tokens, heads])
    is written when given."""
    import torch
    device = _same_device(q, k_pages, v_pages, out, lse)
    T, H, D = q.shape
    if k_pages.dim() != 4 or k_pages.shape != v_pages.shape or k_pages.shape[3] != D:
        raise ValueError("k_pages and v_pages are [pages, page, kv_heads, dim] with q's dim")
    if not k_pages.is_contiguous() or not v_pages.is_contiguous():
        raise ValueError("k_pages and v_pages are contiguous")
    if cu_q.numel() < 1 or k_len.numel() != cu_q.numel() - 1 or block_table.shape[0] != k_len.numel():
        raise ValueError("cu_q holds one offset more than k_len and block_table hold sequences")
    if out is None:
        out = torch.empty((T, H, D), dtype=torch.float32, device=device)
    if out.shape != q.shape or (lse is not None and (lse.shape != (T, H) or not lse.is_contiguous())):
        raise ValueError("out has q's shape, lse is contiguous [tokens, heads]")
    _check(_lib.approx_attention_paged(k_len.numel(), H, k_pages.shape[2], D, T, _int32(cu_q, "cu_q", device),
                                       k_pages.shape[0], k_pages.shape[1], _ptr(k_pages), _ptr(v_pages),
                                       _int32(block_table, "block_table", device, 2), block_table.shape[1],
                                       _int32(k_len, "k_len", device), int(bool(causal)),
                                       D ** -0.5 if scale is None else float(scale), _ptr(q), _heads(q, "q"), _ptr(out),
                                       _heads(out, "out"), _ptr(lse), _stream(stream)), "approx_attention_paged")
    return out


def _rows(t, what, shape):
    """Leading dimension of a row-major 2-D tensor of the given shape."""
    if tuple(t.shape) != tuple(shape) or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{what}: expected {tuple(shape)} with contiguous rows, got {tuple(t.shape)} strides {t.stride()}")
    least = max(1, t.shape[1])
    if t.shape[0] <= 1:
        return least
    if t.stride(0) < least:
        raise ValueError(f"{what}: rows overlap (stride {t.stride(0)} below {least})")
    return t.stride(0)


def _activation(act):
    if act not in ACTIVATIONS:
        raise ValueError(f"act {act!r}: one of {', '.join(ACTIVATIONS)}")
    return ACTIVATIONS[act]


def dense_fwd(x, w, bias=None, act="none", residual=None, keep_z=False, out=None, stream=None):
    """act(x @ w + bias) + residual with approximate products, x [m, k] and
    w [k, n]; with keep_z also x @ w + bias, which dense_bwd needs when there
    is an activation: (y, z)."""
    import torch
    device = _same_device(x, w, bias, residual, out)
    (m, k), n = x.shape, w.shape[1]
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=device)
    z = torch.empty((m, n), dtype=torch.float32, device=device) if keep_z else None
    if bias is not None and (bias.shape != (n,) or not bias.is_contiguous()):
        raise ValueError("bias: n contiguous values")
    _check(_lib.approx_dense_fwd(m, n, k, _ptr(x), _rows(x, "x", (m, k)), _ptr(w), _rows(w, "w", (k, n)), _ptr(bias),
                                 _activation(act), _ptr(residual),
                                 max(1, n) if residual is None else _rows(residual, "residual", (m, n)), _ptr(out),
                                 _rows(out, "out", (m, n)), _ptr(z), max(1, n), _stream(stream)), "approx_dense_fwd")
    return (out, z) if keep_z else out


def dense_bwd(dy, x, w, z=None, act="none", bias=False, dx=None, dw=None, stream=None):
    """Gradients (dx, dw, db) of dense_fwd's y for dy, with z as keep_z returned
    it; db is None without a bias. The residual's gradient is dy."""
    import torch
    device = _same_device(dy, x, w, z, dx, dw)
    (m, k), n = x.shape, w.shape[1]
    if z is None and act != "none":
        raise ValueError(f"the gradient of {act} needs z")
    dx = torch.empty((m, k), dtype=torch.float32, device=device) if dx is None else dx
    dw = torch.empty((k, n), dtype=torch.float32, device=device) if dw is None else dw
    db = torch.empty((n,), dtype=torch.float32, device=device) if bias else None
    _check(_lib.approx_dense_bwd(m, n, k, _ptr(x), _rows(x, "x", (m, k)), _ptr(w), _rows(w, "w", (k, n)), _ptr(z),
                                 max(1, n) if z is None else _rows(z, "z", (m, n)), _activation(act), _ptr(dy),
                                 _rows(dy, "dy", (m, n)), _ptr(dx), _rows(dx, "dx", (m, k)), _ptr(dw),
                                 _rows(dw, "dw", (k, n)), _ptr(db), _stream(stream)), "approx_dense_bwd")
    return dx, dw, db


def conv_out_hw(H, W, R, S, stride, pad):
    return (H + 2 * pad[0] - R) // stride[0] + 1, (W + 2 * pad[1] - S) // stride[1] + 1


def conv2d_fwd(x, w, stride=(1, 1), pad=(0, 0), stream=None):
    """x NHWC, w RSCK -> y NPQK."""
    import torch
    N, H, W, C = x.shape
    R, S, _, K = w.shape
    P, Q = conv_out_hw(H, W, R, S, stride, pad)
    y = torch.empty((N, P, Q, K), dtype=torch.float32, device=x.device)
    approx_conv2d_fwd(N, H, W, C, K, R, S, stride, pad, x, w, y, stream)
    return y


def conv2d_dgrad(dy, w, x_shape, stride=(1, 1), pad=(0, 0), stream=None):
    import torch
    N, H, W, C = x_shape
    R, S, _, K = w.shape
    dx = torch.empty((N, H, W, C), dtype=torch.float32, device=dy.device)
    approx_conv2d_dgrad(N, H, W, C, K, R, S, stride, pad, dy, w, dx, stream)
    return dx


def conv2d_wgrad(x, dy, w_shape, stride=(1, 1), pad=(0, 0), stream=None):
    import torch
    N, H, W, C = x.shape
    R, S, _, K = w_shape
    dw = torch.empty((R, S, C, K), dtype=torch.float32, device=x.device)
    approx_conv2d_wgrad(N, H, W, C, K, R, S, stride, pad, x, dy, dw, stream)
    return dw
