"""Measured cases of the transformer operators with approximate products: attention over packed prompts (forward and
backward), attention of new tokens over a paged cache, and the dense layer with bias, activation and residual.

Every contraction's products are those of a multiplier table: an FP32 operand counts by its sign, its exponent and the top
M bits of its fraction, and the table gives the product of two such fractions. A sum of products that a table reads again
(the attention scores, and dP in the backward pass) is defined to the bit: FP32, ascending, from zero. What is computed and
then enters a table (softmax numerators, dS, dz) is rounded once from 64 bits, because the table cuts it at M bits and an
error of one last place next to such a border moves a product by 2^-M.
"""
import math

import numpy as np
import torch

own = False

LOG2E = 1.4426950408889634
TINY = -64.0                 # numerators and gradients of scores below 2^-64 count as zero


# ------------------------------------------------------------------ tables

def table_entries(model, M):
    """uint16 entries (first << M | second): bit 15 carry, bits 14..0 the top fraction bits of the product."""
    x = np.arange(1 << M, dtype=np.float64) / (1 << M)
    a, b = x[:, None], x[None, :]
    if model == "mitchell":
        p = np.where(a + b < 1, 1 + a + b, 2 * (a + b))
    else:
        p = (1 + a) * (1 + b)
    carry = p >= 2
    frac = np.floor((np.where(carry, p / 2, p) - 1) * (1 << 15)).astype(np.uint16)
    return (frac | (carry.astype(np.uint16) << 15)).reshape(-1)


def table_values(model, M):
    e = table_entries(model, M).astype(np.int64)
    return (1 + (e & 0x7FFF) / 32768.0) * np.where(e >> 15, 2.0, 1.0)


_loaded = None


def _load(case):
    """Loads the case's table into the framework when another one is loaded: a program does this when it starts."""
    global _loaded
    import approximate_multiplier_dnn_amd as am
    if _loaded != (case["model"], case["M"]):
        am.approx_lut_load(table_entries(case["model"], case["M"]), case["M"])
        _loaded = (case["model"], case["M"])
    return am


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a handful of short prompts of a tiny batch: launch latency counts
        dict(name="attn_fwd_few_short", op="attn_fwd", model="mitchell", M=7, seqs=5, lo=1, hi=48, heads=4, kv_heads=2, dim=64,
             causal=True),
        # the attention block's configuration: 16 sequences of 512 tokens, 12 heads of 64
        dict(name="attn_fwd_block", op="attn_fwd", model="mitchell", M=7, seqs=16, lo=512, hi=512, heads=12, kv_heads=12, dim=64,
             causal=True),
        # one long prompt of odd length, grouped heads of 128, a wider multiplier
        dict(name="attn_fwd_long", op="attn_fwd", model="exact", M=8, seqs=1, lo=4001, hi=4001, heads=8, kv_heads=2, dim=128,
             causal=True),
        # fine-tuning on a few short texts, attention in both directions
        dict(name="attn_bwd_short", op="attn_bwd", model="mitchell", M=7, seqs=3, lo=20, hi=150, heads=4, kv_heads=4, dim=64,
             causal=False),
        # a training step's packed batch of ragged texts with grouped heads
        dict(name="attn_bwd_block", op="attn_bwd", model="mitchell", M=7, seqs=8, lo=200, hi=512, heads=12, kv_heads=4, dim=64,
             causal=True),
        # answering one user: the next token over a short cache
        dict(name="paged_token", op="paged", model="mitchell", M=7, seqs=1, new=1, lo=300, hi=300, heads=12, kv_heads=4, dim=64,
             page=16),
        # a serving batch's next tokens over long caches
        dict(name="paged_tokens_long", op="paged", model="mitchell", M=7, seqs=32, new=1, lo=1000, hi=8192, heads=16, kv_heads=4,
             dim=128, page=64),
        # chunks of new prompt tokens over what the cache already holds
        dict(name="paged_chunk", op="paged", model="mitchell", M=7, seqs=4, new=128, lo=500, hi=4000, heads=8, kv_heads=4, dim=64,
             page=16),
        # one token through a layer
        dict(name="dense_fwd_token", op="dense_fwd", model="mitchell", M=7, m=1, n=1024, k=1024, act="gelu", bias=True,
             residual=False, keep=False),
        # the attention block's output projection with its residual
        dict(name="dense_fwd_block", op="dense_fwd", model="mitchell", M=7, m=8192, n=768, k=768, act="none", bias=True,
             residual=True, keep=False),
        # the MLP's hidden layer at its batch
        dict(name="dense_bwd_mlp", op="dense_bwd", model="mitchell", M=7, m=256, n=1024, k=1024, act="relu", bias=True),
        # a transformer layer's first feed-forward product
        dict(name="dense_bwd_block", op="dense_bwd", model="exact", M=7, m=4096, n=2048, k=768, act="gelu", bias=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn_fwd", "attn_bwd", "paged", "dense_fwd", "dense_bwd"])
    case = dict(op=op, model=rng.choice(["mitchell", "exact"]), M=rng.choice([4, 6, 7, 7, 7, 8]))
    if op in ("dense_fwd", "dense_bwd"):
        m, n, k = _log_int(rng, 1, 8192), _log_int(rng, 8, 2500), _log_int(rng, 8, 2500)
        while m * n * k > 8192 * 768 * 768:
            m, n, k = max(1, m // 2), max(8, n * 3 // 4), max(8, k * 3 // 4)
        case.update(m=m, n=n, k=k, act=rng.choice(["none", "relu", "gelu", "silu"]), bias=rng.random() < 0.7)
        if op == "dense_fwd":
            case.update(residual=rng.random() < 0.5, keep=rng.random() < 0.5)
        return case
    kv = rng.choice([1, 2, 3, 4, 8])
    case.update(heads=kv * rng.choice([1, 1, 2, 3, 4, 8]), kv_heads=kv, dim=rng.choice([32, 40, 64, 64, 80, 96, 128, 128]))
    if op == "paged":
        seqs, hi = _log_int(rng, 1, 32), _log_int(rng, 16, 8192)
        new = 1 if rng.random() < 0.5 else _log_int(rng, 1, 192)
        while seqs * hi * new * case["heads"] * case["dim"] > 4 * 4000 * 128 * 8 * 64:
            seqs, new = max(1, seqs // 2), max(1, new // 2)
        lo = rng.randint(1, hi)
        case.update(seqs=seqs, new=new, lo=max(new, lo), hi=max(new, hi), page=rng.choice([8, 16, 16, 32, 64, 100]))
        return case
    seqs, hi = _log_int(rng, 1, 16), _log_int(rng, 1, 4096 if op == "attn_fwd" else 1024)
    most = 16 * 12 * 512 * 512 * 64 * (1 if op == "attn_bwd" else 2)
    while seqs * case["heads"] * case["dim"] * hi * hi > most:
        seqs, hi = max(1, seqs * 3 // 4), max(1, hi * 7 // 8)
    case.update(seqs=seqs, lo=rng.randint(max(1, hi // 4), hi), hi=hi, causal=rng.random() < 0.7)
    return case


def _lengths(case):
    """Lengths of the case's sequences: fixed by the case, so that every seed's inputs have the same sizes."""
    r = np.random.RandomState(case["seqs"] * 7919 + case["lo"] * 31 + case["hi"])
    n = r.randint(case["lo"], case["hi"] + 1, case["seqs"])
    n[r.randint(case["seqs"])] = case["hi"]
    return [int(v) for v in n]


def _offsets(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32), device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * std

    state = dict(case=case, table=torch.tensor(table_values(case["model"], case["M"]), dtype=torch.float32, device="cuda"))
    if case["op"] in ("dense_fwd", "dense_bwd"):
        m, n, k = case["m"], case["n"], case["k"]
        state.update(x=normal(m, k), w=normal(k, n, std=1 / math.sqrt(k)), bias=normal(n, std=0.1) if case["bias"] else None)
        if case["op"] == "dense_fwd":
            state.update(residual=normal(m, n) if case["residual"] else None)
        else:
            state.update(dy=normal(m, n), z=normal(m, n))
        return state
    H, K, D = case["heads"], case["kv_heads"], case["dim"]
    lengths = _lengths(case)
    if case["op"] == "paged":
        page, B = case["page"], case["seqs"]
        new = [min(case["new"], n) for n in lengths]
        pages = [-(-n // page) for n in lengths]
        spare = 3                                      # pages of other users lie between
        order = torch.randperm(sum(pages) + spare, generator=g, device="cuda").to(torch.int32)
        blocks = torch.full((B, max(pages)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(pages):
            blocks[b, :n] = order[at:at + n]
            at += n
        state.update(q=normal(sum(new), H, D), k_pages=normal(at + spare, page, K, D), v_pages=normal(at + spare, page, K, D),
                     blocks=blocks, cu_q=_offsets(new), k_len=torch.tensor(lengths, dtype=torch.int32, device="cuda"),
                     new=new, lengths=lengths)
        return state
    T = sum(lengths)
    # the three parts of one projection's output, as a layer has them
    qkv = normal(T, (H + 2 * K) * D)
    q, k, v = qkv[:, :H * D].view(T, H, D), qkv[:, H * D:(H + K) * D].view(T, K, D), qkv[:, (H + K) * D:].view(T, K, D)
    state.update(q=q, k=k, v=v, cu=_offsets(lengths), lengths=lengths)
    if case["op"] == "attn_bwd":
        # what the forward pass left, and the gradient of its output
        state["o"], state["lse"] = _plain_forward(state)
        state["do"] = normal(T, H, D)
    return state


# ------------------------------------------------------------------ the plain form

def _parts(x, M):
    """Table index and signed power of two of FP32 operands (zero and subnormal: power zero)."""
    bits = x.contiguous().view(torch.int32)
    return ((bits >> (23 - M)) & ((1 << M) - 1)).long(), (bits & -8388608).view(torch.float32)


def _padded(x, lengths, cu):
    """[tokens, heads, dim] as [sequence, head, longest, dim], zero behind each sequence's end."""
    at = cu[:-1, None].long() + torch.arange(max(lengths), device=x.device)[None]
    inside = at < cu[1:, None]
    return (x[at.clamp(max=x.shape[0] - 1)] * inside[..., None, None]).transpose(1, 2), inside


def _packed(x, inside):
    """The inverse of _padded."""
    return x.transpose(1, 2)[inside]


def _group(x, K):
    """[sequence, head, token, dim] as [sequence, kv head, (head of its group, token), dim]."""
    return x.reshape(x.shape[0], K, -1, x.shape[-1])


def _scores(a, b, tab, M):
    """FP32 sums of table products a_i b_j, ascending over the last dimension: one step for each of its positions."""
    (ai, ap), (bi, bp) = _parts(a, M), _parts(b, M)
    s = torch.zeros(a.shape[:-1] + (b.shape[-2],), dtype=torch.float32, device=a.device)
    for p in range(a.shape[-1]):
        s += tab[(ai[..., :, None, p] << M) | bi[..., None, :, p]] * (ap[..., :, None, p] * bp[..., None, :, p])
    return s


def _weighted(wt, x, tab, M, weight_first=True, over_rows=False):
    """Sums of table products of weights wt[i, j] with rows x_j (over j), or x_i (over_rows: over i), one column at a time."""
    (wi, wp), (xi, xp) = _parts(wt, M), _parts(x, M)
    cols = []
    for d in range(x.shape[-1]):
        yi, yp = (xi[..., :, None, d], xp[..., :, None, d]) if over_rows else (xi[..., None, :, d], xp[..., None, :, d])
        index = (wi << M) | yi if weight_first else (yi << M) | wi
        cols.append((tab[index] * (wp * yp)).sum(-2 if over_rows else -1))
    return torch.stack(cols, -1)


def _numerators(t, top):
    """2^(t - top) rounded once to FP32; masked places (t = -inf) and values below 2^-64 are zero."""
    x = t - top
    return torch.where(x >= TINY, torch.exp2(x), 0.0).float()


def _visible(rows, cols, q_len, k_len, causal, groups):
    """[sequence, 1, (group, rows), cols]: which keys each row sees; the last row sees the last key."""
    i = torch.arange(rows, device=q_len.device).repeat(groups)[None, :, None]
    j = torch.arange(cols, device=q_len.device)[None, None, :]
    see = (i < q_len[:, None, None]) & (j < k_len[:, None, None])
    if causal:
        see = see & (j <= i + (k_len - q_len)[:, None, None])
    return see[:, None]


def _attend(q, k, v, see, scale, tab, M):
    """o and lse of grouped, padded rows."""
    t = _scores(q, k, tab, M).double() * (scale * LOG2E)
    t = t.masked_fill(~see, -math.inf)
    top = torch.ceil(t.amax(-1, keepdim=True))
    top = torch.where(top > -math.inf, top, 0.0)
    e = _numerators(t, top)
    total = e.double().sum(-1, keepdim=True)
    o = _weighted(e, v, tab, M) / torch.where(total > 0, total, 1.0).float()
    lse = ((top + torch.log2(total)) / LOG2E).float()
    return o, lse[..., 0]


def _plain_forward(state):
    case, lengths, cu = state["case"], state["lengths"], state["cu"]
    K, M = case["kv_heads"], case["M"]
    (q, inside), (k, _), (v, _) = (_padded(state[x], lengths, cu) for x in "qkv")
    n = (cu[1:] - cu[:-1]).long()
    see = _visible(q.shape[2], k.shape[2], n, n, case["causal"], case["heads"] // K)
    o, lse = _attend(_group(q, K), k, v, see, case["dim"] ** -0.5, state["table"], M)
    return _packed(o.reshape(q.shape), inside), _packed(lse.reshape(q.shape[:3] + (1,)), inside)[..., 0]


def _plain_backward(state):
    case, lengths, cu, tab = state["case"], state["lengths"], state["cu"], state["table"]
    K, M, scale = case["kv_heads"], case["M"], case["dim"] ** -0.5
    (q, inside), (k, _), (v, _), (do, _) = (_padded(state[x], lengths, cu) for x in ("q", "k", "v", "do"))
    delta = (state["do"].double() * state["o"].double()).sum(-1, keepdim=True).float()
    (delta, _), (lse, _) = _padded(delta, lengths, cu), _padded(state["lse"][..., None], lengths, cu)
    n = (cu[1:] - cu[:-1]).long()
    see = _visible(q.shape[2], k.shape[2], n, n, case["causal"], case["heads"] // K)
    shape, q, do, delta, lse = q.shape, _group(q, K), _group(do, K), _group(delta, K), _group(lse, K)
    t = _scores(q, k, tab, M).double() * (scale * LOG2E)
    p = _numerators(t.masked_fill(~see, -math.inf), lse.double() * LOG2E)
    ds = (p.double() * (_scores(do, v, tab, M).double() - delta.double())).float()
    ds = torch.where(ds.abs() >= 2.0 ** TINY, ds, 0.0)
    dv = _weighted(p, do, tab, M, weight_first=False, over_rows=True)
    dk = _weighted(ds, q, tab, M, weight_first=False, over_rows=True) * scale
    dq = _weighted(ds, k, tab, M) * scale
    return _packed(dq.reshape(shape), inside), _packed(dk, inside), _packed(dv, inside)


def _plain_paged(state):
    case = state["case"]
    K, M, page = case["kv_heads"], case["M"], case["page"]
    q, inside = _padded(state["q"], state["new"], state["cu_q"])
    blocks = state["blocks"].clamp(min=0).long()
    k, v = (state[x][blocks].flatten(1, 2)[:, :max(state["lengths"])].transpose(1, 2) for x in ("k_pages", "v_pages"))
    n = (state["cu_q"][1:] - state["cu_q"][:-1]).long()
    see = _visible(q.shape[2], k.shape[2], n, state["k_len"].long(), True, case["heads"] // K)
    o, _ = _attend(_group(q, K), k, v, see, case["dim"] ** -0.5, state["table"], M)
    return _packed(o.reshape(q.shape), inside)


def _product(a, b, tab, M):
    """a b with table products, in pieces of the reduction that bound the memory."""
    (ai, ap), (bi, bp) = _parts(a, M), _parts(b, M)
    c = torch.zeros(a.shape[0], b.shape[1], dtype=torch.float32, device=a.device)
    step = max(1, min(64, (1 << 26) // max(1, c.numel())))
    for p in range(0, a.shape[1], step):
        at = slice(p, p + step)
        c += (tab[(ai[:, None, at] << M) | bi[at].t()[None]] * (ap[:, None, at] * bp[at].t()[None])).sum(-1)
    return c


def _activated(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z / (1 + torch.exp(-z)) if act == "silu" else z


def _slope(z, act):
    """The activation's derivative, in the type of z."""
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def _plain_dense_fwd(state):
    case = state["case"]
    z = _product(state["x"], state["w"], state["table"], case["M"])
    if state["bias"] is not None:
        z = z + state["bias"]
    y = _activated(z, case["act"])
    if state["residual"] is not None:
        y = y + state["residual"]
    return (y, z) if case["keep"] else y


def _plain_dense_bwd(state):
    case, tab = state["case"], state["table"]
    dz = (state["dy"].double() * _slope(state["z"].double(), case["act"])).float()
    dx = _product(dz, state["w"].t(), tab, case["M"])
    dw = _product(state["x"].t(), dz, tab, case["M"])
    return dx, dw, dz.double().sum(0).float() if case["bias"] else None


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        am = _load(case)
        if op == "attn_fwd":
            return am.attention_fwd(state["q"], state["k"], state["v"], state["cu"], state["cu"], causal=case["causal"])
        if op == "attn_bwd":
            return am.attention_bwd(state["do"], state["q"], state["k"], state["v"], state["o"], state["lse"], state["cu"],
                                    state["cu"], causal=case["causal"])
        if op == "paged":
            return am.attention_paged(state["q"], state["k_pages"], state["v_pages"], state["blocks"], state["cu_q"],
                                      state["k_len"])
        if op == "dense_fwd":
            return am.dense_fwd(state["x"], state["w"], bias=state["bias"], act=case["act"], residual=state["residual"],
                                keep_z=case["keep"])
        return am.dense_bwd(state["dy"], state["x"], state["w"], z=state["z"], act=case["act"], bias=case["bias"])
    plain = dict(attn_fwd=_plain_forward, attn_bwd=_plain_backward, paged=_plain_paged, dense_fwd=_plain_dense_fwd,
                 dense_bwd=_plain_dense_bwd)
    return plain[op](state)


# ------------------------------------------------------------------ work

def _pairs(q_lens, k_lens, causal):
    return sum(sum(max(0, min(nk, nk - nq + i + 1)) for i in range(nq)) if causal else nq * nk
               for nq, nk in zip(q_lens, k_lens))


def work(case):
    """A multiply-accumulate with a table product counts as two operations."""
    if case["op"] in ("dense_fwd", "dense_bwd"):
        m, n, k = case["m"], case["n"], case["k"]
        extra = n if case["bias"] else 0
        if case["op"] == "dense_fwd":
            return dict(bytes=4 * (m * k + k * n + m * n * (1 + case["residual"] + case["keep"]) + extra), flops=2 * m * n * k)
        return dict(bytes=4 * (2 * m * n + 2 * m * k + 2 * k * n + extra), flops=4 * m * n * k)
    lengths, H, K, D = _lengths(case), case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "paged":
        new = [min(case["new"], n) for n in lengths]
        return dict(bytes=4 * D * (2 * sum(new) * H + 2 * sum(lengths) * K), flops=4 * D * H * _pairs(new, lengths, True))
    T, pairs = sum(lengths), H * _pairs(lengths, lengths, case["causal"])
    if case["op"] == "attn_fwd":
        return dict(bytes=4 * T * (2 * H * D + 2 * K * D + H), flops=4 * D * pairs)
    return dict(bytes=4 * T * (4 * H * D + 4 * K * D + H), flops=10 * D * pairs)


# ------------------------------------------------------------------ the definition in 64 bits

class _Exact:
    """The multiplier: products of FP32 operands as 64-bit numbers, from frexp and the model's own formula."""

    def __init__(self, model, M):
        x = torch.arange(1 << M, dtype=torch.float64, device="cuda") / (1 << M)
        a, b = x[:, None] + 1, x[None, :] + 1
        p = torch.where(a + b < 3, a + b - 1, 2 * (a + b - 2)) if model == "mitchell" else a * b
        unit = torch.where(p < 2, 2.0 ** 15, 2.0 ** 14)
        self.flat, self.M = (torch.floor(p * unit) / unit).reshape(-1), M

    def operand(self, x):
        f, e = torch.frexp(x.double())                  # |f| in [1/2, 1)
        at = torch.floor((f.abs() * 2 - 1) * (1 << self.M)).clamp(min=0).long()
        unit = torch.sign(f) * torch.ldexp(torch.ones_like(f), e - 1)
        return at, torch.where(x.abs() >= 2.0 ** -126, unit, 0.0)

    def times(self, a, b):
        return self.flat[a[0] * (1 << self.M) + b[0]] * a[1] * b[1]


def _exact_sum(mul, a, b):
    """FP32 ascending sums by definition: each step's 64-bit sum (exact for two FP32 numbers' leading bits) rounded to FP32."""
    a, b = mul.operand(a), mul.operand(b)
    s = torch.zeros(a[0].shape[0], b[0].shape[0], dtype=torch.float64, device="cuda")
    for p in range(a[0].shape[1]):
        s = (s + mul.times([x[:, p, None] for x in a], [x[None, :, p] for x in b])).float().double()
    return s


def _exact_rows(mul, w, x, weight_first=True):
    """64-bit sums over j of products of w[i, j] with x[j, :], in pieces of j."""
    w, x = mul.operand(w), mul.operand(x)
    out = torch.zeros(w[0].shape[0], x[0].shape[1], dtype=torch.float64, device="cuda")
    step = max(1, (1 << 25) // max(1, out.numel()))
    for j in range(0, x[0].shape[0], step):
        a, b = [y[:, j:j + step, None] for y in w], [y[None, j:j + step] for y in x]
        out += (mul.times(a, b) if weight_first else mul.times(b, a)).sum(1)
    return out


def _exact_mask(nq, nk, causal):
    i, j = torch.arange(nq, device="cuda")[:, None], torch.arange(nk, device="cuda")[None]
    return (j <= i + nk - nq) if causal else torch.ones(nq, nk, dtype=torch.bool, device="cuda")


def _exact_attention(mul, q, k, v, scale, causal):
    see = _exact_mask(q.shape[0], k.shape[0], causal)
    x = torch.where(see, _exact_sum(mul, q, k) * scale / math.log(2), -math.inf)
    top = torch.ceil(x.max(1, keepdim=True).values)
    e = torch.pow(2.0, x - top)
    e = torch.where(e >= 2.0 ** TINY, e, 0.0).float()
    total = e.double().sum(1, keepdim=True)
    return _exact_rows(mul, e, v) / total, (top + torch.log2(total))[:, 0] * math.log(2)


def exact(case, seed):
    state = prepare(case, seed)
    mul = _Exact(case["model"], case["M"])
    if case["op"] == "dense_fwd":
        z = _exact_rows(mul, state["x"], state["w"])
        if state["bias"] is not None:
            z = z + state["bias"].double()
        act = dict(none=lambda u: u, relu=lambda u: torch.relu(u), silu=lambda u: u * torch.sigmoid(u),
                   gelu=lambda u: u * torch.special.ndtr(u))[case["act"]]
        y = act(z)
        if state["residual"] is not None:
            y = y + state["residual"].double()
        return (y, z) if case["keep"] else y
    if case["op"] == "dense_bwd":
        z = state["z"].double()
        gauss = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        sig = torch.sigmoid(z)
        slope = dict(none=lambda: torch.ones_like(z), relu=lambda: torch.sign(z).clamp(min=0),
                     silu=lambda: sig + z * sig * (1 - sig), gelu=lambda: torch.special.ndtr(z) + z * gauss)[case["act"]]()
        dz = (state["dy"].double() * slope).float()
        dx = _exact_rows(mul, dz, state["w"].t())
        dw = _exact_rows(mul, state["x"].t(), dz)
        return dx, dw, dz.double().sum(0) if case["bias"] else None
    H, K, scale = case["heads"], case["kv_heads"], 1 / math.sqrt(case["dim"])
    lengths = state["lengths"]
    if case["op"] == "paged":
        o = torch.zeros(state["q"].shape, dtype=torch.float64, device="cuda")
        at = 0
        for b, (n, new) in enumerate(zip(lengths, state["new"])):
            pages = [x for x in state["blocks"][b].tolist() if x >= 0]
            k, v = torch.cat([state["k_pages"][x] for x in pages])[:n], torch.cat([state["v_pages"][x] for x in pages])[:n]
            for h in range(H):
                o[at:at + new, h] = _exact_attention(mul, state["q"][at:at + new, h], k[:, h * K // H], v[:, h * K // H], scale, True)[0]
            at += new
        return o
    T, D = state["q"].shape[0], case["dim"]
    o, lse = torch.zeros(T, H, D, dtype=torch.float64, device="cuda"), torch.zeros(T, H, dtype=torch.float64, device="cuda")
    dq, dk, dv = torch.zeros_like(o), torch.zeros(T, K, D, dtype=torch.float64, device="cuda"), torch.zeros(T, K, D, dtype=torch.float64, device="cuda")
    at = 0
    for n in lengths:
        here = slice(at, at + n)
        at += n
        for h in range(H):
            g = h * K // H
            q, k, v = state["q"][here, h], state["k"][here, g], state["v"][here, g]
            if case["op"] == "attn_fwd":
                o[here, h], lse[here, h] = _exact_attention(mul, q, k, v, scale, case["causal"])
                continue
            do = state["do"][here, h]
            delta = (do.double() * state["o"][here, h].double()).sum(1).float().double()
            x = _exact_sum(mul, q, k) * scale - state["lse"][here, h, None].double()
            p = torch.where(_exact_mask(n, n, case["causal"]), torch.exp(x), 0.0)
            p = torch.where(p >= 2.0 ** TINY, p, 0.0).float()
            ds = (p.double() * (_exact_sum(mul, do, v) - delta[:, None])).float()
            ds = torch.where(ds.abs() >= 2.0 ** TINY, ds, 0.0)
            dq[here, h] = _exact_rows(mul, ds, k) * scale
            dk[here, g] += _exact_rows(mul, ds.t(), q, weight_first=False) * scale
            dv[here, g] += _exact_rows(mul, p.t(), do, weight_first=False)
    return (o, lse) if case["op"] == "attn_fwd" else (dq, dk, dv)
