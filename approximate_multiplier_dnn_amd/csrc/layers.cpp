// layers.cpp -- the C ABI's attention and dense-layer calls: argument checks,
// panel layouts in the stream's scratch arena, and launch plans. Every
// arithmetic step runs in attention.hip, paged.hip, dense.hip and kernels.hip.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/approx_mul.h"
#include "attention.h"
#include "dense.h"
#include "host.h"

namespace {

using amx::AttnDecodeParams;
using amx::AttnParams;
using amx::AttnTensor;
using amx::HostTable;
using amx::Word;

constexpr double kLog2e = 1.4426950408889634074;
constexpr int64_t kMaxRows = (int64_t)1 << 30;
// Scales whose 64-bit scores and FP32 gradients stay in range.
constexpr double kLeastScale = 0x1p-100, kMostScale = 0x1p100;
// Rows per sequence (tokens x heads of a group) from which a paged call
// decodes the cache into panels for the packed kernel, and the panels' limit.
// Four chunks of 128 tokens (256 rows) over up to 4000 keys: 510 us in blocks
// of 16 rows, 300 us in panels.
constexpr int64_t kPanelRows = 24;
constexpr int64_t kPanelBytes = (int64_t)4 << 30;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return cdiv(a, b) * b; }

// Hands out 256-byte aligned parts of one scratch request: run once without
// memory to get its size, then with it.
struct Carver {
    char* base = nullptr;
    size_t used = 0;
    template <typename T>
    T* take(int64_t count)
    {
        T* p = base == nullptr ? nullptr : reinterpret_cast<T*>(base + used);
        used += (size_t)round_up((int64_t)sizeof(T) * count, 256);
        return p;
    }
};

// Argument checks shared by the attention calls. ld*: floats between tokens.
int check_heads(int nseq, int heads, int kv_heads, int dim, int total_q, double scale)
{
    if (nseq < 0 || heads < 1 || kv_heads < 1 || heads % kv_heads != 0 || dim < 1 || total_q < 0) return APPROX_EINVAL;
    if (!(scale >= kLeastScale && scale <= kMostScale)) return APPROX_EINVAL;      // NaN too
    if (dim > amx::kAttnMaxDim) return APPROX_EUNSUPPORTED;
    if ((int64_t)total_q * heads >= kMaxRows) return APPROX_EUNSUPPORTED;
    return APPROX_OK;
}

bool too_small(int ld, int heads, int dim) { return ld < (int64_t)heads * dim; }

// Largest sum of the biased exponents of q and k for which |c s| stays below
// 2^40: |s| < 2^(sum - 254 + 2) * 128.
int score_limit(double c) { return 254 + 40 - 9 - (int)std::ceil(std::log2(c)); }

// Chunks of each tile's range, so that the items (tiles x chunks) are about
// 2304 (three or more for each workgroup's turn at the counter), and a chunk
// keeps at least two steps of 16 NW of the average range. A function of the
// shapes only.
int split_for(int64_t tiles, int64_t blocks, int NW)
{
    constexpr int64_t kItems = 2304;
    const int64_t want = cdiv(kItems, std::max<int64_t>(1, tiles));
    return (int)std::max<int64_t>(1, std::min<int64_t>({want, blocks / (2 * NW), amx::kAttnMaxSplits}));
}

struct Shape {
    int nseq, H, K, D, total_q, total_k, causal;
    double scale;
    const int *cu_q, *cu_k;
};

void fill_common(AttnParams& p, const Shape& s, const HostTable& t)
{
    p.cu_q = s.cu_q;
    p.cu_k = s.cu_k;
    p.nseq = s.nseq;
    p.K = s.K;
    p.G = s.H / s.K;
    p.D = s.D;
    p.D4 = (int)round_up(s.D, 4);
    p.Dp = (int)round_up(s.D, 16);
    p.NW = p.Dp / 16;
    p.total_q = s.total_q;
    p.total_k = s.total_k;
    p.RQ = s.total_q * p.G;
    p.RQp = (int)round_up(p.RQ, amx::kAttnTile);
    p.TKp = (int)round_up(std::max(s.total_k, 1), amx::kAttnTile);
    p.causal = s.causal;
    p.c = s.scale * kLog2e;
    p.scale = (float)s.scale;
    p.M = t.M;
    p.elo = t.elo;
    p.ehi = t.ehi;
    p.smax = score_limit(p.c);
    p.force_checked = t.force_checked;
}

enum PanelKind { LANE, TR, ROW };

Word* panel(Carver& c, const AttnParams& p, int Rp, PanelKind kind)
{
    return c.take<Word>((int64_t)p.K * Rp * (kind == ROW ? p.Dp : p.D4));
}

AttnTensor tensor(const float* src, int ld, int R, int G, int Rp)
{
    AttnTensor t{};
    t.src = src;
    t.ld = ld;
    t.R = R;
    t.G = G;
    t.fd_G = amx::make_fastdiv((uint32_t)G);
    t.Rp = Rp;
    return t;
}

void fill_decode(AttnDecodeParams& d, const AttnParams& p)
{
    d.K = p.K;
    d.D = p.D;
    d.D4 = p.D4;
    d.Dp = p.Dp;
    d.M = p.M;
    d.elo = p.elo;
    d.ehi = p.ehi;
}

// The packed forward pass: p's geometry and outputs, d's three tensors.
// blocks: 16-key blocks of an average sequence.
int run_forward(AttnParams& p, AttnDecodeParams& d, int64_t blocks, const HostTable& t, hipStream_t stream)
{
    p.lut = t.lane_first;
    p.tiles = (int)(cdiv(p.RQ, amx::kAttnTile) + p.nseq);
    p.splits = split_for(cdiv(p.RQ, amx::kAttnTile) * p.K, blocks, p.NW);
    if ((int64_t)p.tiles * p.K * p.splits >= INT32_MAX / 2) return APPROX_EUNSUPPORTED;
    fill_decode(d, p);
    d.count = 3;
    Carver c;
    for (int pass = 0; pass < 2; ++pass) {
        c.used = 0;
        d.stats = c.take<uint32_t>(4 * amx::kAttnSlots);
        d.next = c.take<int>(2);
        d.t[0].lane = panel(c, p, p.RQp, LANE);
        d.t[1].tr = panel(c, p, p.TKp, TR);
        d.t[2].row = panel(c, p, p.TKp, ROW);
        if (d.t[1].cache) d.cache.mask = c.take<uint16_t>(p.TKp / amx::kAttnBlock);
        if (p.splits > 1) {
            const int64_t rows = (int64_t)p.splits * p.K * p.RQ;
            p.part0 = c.take<float>(rows * p.Dp);
            p.part_m = c.take<double>(rows);
            p.part_l = c.take<double>(rows);
        }
        if (pass == 0) {
            const int rc = amx::host_scratch(t.dev, stream, c.used, &c.base);
            if (rc != APPROX_OK) return rc;
        }
    }
    p.stats = d.stats;
    p.next = d.next;
    p.q_lane = d.t[0].lane;
    p.k_tr = d.t[1].tr;
    p.v_row = d.t[2].row;
    p.k_mask = d.cache.mask;
    if (amx::launch_attn_decode(d, stream) != hipSuccess) return APPROX_EHIP;
    return amx::launch_attn_fwd(p, stream) == hipSuccess ? APPROX_OK : APPROX_EHIP;
}

}  // namespace

extern "C" int approx_attention_fwd(int nseq, int heads, int kv_heads, int dim, int total_q, int total_k,
                                    const int* cu_q, const int* cu_k, int causal, double scale, const float* q, int ldq,
                                    const float* k, int ldk, const float* v, int ldv, float* o, int ldo, float* lse,
                                    void* stream_v)
{
    int rc = check_heads(nseq, heads, kv_heads, dim, total_q, scale);
    if (rc != APPROX_OK) return rc;
    if (total_k < 0 || (causal != 0 && causal != 1)) return APPROX_EINVAL;
    if (too_small(ldq, heads, dim) || too_small(ldk, kv_heads, dim) || too_small(ldv, kv_heads, dim) ||
        too_small(ldo, heads, dim))
        return APPROX_EINVAL;
    if (total_k >= kMaxRows) return APPROX_EUNSUPPORTED;
    if (nseq == 0 || total_q == 0) return APPROX_OK;
    if (cu_q == nullptr || cu_k == nullptr || q == nullptr || o == nullptr) return APPROX_EINVAL;
    if (total_k > 0 && (k == nullptr || v == nullptr)) return APPROX_EINVAL;
    HostTable t;
    rc = amx::host_table(&t);
    if (rc != APPROX_OK) return rc;
    hipStream_t stream = static_cast<hipStream_t>(stream_v);

    AttnParams p{};
    fill_common(p, Shape{nseq, heads, kv_heads, dim, total_q, total_k, causal, scale, cu_q, cu_k}, t);
    p.o = o;
    p.ldo = ldo;
    p.lse = lse;
    AttnDecodeParams d{};
    d.t[0] = tensor(q, ldq, p.RQ, p.G, p.RQp);
    d.t[1] = tensor(k, ldk, total_k, 1, p.TKp);
    d.t[2] = tensor(v, ldv, total_k, 1, p.TKp);
    return run_forward(p, d, cdiv(total_k, (int64_t)amx::kAttnBlock * nseq), t, stream);
}

extern "C" int approx_attention_bwd(int nseq, int heads, int kv_heads, int dim, int total_q, int total_k,
                                    const int* cu_q, const int* cu_k, int causal, double scale, const float* q, int ldq,
                                    const float* k, int ldk, const float* v, int ldv, const float* o, int ldo,
                                    const float* dout, int lddo, const float* lse, float* dq, int lddq, float* dk,
                                    int lddk, float* dv, int lddv, void* stream_v)
{
    int rc = check_heads(nseq, heads, kv_heads, dim, total_q, scale);
    if (rc != APPROX_OK) return rc;
    if (total_k < 0 || (causal != 0 && causal != 1)) return APPROX_EINVAL;
    if (too_small(ldq, heads, dim) || too_small(ldk, kv_heads, dim) || too_small(ldv, kv_heads, dim) ||
        too_small(ldo, heads, dim) || too_small(lddo, heads, dim) || too_small(lddq, heads, dim) ||
        too_small(lddk, kv_heads, dim) || too_small(lddv, kv_heads, dim))
        return APPROX_EINVAL;
    if (total_k >= kMaxRows) return APPROX_EUNSUPPORTED;
    if (nseq == 0 || (total_q == 0 && total_k == 0)) return APPROX_OK;
    if (cu_q == nullptr || cu_k == nullptr) return APPROX_EINVAL;
    if (total_q > 0 && (q == nullptr || o == nullptr || dout == nullptr || lse == nullptr || dq == nullptr)) return APPROX_EINVAL;
    if (total_k > 0 && (k == nullptr || v == nullptr || dk == nullptr || dv == nullptr)) return APPROX_EINVAL;
    HostTable t;
    rc = amx::host_table(&t);
    if (rc != APPROX_OK) return rc;
    hipStream_t stream = static_cast<hipStream_t>(stream_v);

    AttnParams p{};
    fill_common(p, Shape{nseq, heads, kv_heads, dim, total_q, total_k, causal, scale, cu_q, cu_k}, t);
    p.RQp = std::max(p.RQp, amx::kAttnTile);
    p.dq = dq;
    p.dk = dk;
    p.dv = dv;
    p.lddq = lddq;
    p.lddk = lddk;
    p.lddv = lddv;
    AttnParams kp = p;               // the keys' pass
    p.lut = t.lane_first;
    kp.lut = t.uniform_first;
    p.tiles = (int)(cdiv(p.RQ, amx::kAttnTile) + nseq);
    kp.tiles = (int)(cdiv(total_k, amx::kAttnTile) + nseq);
    p.splits = split_for(cdiv(p.RQ, amx::kAttnTile) * p.K, cdiv(total_k, (int64_t)amx::kAttnBlock * nseq), p.NW);
    kp.splits = split_for(cdiv(total_k, amx::kAttnTile) * p.K, cdiv(p.RQ, (int64_t)amx::kAttnBlock * nseq), p.NW);
    if ((int64_t)p.tiles * p.K * p.splits >= INT32_MAX / 2 || (int64_t)kp.tiles * p.K * kp.splits >= INT32_MAX / 2)
        return APPROX_EUNSUPPORTED;

    AttnDecodeParams d{};
    fill_decode(d, p);
    d.count = 4;
    d.t[0] = tensor(q, ldq, p.RQ, p.G, p.RQp);
    d.t[1] = tensor(dout, lddo, p.RQ, p.G, p.RQp);
    d.t[2] = tensor(k, ldk, total_k, 1, p.TKp);
    d.t[3] = tensor(v, ldv, total_k, 1, p.TKp);
    d.o = o;
    d.ldo = ldo;
    d.lse = lse;
    Carver c;
    for (int pass = 0; pass < 2; ++pass) {
        c.used = 0;
        d.stats = c.take<uint32_t>(4 * amx::kAttnSlots);
        d.next = c.take<int>(2);
        for (int i = 0; i < 4; ++i) {
            d.t[i].lane = panel(c, p, d.t[i].Rp, LANE);
            d.t[i].tr = panel(c, p, d.t[i].Rp, TR);
            d.t[i].row = i == 3 ? nullptr : panel(c, p, d.t[i].Rp, ROW);
        }
        d.delta = c.take<float>((int64_t)p.K * p.RQp);
        d.rowlse = c.take<float>((int64_t)p.K * p.RQp);
        // both passes' partials share one place: dQ is summed before the keys' pass starts
        const size_t before = c.used;
        if (p.splits > 1) p.part0 = c.take<float>((int64_t)p.splits * p.K * p.RQ * p.Dp);
        const size_t after = c.used;
        c.used = before;
        if (kp.splits > 1) {
            kp.part0 = c.take<float>((int64_t)kp.splits * p.K * total_k * p.Dp);
            kp.part1 = c.take<float>((int64_t)kp.splits * p.K * total_k * p.Dp);
        }
        c.used = std::max(c.used, after);
        if (pass == 0) {
            rc = amx::host_scratch(t.dev, stream, c.used, &c.base);
            if (rc != APPROX_OK) return rc;
        }
    }
    for (AttnParams* a : {&p, &kp}) {
        a->stats = d.stats;
        a->next = a == &p ? d.next : d.next + 1;
        a->q_lane = d.t[0].lane; a->q_tr = d.t[0].tr; a->q_row = d.t[0].row;
        a->do_lane = d.t[1].lane; a->do_tr = d.t[1].tr; a->do_row = d.t[1].row;
        a->k_lane = d.t[2].lane; a->k_tr = d.t[2].tr; a->k_row = d.t[2].row;
        a->v_lane = d.t[3].lane; a->v_tr = d.t[3].tr;
        a->delta = d.delta;
        a->rowlse = d.rowlse;
    }
    if (amx::launch_attn_decode(d, stream) != hipSuccess) return APPROX_EHIP;
    if (total_q > 0 && amx::launch_attn_bwd(p, false, stream) != hipSuccess) return APPROX_EHIP;
    if (total_k > 0 && amx::launch_attn_bwd(kp, true, stream) != hipSuccess) return APPROX_EHIP;
    return APPROX_OK;
}

extern "C" int approx_attention_paged(int nseq, int heads, int kv_heads, int dim, int total_q, const int* cu_q,
                                      int num_pages, int page, const float* k_pages, const float* v_pages,
                                      const int* block_table, int table_ld, const int* k_len, int causal, double scale,
                                      const float* q, int ldq, float* o, int ldo, float* lse, void* stream_v)
{
    int rc = check_heads(nseq, heads, kv_heads, dim, total_q, scale);
    if (rc != APPROX_OK) return rc;
    if (num_pages < 0 || page < 1 || table_ld < 0 || (causal != 0 && causal != 1)) return APPROX_EINVAL;
    if (too_small(ldq, heads, dim) || too_small(ldo, heads, dim)) return APPROX_EINVAL;
    if ((int64_t)num_pages * page >= kMaxRows || (int64_t)table_ld * page >= kMaxRows) return APPROX_EUNSUPPORTED;
    if (nseq == 0 || total_q == 0) return APPROX_OK;
    if (cu_q == nullptr || k_len == nullptr || q == nullptr || o == nullptr) return APPROX_EINVAL;
    if (num_pages == 0) table_ld = 0;                 // no page: every row is empty
    if (table_ld > 0 && (block_table == nullptr || k_pages == nullptr || v_pages == nullptr)) return APPROX_EINVAL;
    HostTable t;
    rc = amx::host_table(&t);
    if (rc != APPROX_OK) return rc;
    hipStream_t stream = static_cast<hipStream_t>(stream_v);

    const int64_t rows = cdiv(total_q, nseq) * (heads / kv_heads);   // of an average sequence
    const int64_t stride = round_up((int64_t)table_ld * page, amx::kAttnTile), all = nseq * stride;
    const int64_t panels = all * kv_heads * (round_up(dim, 4) + round_up(dim, 16)) * (int64_t)sizeof(Word);
    if (rows >= kPanelRows && table_ld > 0 && all < kMaxRows && panels <= kPanelBytes) {
        // chunks: the cache's keys decoded once for all the rows, then the
        // packed forward pass
        AttnParams p{};
        fill_common(p, Shape{nseq, heads, kv_heads, dim, total_q, (int)all, causal, scale, cu_q, nullptr}, t);
        p.k_len = k_len;
        p.k_stride = (int)stride;
        p.k_most = table_ld * page;
        p.o = o;
        p.ldo = ldo;
        p.lse = lse;
        AttnDecodeParams d{};
        d.t[0] = tensor(q, ldq, p.RQ, p.G, p.RQp);
        d.t[1] = tensor(k_pages, dim * 4, (int)all, 1, p.TKp);
        d.t[2] = tensor(v_pages, dim * 4, (int)all, 1, p.TKp);
        d.t[1].cache = d.t[2].cache = 1;
        d.cache.k_len = k_len;
        d.cache.table = block_table;
        d.cache.table_ld = table_ld;
        d.cache.page = page;
        d.cache.num_pages = num_pages;
        d.cache.stride = (int)stride;
        d.cache.fd_page = amx::make_fastdiv((uint32_t)page);
        d.cache.fd_stride = amx::make_fastdiv((uint32_t)stride);
        return run_forward(p, d, stride / amx::kAttnBlock, t, stream);
    }

    amx::PagedParams p{};
    p.cu_q = cu_q;
    p.k_len = k_len;
    p.table = block_table;
    p.kp = k_pages;
    p.vp = v_pages;
    p.nseq = nseq;
    p.K = kv_heads;
    p.G = heads / kv_heads;
    p.D = dim;
    p.D4 = (int)round_up(dim, 4);
    p.Dp = (int)round_up(dim, 16);
    p.total_q = total_q;
    p.RQ = total_q * p.G;
    p.page = page;
    p.num_pages = num_pages;
    p.table_ld = table_ld;
    p.fd_page = amx::make_fastdiv((uint32_t)page);
    p.causal = causal;
    p.vec = dim % 4 == 0 && (reinterpret_cast<uintptr_t>(k_pages) & 15) == 0 ? 1 : 0;
    p.c = scale * kLog2e;
    p.M = t.M;
    p.elo = t.elo;
    p.ehi = t.ehi;
    p.smax = score_limit(p.c);
    p.force_checked = t.force_checked;
    p.lut = t.uniform_first;
    p.NR = rows <= 4 ? 4 : rows <= 8 ? 8 : 16;
    p.blocks = (int)(cdiv(p.RQ, p.NR) + nseq);
    const int64_t keys = std::max<int64_t>(1, (int64_t)table_ld * page);
    const int64_t heads_blocks = std::max<int64_t>(1, std::max<int64_t>(cdiv(p.RQ, p.NR), nseq) * p.K);
    const int64_t want = cdiv(256 * 12 * 2, heads_blocks);
    // 64 keys fill a wave; 32 when there are few items (a wave's time per item counts then)
    p.chunk = cdiv(keys, want) <= 32 ? 32 : (int)round_up(cdiv(keys, want), 64);
    p.splits = (int)cdiv(keys, p.chunk);
    if ((int64_t)p.blocks * p.K * p.splits >= INT32_MAX) return APPROX_EUNSUPPORTED;
    p.q = q;
    p.ldq = ldq;
    p.o = o;
    p.ldo = ldo;
    p.lse = lse;

    Carver c;
    for (int pass = 0; pass < 2 && p.splits > 1; ++pass) {
        c.used = 0;
        const int64_t n = (int64_t)p.splits * p.K * p.RQ;
        p.part0 = c.take<float>(n * p.Dp);
        p.part_m = c.take<double>(n);
        p.part_l = c.take<double>(n);
        if (pass == 0) {
            rc = amx::host_scratch(t.dev, stream, c.used, &c.base);
            if (rc != APPROX_OK) return rc;
        }
    }
    return amx::launch_attn_paged(p, stream) == hipSuccess ? APPROX_OK : APPROX_EHIP;
}

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

extern "C" int approx_dense_fwd(int m, int n, int k, const float* X, int ldx, const float* W, int ldw, const float* bias,
                                int act, const float* residual, int ldr, float* Y, int ldy, float* Z, int ldz, void* stream_v)
{
    if (act < 0 || act >= amx::ACT_COUNT) return APPROX_EINVAL;
    if (m < 0 || n < 0 || k < 0 || ldy < std::max(1, n)) return APPROX_EINVAL;
    if (residual != nullptr && ldr < std::max(1, n)) return APPROX_EINVAL;
    if (Z != nullptr && ldz < std::max(1, n)) return APPROX_EINVAL;
    if (m > 0 && n > 0 && Y == nullptr) return APPROX_EINVAL;
    // the sums go to Z when it is wanted, else to Y
    float* sums = Z != nullptr ? Z : Y;
    const int lds = Z != nullptr ? ldz : ldy;
    amx::EpilogueParams p{};
    p.sums = sums;
    p.bias = bias;
    p.residual = residual;
    p.z = Z;
    p.y = Y;
    p.lds = lds;
    p.ldr = ldr;
    p.ldz = ldz;
    p.ldy = ldy;
    p.m = m;
    p.n = n;
    p.act = act;
    p.vec = ((n | lds | ldy | (residual ? ldr : 0)) & 3) == 0 && aligned16(sums) && aligned16(Y) && aligned16(bias) && aligned16(residual);
    if (bias == nullptr && act == amx::ACT_NONE && residual == nullptr && Z == nullptr)
        return approx_gemm(0, 0, m, n, k, X, ldx, W, ldw, Y, ldy, stream_v);
    bool fused = false;
    const int rc = amx::host_dense(m, n, k, X, ldx, W, ldw, sums, lds, p, &fused, static_cast<hipStream_t>(stream_v));
    if (rc != APPROX_OK || m == 0 || n == 0 || fused) return rc;
    return amx::launch_epilogue(p, static_cast<hipStream_t>(stream_v)) == hipSuccess ? APPROX_OK : APPROX_EHIP;
}

extern "C" int approx_dense_bwd(int m, int n, int k, const float* X, int ldx, const float* W, int ldw, const float* Z, int ldz,
                                int act, const float* dY, int lddy, float* dX, int lddx, float* dW, int lddw, float* db,
                                void* stream_v)
{
    if (act < 0 || act >= amx::ACT_COUNT) return APPROX_EINVAL;
    if (m < 0 || n < 0 || k < 0 || lddy < std::max(1, n)) return APPROX_EINVAL;
    if (act != amx::ACT_NONE && ldz < std::max(1, n)) return APPROX_EINVAL;
    if (dX != nullptr && (lddx < std::max(1, k) || ldw < std::max(1, n))) return APPROX_EINVAL;
    if (dW != nullptr && (lddw < std::max(1, n) || ldx < std::max(1, k))) return APPROX_EINVAL;
    if (m > 0 && n > 0 && (dY == nullptr || (act != amx::ACT_NONE && Z == nullptr))) return APPROX_EINVAL;
    if (m > 0 && k > 0 && n > 0 && ((dX != nullptr && W == nullptr) || (dW != nullptr && X == nullptr))) return APPROX_EINVAL;
    HostTable t;
    int rc = amx::host_table(&t);
    if (rc != APPROX_OK) return rc;
    hipStream_t stream = static_cast<hipStream_t>(stream_v);
    const float* dz = dY;
    int lddz = lddy;
    if (n > 0 && (db != nullptr || (act != amx::ACT_NONE && m > 0))) {
        amx::DzParams p{};
        p.dy = dY;
        p.z = act != amx::ACT_NONE ? Z : nullptr;
        p.lddy = lddy;
        p.ldz = ldz;
        p.m = m;
        p.n = n;
        p.act = act;
        // about 1024 workgroups, at least 16 rows each
        p.rows = (int)std::max<int64_t>(16, cdiv((int64_t)m * cdiv(n, 64), 1024));
        const int64_t chunks = cdiv(std::max(m, 1), p.rows);
        Carver c;
        float* own = nullptr;
        for (int pass = 0; pass < 2; ++pass) {
            c.used = 0;
            own = act != amx::ACT_NONE ? c.take<float>((int64_t)m * n) : nullptr;
            p.part = db != nullptr ? c.take<double>(chunks * n) : nullptr;
            if (pass == 0) {
                rc = amx::host_kept(t.dev, stream, c.used, &c.base);
                if (rc != APPROX_OK) return rc;
            }
        }
        p.dz = own;
        if (amx::launch_dz(p, db, stream) != hipSuccess) return APPROX_EHIP;
        if (own != nullptr) {
            dz = own;
            lddz = n;
        }
    }
    // dX = dz W^T and dW = X^T dz in one grouped call
    int count = 0, tA[2], tB[2], ms[2], ns[2], ks[2], las[2], lbs[2], lcs[2];
    const float *As[2], *Bs[2];
    float* Cs[2];
    auto add = [&](int ta, int tb, int mm, int nn, int kk, const float* A, int la, const float* B, int lb, float* C, int lc) {
        if (mm == 0 || nn == 0) return;
        tA[count] = ta; tB[count] = tb; ms[count] = mm; ns[count] = nn; ks[count] = kk;
        As[count] = A; las[count] = la; Bs[count] = B; lbs[count] = lb; Cs[count] = C; lcs[count] = lc;
        ++count;
    };
    if (dX != nullptr) add(0, 1, m, k, n, dz, lddz, W, ldw, dX, lddx);
    if (dW != nullptr) add(1, 0, k, n, m, X, ldx, dz, lddz, dW, lddw);
    if (count == 0) return APPROX_OK;
    return approx_gemm_grouped(count, tA, tB, ms, ns, ks, As, las, Bs, lbs, Cs, lcs, stream_v);
}
