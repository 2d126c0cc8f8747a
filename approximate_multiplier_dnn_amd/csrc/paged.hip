// paged.hip -- attention of new tokens over a paged cache with approximate
// products, gfx950.
#include "attention_device.h"

namespace amx {

// Few rows over many keys, read from the cache as it lies: a wave takes a
// block of NR rows (uniform operands, the products' first) and a chunk of
// keys, 64 at a time. Scores: one key per lane, its elements decoded as they
// are read. The numerators then go through LDS as Words, 16 keys at a time,
// and become the uniform operand of P V, whose lanes are the value's columns.
// Each key and value element is read once per row block and serves NR
// products; for a token or two the cache's bytes bound the kernel, for more
// rows the table lookups.
constexpr int kPagedKeys = 64;
template <int TAB>
constexpr int paged_threads()
{
    return TAB == AT_LDS8 ? 512 : 256;        // at M = 8 one workgroup's table fills a CU's LDS
}

// Range of the cache elements read: `big` the largest and `small` the least
// non-zero magnitude bits (shifted left by one, less one).
struct Seen {
    uint32_t big, small;
};

// Lane word of one cache element (fast path), folded into the range.
template <int TAB>
__device__ __forceinline__ void cache_word(uint32_t bits, int M, uint32_t& w, uint32_t& se, Seen& r)
{
    const uint32_t t = bits << 1;
    r.big = max(r.big, t);
    if constexpr (TAB == AT_NATIVE) {
        w = 0u;
        se = bits;
    } else {
        r.small = min(r.small, t - 1u);                // zero wraps past every magnitude
        w = t == 0u ? (2u << M) : (bits >> (22 - M)) & ((2u << M) - 2u);
        se = bits & 0xFF800000u;
    }
}

// A wave's item: rows r_lo .. r_end - 1 (up to NR) of one kv head, keys first
// .. last - 1 of their sequence.
template <int NR>
struct PagedSpan {
    int h, qs, r_lo, r_end, klen, lim_lo, first, last;
    const int* pages;
    const Word* q;

    __device__ __forceinline__ PagedSpan(const PagedParams& p, const Span& sp, int head, int split)
    {
        h = head;
        qs = sp.qs;
        r_lo = sp.qs * p.G + sp.tile * NR;
        r_end = min(r_lo + NR, (sp.qs + sp.qn) * p.G);
        klen = min(max(p.k_len[sp.seq], 0), p.table_ld * p.page);
        shift = klen - sp.qn + 1;
        lim_lo = limit(p, r_lo);
        first = split * p.chunk;
        last = min(limit(p, r_end - 1), first + p.chunk);
        pages = p.table + (int64_t)sp.seq * p.table_ld;
        q = p.q_flat + (int64_t)h * p.D4 * p.Fp + r_lo;
    }
    int shift;
    // row r sees keys below limit(r); rows past the block's end repeat the last
    __device__ __forceinline__ int limit(const PagedParams& p, int r) const
    {
        return p.causal ? min(klen, max(0, min(r, r_end - 1) / p.G - qs + shift)) : klen;
    }
    // This lane's key of the 64 from j0 on (below end): its row in the cache (of page 0
    // where there is none) and the rows that see it.
    __device__ __forceinline__ int place(const PagedParams& p, int j0, int end, uint32_t& in) const
    {
        const int j = j0 + (int)(threadIdx.x & 63), key = min(j, end - 1);
        const int pg = (int)fdiv32((uint32_t)key, p.fd_page);
        const int page = pages[pg];
        const bool there = page >= 0 && page < p.num_pages && j < end;
        in = there ? (1u << NR) - 1u : 0u;
        if (there && key >= lim_lo) {
#pragma unroll
            for (int r = 0; r < NR; ++r)
                if (key >= limit(p, r_lo + r)) in &= ~(1u << r);
        }
        return (there ? page : 0) * p.page + (key - pg * p.page);
    }
    __device__ __forceinline__ const float* key_row(const PagedParams& p, int at) const
    {
        return p.kp + ((int64_t)at * p.K + h) * p.D;
    }
};

// Uniform words of one step: NR columns.
template <int NQ>
__device__ __forceinline__ void load_columns(const void* row, uint32_t (&q)[NQ])
{
    const uint4* src = reinterpret_cast<const uint4*>(row) + (threadIdx.x & 3u);
    const uint4 a = src[0];
    q[0] = a.x; q[1] = a.y; q[2] = a.z; q[3] = a.w;
    if constexpr (NQ == 8) {
        const uint4 b = src[4];
        q[4] = b.x; q[5] = b.y; q[6] = b.z; q[7] = b.w;
    }
}

// Four elements of a key, zero from D on.
__device__ __forceinline__ uint4 key_four(const PagedParams& p, const float* row, int d)
{
    if (p.vec) return *reinterpret_cast<const uint4*>(row + d);
    uint4 x;
    x.x = d < p.D ? __float_as_uint(row[d]) : 0u;
    x.y = d + 1 < p.D ? __float_as_uint(row[d + 1]) : 0u;
    x.z = d + 2 < p.D ? __float_as_uint(row[d + 2]) : 0u;
    x.w = d + 3 < p.D ? __float_as_uint(row[d + 3]) : 0u;
    return x;
}

// Words of 16 lanes' numerators into LDS ([16][NR]); absent: the word of a
// row that does not see the key.
constexpr uint32_t kAbsent = 0xFFFFFFFFu;
template <int NR>
__device__ __forceinline__ void put_numerators(const PagedParams& p, const float (&e)[NR], uint32_t in, bool mark, uint32_t* buf)
{
    uint32_t* dst = buf + (threadIdx.x & 15) * 2 * NR;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        int lo = 0, hi = 0;
        const Word o = attn_word(__float_as_uint(e[r]), p.M, false, p.elo, p.ehi, lo, hi);
        dst[2 * r] = mark && !((in >> r) & 1u) ? kAbsent : o.w;
        dst[2 * r + 1] = o.se;
    }
}

template <int TAB, int NR, int VC>
__device__ __forceinline__ void paged_store(const PagedParams& p, const PagedSpan<NR>& b, int split, int v0, const float (&acc)[VC][NR],
                                            const double (&m)[NR], const double (&l)[NR], uint32_t bad)
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        double t = l[r];
        for (int off = 32; off > 0; off >>= 1) t += __shfl_xor(t, off, 64);
        if (__any((bad >> r) & 1u)) t = __builtin_nan("");
        if (b.r_lo + r >= b.r_end) continue;
        const int row = b.r_lo + r;
        if (p.splits > 1) {
            const int64_t at = ((int64_t)split * p.K + b.h) * p.RQ + row;
            if (lane == 0) {
                p.part_m[at] = m[r];
                p.part_l[at] = t;
            }
            if (t != 0.0)
#pragma unroll
                for (int v = 0; v < VC; ++v) p.part0[at * p.Dp + lane + 64 * (v0 + v)] = acc[v][r];
        } else {
            const int tok = row / p.G, hh = b.h * p.G + (row - tok * p.G);
            const float inv = t == 0.0 ? 0.0f : (float)(1.0 / t);
#pragma unroll
            for (int v = 0; v < VC; ++v)
                if (lane + 64 * (v0 + v) < p.D)
                    p.o[(int64_t)tok * p.ldo + (int64_t)hh * p.D + lane + 64 * (v0 + v)] = acc[v][r] * inv;
            if (p.lse != nullptr && lane == 0)
                p.lse[(int64_t)tok * (p.K * p.G) + hh] =
                    t == 0.0 ? -__builtin_inff() : (float)((m[r] + log2(t)) * 0.69314718055994530942);
        }
    }
}

// The item on the fast path; false (nothing written) when a key or value lies
// outside the fast range.
template <int TAB, int NR, int VC>
__device__ __forceinline__ bool paged_item(const PagedParams& p, const PagedSpan<NR>& b, int split, const unsigned char* lut,
                                           uint32_t* buf, int q_hi)
{
    constexpr int NQ = NR <= 8 ? 4 : 8;
    const int lane = threadIdx.x & 63;
    float acc[VC][NR];
    double m[NR], l[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        m[r] = -__builtin_inf();
        l[r] = 0.0;
#pragma unroll
        for (int v = 0; v < VC; ++v) acc[v][r] = 0.0f;
    }
    Seen ks{0u, 0xFFFFFFFFu}, vs{0u, 0xFFFFFFFFu};
    const int64_t step = (int64_t)p.K * p.D;
    const float* vbase = p.vp + (int64_t)b.h * p.D;
#pragma unroll 1
    for (int j0 = b.first; j0 < b.last; j0 += kPagedKeys) {
        uint32_t in;
        const int at = b.place(p, j0, b.last, in);
        const float* krow = b.key_row(p, at);
        float s[1][NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) s[0][r] = 0.0f;
        uint4 x = key_four(p, krow, 0);
#pragma unroll 1
        for (int d = 0; d < p.D4; d += 4) {
            uint32_t wa[4], sa[4], u[4][NQ];
#pragma unroll
            for (int i = 0; i < 4; ++i) load_columns(b.q + (int64_t)(d + i) * p.Fp, u[i]);
            const uint4 y = x;
            x = key_four(p, krow, min(d + 4, p.D4 - 4));
            cache_word<TAB>(y.x, p.M, wa[0], sa[0], ks);
            cache_word<TAB>(y.y, p.M, wa[1], sa[1], ks);
            cache_word<TAB>(y.z, p.M, wa[2], sa[2], ks);
            cache_word<TAB>(y.w, p.M, wa[3], sa[3], ks);
            fold<TAB, 4, 1, NR, NQ>(wa, sa, u, s, lut);
        }
        bool more = false;
#pragma unroll
        for (int r = 0; r < NR; ++r) more = more || (((in >> r) & 1u) && (double)s[0][r] * p.c > m[r]);
        if (__any(more)) {
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                float top = (in >> r) & 1u ? s[0][r] : -__builtin_inff();
                for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
                const double mn = fmax(m[r], __builtin_ceil((double)top * p.c));
                const int d = mn > m[r] ? (int)fmax(m[r] - mn, -4096.0) : 0;
                l[r] = __builtin_ldexp(l[r], d);
#pragma unroll
                for (int v = 0; v < VC; ++v) acc[v][r] = __builtin_ldexpf(acc[v][r], d);
                m[r] = mn;
            }
        }
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const float e = exp2_once(__builtin_fma((double)s[0][r], p.c, -m[r]));
            s[0][r] = (in >> r) & 1u ? e : 0.0f;
            l[r] += (double)s[0][r];
            if (r & 1) __builtin_amdgcn_sched_barrier(0);    // few temporaries at a time
        }
        // P V: the values' rows, 4 keys requested ahead
        const int count = min(kPagedKeys, b.last - j0);
        auto load = [&](int key, uint32_t (&w)[VC]) {
            const int64_t row = __builtin_amdgcn_readlane(at, key);
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                const int d = lane + 64 * v;
                w[v] = d < p.D ? __float_as_uint(vbase[row * step + d]) : 0u;
            }
        };
        uint32_t w[4][VC];
#pragma unroll
        for (int i = 0; i < 4; ++i) load(i, w[i]);
#pragma unroll 1
        for (int k0 = 0; k0 < count; k0 += 4) {
            if ((k0 & 15) == 0) {
                __builtin_amdgcn_wave_barrier();
                if ((lane & ~15) == k0) put_numerators(p, s[0], in, false, buf);
                __builtin_amdgcn_wave_barrier();
            }
            uint32_t y[4][VC];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int v = 0; v < VC; ++v) y[i][v] = w[i][v];
#pragma unroll
            for (int i = 0; i < 4; ++i) load(min(k0 + 4, kPagedKeys - 4) + i, w[i]);
            uint32_t u[4][NQ];
#pragma unroll
            for (int i = 0; i < 4; ++i) load_columns(buf + ((k0 & 15) + i) * 2 * NR, u[i]);
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                uint32_t wa[4], sa[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) cache_word<TAB>(y[i][v], p.M, wa[i], sa[i], vs);
                float(&a)[1][NR] = *reinterpret_cast<float(*)[1][NR]>(&acc[v]);
                fold<TAB, 4, 1, NR, NQ>(wa, sa, u, a, lut);
            }
        }
        const uint32_t most = (uint32_t)min(kFastHi, p.smax - q_hi);
        const uint32_t least = ((uint32_t)kFastLo << 24) - 1u;
        if (__any(ks.big >> 24 > most || vs.big >> 24 > (uint32_t)kFastHi || ks.small < least || vs.small < least)) return false;
    }
    paged_store<TAB, NR, VC>(p, b, split, 0, acc, m, l, 0u);
    return true;
}

// Scores of this lane's key on the checked path.
template <int TAB, int NR>
__device__ __forceinline__ void paged_scores_checked(const PagedParams& p, const PagedSpan<NR>& b, const float* krow, float (&s)[NR],
                                                     const unsigned char* lut)
{
#pragma unroll
    for (int r = 0; r < NR; ++r) s[r] = 0.0f;
#pragma unroll 1
    for (int d = 0; d < p.D; ++d) {
        int lo = 0, hi = 0;
        uint32_t u[NR <= 8 ? 4 : 8];
        load_columns(b.q + (int64_t)d * p.Fp, u);
        const Word w = attn_word(__float_as_uint(krow[d]), p.M, true, p.elo, p.ehi, lo, hi);
        fold_checked<TAB>(w.w, w.se, u, s, lut, p.elo, p.ehi, true);
    }
}

// The same on the checked path, kept small rather than fast: 64 columns of
// the values at a time, the scores computed again for each. As in the packed
// forward pass, the rows' maxima over all their keys come first.
template <int TAB, int NR>
__device__ __forceinline__ void paged_item_checked(const PagedParams& p, const PagedSpan<NR>& b, int split, const unsigned char* lut,
                                                   uint32_t* buf)
{
    constexpr int NQ = NR <= 8 ? 4 : 8;
    const int lane = threadIdx.x & 63;
    const int all = b.limit(p, b.r_end - 1);
    double m[NR];
    float top[NR];
    uint32_t bad = 0u;                              // bit r: a seen score of row r is NaN or +Inf
#pragma unroll
    for (int r = 0; r < NR; ++r) top[r] = -__builtin_inff();
#pragma unroll 1
    for (int j0 = 0; j0 < all; j0 += kPagedKeys) {
        uint32_t in;
        float s[NR];
        const int at = b.place(p, j0, all, in);
        paged_scores_checked<TAB, NR>(p, b, b.key_row(p, at), s, lut);
#pragma unroll
        for (int r = 0; r < NR; ++r)
            if ((in >> r) & 1u) {
                if (s[r] < __builtin_inff()) top[r] = fmaxf(top[r], s[r]);
                else bad |= 1u << r;
            }
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        for (int off = 32; off > 0; off >>= 1) top[r] = fmaxf(top[r], __shfl_xor(top[r], off, 64));
        m[r] = __builtin_ceil((double)top[r] * p.c);
    }
#pragma unroll 1
    for (int v = 0; v < p.Dp / 64; ++v) {
        float acc[1][NR];
        double l[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            l[r] = 0.0;
            acc[0][r] = 0.0f;
        }
#pragma unroll 1
        for (int j0 = b.first; j0 < b.last; j0 += kPagedKeys) {
            uint32_t in;
            float s[NR];
            const int at = b.place(p, j0, b.last, in);
            paged_scores_checked<TAB, NR>(p, b, b.key_row(p, at), s, lut);
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const float e = exp2_once(__builtin_fma((double)s[r], p.c, -m[r]));
                s[r] = ((in >> r) & 1u) && s[r] < __builtin_inff() ? e : 0.0f;
                l[r] += (double)s[r];
            }
            const int count = min(kPagedKeys, b.last - j0), d = lane + 64 * v;
#pragma unroll 1
            for (int k = 0; k < count; ++k) {
                if ((k & 15) == 0) {
                    __builtin_amdgcn_wave_barrier();
                    if ((lane & ~15) == k) put_numerators(p, s, in, true, buf);
                    __builtin_amdgcn_wave_barrier();
                }
                const int64_t row = __builtin_amdgcn_readlane(at, k);
                int lo = 0, hi = 0;
                const Word w = attn_word(d < p.D ? __float_as_uint(p.vp[(row * p.K + b.h) * p.D + d]) : 0u, p.M, true, p.elo, p.ehi, lo, hi);
                uint32_t u[NQ];
                load_columns(buf + (k & 15) * 2 * NR, u);
                // rows that do not see the key: no lookup of the mark, no part in the sum
                uint32_t cols = 0u;
#pragma unroll
                for (int r = 0; r < NR; ++r) cols |= uniform_word(u, r, 0) != kAbsent ? 1u << r : 0u;
#pragma unroll
                for (int i = 0; i < NQ; i += 2) u[i] = u[i] == kAbsent ? 0u : u[i];
                fold_checked<TAB>(w.w, w.se, u, acc[0], lut, p.elo, p.ehi, true, cols);
            }
        }
        paged_store<TAB, NR, 1>(p, b, split, v, acc, m, l, bad);
    }
}

template <int TAB, int NR, int VC>
__global__ __launch_bounds__(paged_threads<TAB>(), 2) void attn_paged_kernel(PagedParams p)
{
    constexpr int W = paged_threads<TAB>() / 64;
    __shared__ __align__(16) unsigned char lds[table_lds<TAB>() + 16];
    // a step's columns are read as 8 or 16 Words: the last row's may pass NR
    __shared__ __align__(16) uint32_t words[W][16 * NR * 2 + 8];
    const unsigned char* lut = stage_table<TAB>(p.lut, p.M, lds);
    int q_lo, q_hi;
    tensor_range(p.stats, 0, q_lo, q_hi);
    const bool q_fast = !p.force_checked && p.elo == 1 && range_fast<TAB>(q_lo, q_hi) && q_hi < p.smax;
    for (int64_t itm = (int64_t)blockIdx.x * W + (threadIdx.x >> 6); itm < p.items; itm += (int64_t)gridDim.x * W) {
        const int item = __builtin_amdgcn_readfirstlane((int)itm);
        const int h = item % p.K, r = item / p.K;
        const int split = r % p.splits, t = r / p.splits;
        const Span sp = find_tile(p.cu_q, p.total_q, p.cu_q, p.total_q, p.nseq, false, p.G, NR, t);
        if (sp.tile < 0) continue;
        const PagedSpan<NR> b(p, sp, h, split);
        uint32_t* buf = words[__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)];
        if (!q_fast || !paged_item<TAB, NR, VC>(p, b, split, lut, buf, q_hi)) paged_item_checked<TAB, NR>(p, b, split, lut, buf);
    }
}

template <int TAB, int NR, int VC>
static hipError_t run_paged(const PagedParams& p, hipStream_t s)
{
    static Resident cache;
    constexpr int NT = paged_threads<TAB>();
    const int64_t want = (p.items + NT / 64 - 1) / (NT / 64);
    const int grid = (int)std::min<int64_t>(want, resident(cache, 0, reinterpret_cast<const void*>(&attn_paged_kernel<TAB, NR, VC>), NT, 0));
    if (grid < 1) return hipErrorInvalidValue;
    attn_paged_kernel<TAB, NR, VC><<<grid, NT, 0, s>>>(p);
    return hipGetLastError();
}

template <int TAB>
static hipError_t run_paged_rows(const PagedParams& p, hipStream_t s)
{
    if (p.Dp <= 64)
        return p.NR == 4 ? run_paged<TAB, 4, 1>(p, s) : p.NR == 8 ? run_paged<TAB, 8, 1>(p, s) : run_paged<TAB, 16, 1>(p, s);
    return p.NR == 4 ? run_paged<TAB, 4, 2>(p, s) : p.NR == 8 ? run_paged<TAB, 8, 2>(p, s) : run_paged<TAB, 16, 2>(p, s);
}

hipError_t launch_attn_paged(const PagedParams& p, hipStream_t s)
{
    hipError_t e;
    switch (attn_table_kind(p.M)) {
    case AT_LDS: e = run_paged_rows<AT_LDS>(p, s); break;
    case AT_LDS8: e = run_paged_rows<AT_LDS8>(p, s); break;
    case AT_GLOBAL: e = run_paged_rows<AT_GLOBAL>(p, s); break;
    default: e = run_paged_rows<AT_NATIVE>(p, s); break;
    }
    if (e != hipSuccess || p.splits == 1) return e;
    return launch_join(AttnJoinParams{p.cu_q, p.nseq, p.K, p.G, p.D, p.Dp, p.total_q, p.RQ, p.splits, p.part0, p.part_m,
                                      p.part_l, p.o, p.ldo, p.lse}, s);
}

}  // namespace amx
