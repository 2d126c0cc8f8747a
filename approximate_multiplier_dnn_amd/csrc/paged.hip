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
// Waves of a workgroup: 4 (8 measured 326 against 263 us for 32 tokens over
// caches up to 8192 keys: its items end less evenly); at M = 8, where one
// workgroup's table fills a CU's LDS, 6 or 8.
template <int TAB>
constexpr int paged_waves(int NR)
{
    return TAB == AT_LDS8 ? (NR == 16 ? 6 : 8) : 4;
}

// Range of the cache elements read: `big` the largest and `small` the least
// non-zero magnitude bits (shifted left by one, less one).
struct Seen {
    uint32_t big, small;
};

// Lane word of one cache element (fast path), folded into the range.
template <int TAB>
__device__ __forceinline__ void cache_word(uint32_t bits, int M, uint32_t base, uint32_t& w, uint32_t& se, Seen& r)
{
    const uint32_t t = bits << 1;
    r.big = max(r.big, t);
    if constexpr (TAB == AT_NATIVE) {
        w = 0u;
        se = bits;
    } else {
        r.small = min(r.small, t - 1u);                // zero wraps past every magnitude
        w = base + (t == 0u ? (2u << M) : (bits >> (22 - M)) & ((2u << M) - 2u));
        se = bits & 0xFF800000u;
    }
}

// A wave's item: rows r_lo .. r_end - 1 (up to NR) of one kv head, keys first
// .. last - 1 of their sequence.
template <int NR>
struct PagedSpan {
    int h, qs, r_lo, r_end, klen, lim_lo, first, last;
    const int* pages;

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

// Joins the waves' results through LDS (in the table's place: every wave is
// done with it) and writes the rows: the outputs, or one partial per
// workgroup.
template <int NR, int VC>
struct JoinRegion {
    float sum[NR][64 * VC];
    double m[NR], l[NR];
};

template <int W, int NR, int VC>
__device__ __forceinline__ void paged_store(const PagedParams& p, const PagedSpan<NR>& b, int g, int groups, int wave,
                                            const float (&acc)[VC][NR], const double (&m)[NR], const double (&l)[NR], uint32_t bad,
                                            JoinRegion<NR, VC>* region)
{
    const int lane = threadIdx.x & 63;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        double t = l[r];
        for (int off = 32; off > 0; off >>= 1) t += __shfl_xor(t, off, 64);
        if (__any((bad >> r) & 1u)) t = __builtin_nan("");
        if (lane == 0) {
            region[wave].m[r] = m[r];
            region[wave].l[r] = t;
        }
#pragma unroll
        for (int v = 0; v < VC; ++v) region[wave].sum[r][lane + 64 * v] = acc[v][r];
    }
    __syncthreads();
    for (int r = wave; r < NR && b.r_lo + r < b.r_end; r += W) {
        double top = -__builtin_inf(), total = 0.0;
        for (int w = 0; w < W; ++w)
            if (region[w].l[r] != 0.0) top = fmax(top, region[w].m[r]);
        float sum[VC];
#pragma unroll
        for (int v = 0; v < VC; ++v) sum[v] = 0.0f;
        for (int w = 0; w < W; ++w) {
            const double lw = region[w].l[r];
            if (lw == 0.0) continue;                    // no key of its own
            const int d = (int)fmax(region[w].m[r] - top, -4096.0);
            total += __builtin_ldexp(lw, d);
#pragma unroll
            for (int v = 0; v < VC; ++v) sum[v] += __builtin_ldexpf(region[w].sum[r][lane + 64 * v], d);
        }
        const int row = b.r_lo + r;
        if (groups > 1) {
            const int64_t at = ((int64_t)g * p.K + b.h) * p.RQ + row;
            if (lane == 0) {
                p.part_m[at] = top;
                p.part_l[at] = total;
            }
#pragma unroll
            for (int v = 0; v < VC; ++v)
                if (lane + 64 * v < p.Dp) p.part0[at * p.Dp + lane + 64 * v] = sum[v];
        } else {
            const int tok = row / p.G, hh = b.h * p.G + (row - tok * p.G);
            const float inv = total == 0.0 ? 0.0f : (float)(1.0 / total);
#pragma unroll
            for (int v = 0; v < VC; ++v)
                if (lane + 64 * v < p.D) p.o[(int64_t)tok * p.ldo + (int64_t)hh * p.D + lane + 64 * v] = sum[v] * inv;
            if (p.lse != nullptr && lane == 0)
                p.lse[(int64_t)tok * (p.K * p.G) + hh] =
                    total == 0.0 ? -__builtin_inff() : (float)((top + log2(total)) * 0.69314718055994530942);
        }
    }
}

// A workgroup past a sequence's keys: no part in its rows' sums.
template <int NR>
__device__ __forceinline__ void paged_empty(const PagedParams& p, const PagedSpan<NR>& b, int g)
{
    const int r = b.r_lo + (int)threadIdx.x;
    if (r < b.r_end) p.part_l[((int64_t)g * p.K + b.h) * p.RQ + r] = 0.0;
}

// The item on the fast path; false when a key or value lies outside the fast
// range (then the results are not used). qw: the rows' uniform words [D4][NR] in LDS.
template <int TAB, int NR, int VC>
__device__ __forceinline__ bool paged_item(const PagedParams& p, const PagedSpan<NR>& b, const Table& lut, const uint32_t* qw,
                                           uint32_t* buf, int q_hi, float (&acc)[VC][NR], double (&m)[NR], double (&l)[NR])
{
    constexpr int NQ = NR <= 8 ? 4 : 8;
    constexpr int KB = 4;                              // 16-byte pieces of a key requested together
    constexpr int VK = VC == 1 ? 8 : 4;                // keys whose values are requested ahead
    const int lane = threadIdx.x & 63;
    Seen ks{0u, 0xFFFFFFFFu}, vs{0u, 0xFFFFFFFFu};
    const int64_t step = (int64_t)p.K * p.D;
    const float* vbase = p.vp + (int64_t)b.h * p.D;
#pragma unroll 1
    for (int j0 = b.first; j0 < b.last; j0 += kPagedKeys) {
        uint32_t in;
        const int at = b.place(p, j0, b.last, in);
        const float* krow = b.key_row(p, at);
        // Each lane reads its own key: a line's pieces are requested together,
        // while it is in the cache (one piece per step fetched every line
        // about eight times over)
        uint4 x[KB];
#pragma unroll
        for (int i = 0; i < KB; ++i) x[i] = key_four(p, krow, min(4 * i, p.D4 - 4));
        // the values of the first keys, requested before the scores' work
        auto load = [&](int key, uint32_t (&w)[VC]) {
            const int64_t row = __builtin_amdgcn_readlane(at, key);
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                const int d = lane + 64 * v;
                w[v] = d < p.D ? __float_as_uint(vbase[row * step + d]) : 0u;
            }
        };
        float s[1][NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) s[0][r] = 0.0f;
        uint32_t u[2][4][NQ];                          // the rows' words, four positions ahead
#pragma unroll
        for (int t = 0; t < 4; ++t) load_columns(qw + t * 2 * NR, u[0][t]);
#pragma unroll 1
        for (int d0 = 0; d0 < p.D4; d0 += 4 * KB) {
            uint4 y[KB];
#pragma unroll
            for (int i = 0; i < KB; ++i) y[i] = x[i];
            if (d0 + 4 * KB < p.D4) {
#pragma unroll
                for (int i = 0; i < KB; ++i) x[i] = key_four(p, krow, min(d0 + 4 * (KB + i), p.D4 - 4));
            }
#pragma unroll
            for (int i = 0; i < KB; ++i) {
                const int d = d0 + 4 * i;
                if (d < p.D4) {                        // uniform
                    uint32_t wa[4], sa[4];
                    const int next = min(d + 4, p.D4 - 4);
#pragma unroll
                    for (int t = 0; t < 4; ++t) load_columns(qw + (next + t) * 2 * NR, u[(i + 1) & 1][t]);
                    cache_word<TAB>(y[i].x, p.M, lut.lds, wa[0], sa[0], ks);
                    cache_word<TAB>(y[i].y, p.M, lut.lds, wa[1], sa[1], ks);
                    cache_word<TAB>(y[i].z, p.M, lut.lds, wa[2], sa[2], ks);
                    cache_word<TAB>(y[i].w, p.M, lut.lds, wa[3], sa[3], ks);
                    fold<TAB, 4, 1, NR, NQ>(wa, sa, u[i & 1], s, lut);
                }
            }
        }
        uint32_t w[VK][VC];
#pragma unroll
        for (int i = 0; i < VK; ++i) load(i, w[i]);
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
        const int count = min(kPagedKeys, b.last - j0);
#pragma unroll 1
        for (int k0 = 0; k0 < count; k0 += VK) {
            if ((k0 & 15) == 0) {
                __builtin_amdgcn_wave_barrier();
                if ((lane & ~15) == k0) put_numerators(p, s[0], in, false, buf);
                __builtin_amdgcn_wave_barrier();
            }
            uint32_t y[VK][VC], e[2][4][NQ];
#pragma unroll
            for (int i = 0; i < 4; ++i) load_columns(buf + ((k0 & 15) + i) * 2 * NR, e[0][i]);
#pragma unroll
            for (int i = 0; i < VK; ++i)
#pragma unroll
                for (int v = 0; v < VC; ++v) y[i][v] = w[i][v];
            if (k0 + VK < count) {
#pragma unroll
                for (int i = 0; i < VK; ++i) load(k0 + VK + i, w[i]);
            }
#pragma unroll
            for (int i = 0; i < 4 && VK > 4; ++i) load_columns(buf + ((k0 & 15) + 4 + i) * 2 * NR, e[1][i]);
#pragma unroll
            for (int h4 = 0; h4 < VK; h4 += 4) {
#pragma unroll
                for (int v = 0; v < VC; ++v) {
                    uint32_t wa[4], sa[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) cache_word<TAB>(y[h4 + i][v], p.M, lut.lds, wa[i], sa[i], vs);
                    float(&a)[1][NR] = *reinterpret_cast<float(*)[1][NR]>(&acc[v]);
                    fold<TAB, 4, 1, NR, NQ>(wa, sa, e[h4 / 4], a, lut);
                }
            }
        }
        const uint32_t most = (uint32_t)min(kFastHi, p.smax - q_hi);
        const uint32_t least = ((uint32_t)kFastLo << 24) - 1u;
        if (__any(ks.big >> 24 > most || vs.big >> 24 > (uint32_t)kFastHi || ks.small < least || vs.small < least)) return false;
    }
    return true;
}

// Scores of this lane's key on the checked path.
template <int TAB, int NR>
__device__ __forceinline__ void paged_scores_checked(const PagedParams& p, const uint32_t* qw, const float* krow, float (&s)[NR],
                                                     const Table& lut)
{
#pragma unroll
    for (int r = 0; r < NR; ++r) s[r] = 0.0f;
#pragma unroll 1
    for (int d = 0; d < p.D; ++d) {
        int lo = 0, hi = 0;
        uint32_t u[NR <= 8 ? 4 : 8];
        load_columns(qw + d * 2 * NR, u);
        const Word w = attn_word(__float_as_uint(krow[d]), p.M, true, p.elo, p.ehi, lo, hi);
        fold_checked<TAB>(w.w + lut.lds, w.se, u, s, lut, p.elo, p.ehi, true);
    }
}

// The same on the checked path, kept small rather than fast. As in the packed
// forward pass, the rows' maxima over all their keys come first. bad: bit r, a
// seen score of row r is NaN or +Inf.
template <int TAB, int NR, int VC>
__device__ __forceinline__ void paged_item_checked(const PagedParams& p, const PagedSpan<NR>& b, const Table& lut, const uint32_t* qw,
                                                   uint32_t* buf, float (&acc)[VC][NR], double (&m)[NR], double (&l)[NR], uint32_t& bad)
{
    constexpr int NQ = NR <= 8 ? 4 : 8;
    const int lane = threadIdx.x & 63;
    const int all = b.limit(p, b.r_end - 1);
    float top[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) top[r] = -__builtin_inff();
#pragma unroll 1
    for (int j0 = 0; j0 < all; j0 += kPagedKeys) {
        uint32_t in;
        float s[NR];
        const int at = b.place(p, j0, all, in);
        paged_scores_checked<TAB, NR>(p, qw, b.key_row(p, at), s, lut);
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
        l[r] = 0.0;
#pragma unroll
        for (int v = 0; v < VC; ++v) acc[v][r] = 0.0f;
    }
#pragma unroll 1
    for (int j0 = b.first; j0 < b.last; j0 += kPagedKeys) {
        uint32_t in;
        float s[NR];
        const int at = b.place(p, j0, b.last, in);
        paged_scores_checked<TAB, NR>(p, qw, b.key_row(p, at), s, lut);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const float e = exp2_once(__builtin_fma((double)s[r], p.c, -m[r]));
            s[r] = ((in >> r) & 1u) && s[r] < __builtin_inff() ? e : 0.0f;
            l[r] += (double)s[r];
        }
        const int count = min(kPagedKeys, b.last - j0);
#pragma unroll 1
        for (int k = 0; k < count; ++k) {
            if ((k & 15) == 0) {
                __builtin_amdgcn_wave_barrier();
                if ((lane & ~15) == k) put_numerators(p, s, in, true, buf);
                __builtin_amdgcn_wave_barrier();
            }
            const int64_t row = __builtin_amdgcn_readlane(at, k);
            uint32_t u[NQ];
            load_columns(buf + (k & 15) * 2 * NR, u);
            // rows that do not see the key: no lookup of the mark, no part in the sum
            uint32_t cols = 0u;
#pragma unroll
            for (int r = 0; r < NR; ++r) cols |= uniform_word(u, r, 0) != kAbsent ? 1u << r : 0u;
#pragma unroll
            for (int i = 0; i < NQ; i += 2) u[i] = u[i] == kAbsent ? 0u : u[i];
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                const int d = lane + 64 * v;
                int lo = 0, hi = 0;
                const Word w = attn_word(d < p.D ? __float_as_uint(p.vp[(row * p.K + b.h) * p.D + d]) : 0u, p.M, true, p.elo, p.ehi, lo, hi);
                fold_checked<TAB>(w.w + lut.lds, w.se, u, acc[v], lut, p.elo, p.ehi, true, cols);
            }
        }
    }
}

// Items: a block of rows of one kv head and W consecutive chunks of keys, one
// per wave. The rows are decoded into LDS once for the workgroup.
template <int TAB, int NR, int VC>
__global__ __launch_bounds__(64 * paged_waves<TAB>(NR), NR == 4 ? 4 : 2) void attn_paged_kernel(PagedParams p)
{
    constexpr int W = paged_waves<TAB>(NR);
    constexpr int kRegion = W * (int)sizeof(JoinRegion<NR, VC>);
    __shared__ __align__(16) unsigned char lds[table_lds<TAB>() > kRegion ? table_lds<TAB>() : kRegion];
    // a step's columns are read as 8 or 16 Words: the last row's may pass NR
    __shared__ __align__(16) uint32_t qw[kAttnMaxDim * NR * 2 + 16];
    __shared__ __align__(16) uint32_t words[W][16 * NR * 2 + 8];
    __shared__ int range[2 * W];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    uint32_t* buf = words[wave];
    // one item per workgroup: lengths differ, and the hardware hands out the
    // workgroups as others end (a persistent grid's fixed shares left half of
    // the waves idle at the end)
    const int groups = (p.splits + W - 1) / W;
    const int g = blockIdx.x % groups, r = blockIdx.x / groups;
    const int h = r % p.K, t = r / p.K;
    const Span sp = find_tile(p.cu_q, p.total_q, p.cu_q, p.total_q, p.nseq, false, p.G, NR, t);
    if (sp.tile < 0) return;
    const int r_lo = sp.qs * p.G + sp.tile * NR, r_end = min(r_lo + NR, (sp.qs + sp.qn) * p.G);
    const int split = g * W + wave;
    const PagedSpan<NR> b(p, sp, h, split);
    if (g > 0 && g * W * p.chunk >= b.limit(p, r_end - 1)) {
        paged_empty<NR>(p, b, g);
        return;
    }
    int lo = 255, hi = 0;
    for (int i = wave; i < NR; i += W) {
        const int row = min(r_lo + i, r_end - 1), tok = row / p.G;
        const float* src = p.q + (int64_t)tok * p.ldq + (int64_t)(h * p.G + row - tok * p.G) * p.D;
        for (int d = lane; d < p.D4; d += 64) {
            const Word w = attn_word(d < p.D && r_lo + i < r_end ? __float_as_uint(src[d]) : 0u, p.M, false, p.elo, p.ehi, lo, hi);
            *reinterpret_cast<uint2*>(qw + (d * NR + i) * 2) = make_uint2(w.w, w.se);
        }
    }
    for (int off = 32; off > 0; off >>= 1) {
        lo = min(lo, __shfl_xor(lo, off, 64));
        hi = max(hi, __shfl_xor(hi, off, 64));
    }
    if (lane == 0) {
        range[2 * wave] = lo;
        range[2 * wave + 1] = hi;
    }
    const Table lut = stage_table<TAB>(p.lut, p.M, lds);
    __syncthreads();
    for (int i = 0; i < W; ++i) {
        lo = min(lo, range[2 * i]);
        hi = max(hi, range[2 * i + 1]);
    }
    const bool q_fast = !p.force_checked && p.elo == 1 && range_fast<TAB>(lo, hi) && hi < p.smax;
    float acc[VC][NR];
    double m[NR], l[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        m[i] = -__builtin_inf();
        l[i] = 0.0;
#pragma unroll
        for (int v = 0; v < VC; ++v) acc[v][i] = 0.0f;
    }
    uint32_t bad = 0u;
    if (b.first < b.last && (!__any(q_fast) || !paged_item<TAB, NR, VC>(p, b, lut, qw, buf, hi, acc, m, l)))
        paged_item_checked<TAB, NR, VC>(p, b, lut, qw, buf, acc, m, l, bad);
    paged_store<W, NR, VC>(p, b, g, groups, wave, acc, m, l, bad, reinterpret_cast<JoinRegion<NR, VC>*>(lds));
}

template <int TAB, int NR, int VC>
static hipError_t run_paged(const PagedParams& p, hipStream_t s)
{
    constexpr int W = paged_waves<TAB>(NR);
    const int groups = (p.splits + W - 1) / W;
    attn_paged_kernel<TAB, NR, VC><<<(unsigned)((int64_t)p.blocks * p.K * groups), 64 * W, 0, s>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || groups == 1) return e;
    return launch_join(AttnJoinParams{p.cu_q, p.nseq, p.K, p.G, p.D, p.Dp, p.total_q, p.RQ, groups, p.part0, p.part_m,
                                      p.part_l, p.o, p.ldo, p.lse}, s);
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
    switch (attn_table_kind(p.M)) {
    case AT_LDS: return run_paged_rows<AT_LDS>(p, s);
    case AT_LDS8: return run_paged_rows<AT_LDS8>(p, s);
    case AT_GLOBAL: return run_paged_rows<AT_GLOBAL>(p, s);
    default: return run_paged_rows<AT_NATIVE>(p, s);
    }
}

}  // namespace amx
