// attention.hip -- attention with approximate products for gfx950: packed
// prompts (forward and backward).
//
// Forward, for a row i of a kv head (a token and a head of its group) and the
// keys j it sees:
//   s_ij = FP32 sum over d, ascending from +0, of T(q_id, k_jd)
//   E_ij = RN32(2^(c s_ij - m_i)), c = scale log2(e), m_i = ceil(max_j c s_ij)
//   o_id = sum_j T(E_ij, v_jd) / sum_j E_ij
// with T the loaded multiplier's product. The table sees only the top M
// fraction bits of E_ij, so E_ij is computed in 64 bits and rounded once (an
// error of one last place next to such a border would move the product by
// 2^-M). m_i is an integer: replacing a running maximum by a larger one
// scales the sums by a power of two and changes no mantissa, so one pass over
// the keys gives the two-pass result, and chunks of keys join exactly.
//
// A tile is 64 rows of a kv head, one per lane, and its waves share each step
// of 16 (or, in calls that leave the GPU mostly empty, 8) keys per wave: wave
// w computes the scores of its own keys, hands their numerators to the others
// through LDS, and sums its own 16 (or 8) value columns over all the step's
// keys. The keys, then the values' columns, are uniform operands spread over
// the lanes of each quad (product.h). What bounds the loops is the rate of
// table lookups (one 16-bit LDS read per product), as in the GEMM kernel.
#include "attention_device.h"

#include <cstdlib>

namespace amx {

// ------------------------------------------------------------------ decode

// Decodes 64 rows of one kv head per step through LDS into the panels asked
// for. Bound by HBM: 4 bytes read and 8 written per element and panel.
// (8192 tokens of 3 x 12 heads of 64, 226 MB: 50 us, 4.5 TB/s, where a large
// copy moves 4.9; with 256 workgroups per tensor and LDS for 128 columns, too
// few in flight: 66 us.)
constexpr int kDecodeThreads = 256;
__global__ __launch_bounds__(kDecodeThreads) void attn_decode_kernel(AttnDecodeParams p)
{
    extern __shared__ uint32_t tile[];               // [64][Dp + 1]
    __shared__ int range[2 * (kDecodeThreads / 64)];
    const AttnTensor& t = p.t[blockIdx.y];
    const int tid = threadIdx.x, S = p.Dp + 1;
    const int blocks = t.Rp / kAttnTile;
    const bool vec = ((t.ld | p.D) & 3) == 0 && (reinterpret_cast<uintptr_t>(t.src) & 15) == 0;
    if (p.next != nullptr && blockIdx.x == 0 && blockIdx.y == 0 && tid < 2) p.next[tid] = 0;   // the item counters
    int lo = 255, hi = 0;
    for (int64_t item = blockIdx.x; item < (int64_t)blocks * p.K; item += gridDim.x) {
        const int h = (int)(item / blocks), r0 = (int)(item - (int64_t)h * blocks) * kAttnTile;
        const AttnCache& ca = p.cache;
        int j0 = 0, klen = 0;                            // a cache's block: its keys j0 .. j0 + 63
        const int* pages = nullptr;
        if (t.cache) {
            const int b = (int)fdiv32((uint32_t)r0, ca.fd_stride);
            j0 = r0 - b * ca.stride;
            klen = min(max(ca.k_len[b], 0), ca.table_ld * ca.page);
            if (j0 >= klen) continue;                    // uniform
            pages = ca.table + (int64_t)b * ca.table_ld;
        }
        __syncthreads();
        // 16 or 32 threads per row (Dp <= 64 or 128), four elements each
        const int cols = p.Dp <= 64 ? 16 : 32, d = (tid & (cols - 1)) * 4;
        if (d < p.Dp) {
#pragma unroll 4
            for (int rr = tid / cols; rr < kAttnTile; rr += kDecodeThreads / cols) {
                const int r = r0 + rr;
                uint32_t x[4] = {0u, 0u, 0u, 0u};
                const float* src = nullptr;
                if (t.cache) {
                    const int j = j0 + rr, pg = (int)fdiv32((uint32_t)j, ca.fd_page);
                    const int page = j < klen ? pages[pg] : -1;
                    if (page >= 0 && page < ca.num_pages)
                        src = t.src + (((int64_t)page * ca.page + (j - pg * ca.page)) * p.K + h) * p.D + d;
                } else if (r < t.R) {
                    const int tok = (int)fdiv32((uint32_t)r, t.fd_G), hh = h * t.G + (r - tok * t.G);
                    src = t.src + (int64_t)tok * t.ld + (int64_t)hh * p.D + d;
                }
                if (src != nullptr) {
                    if (vec) {
                        if (d < p.D) {
                            const uint4 v = *reinterpret_cast<const uint4*>(src);
                            x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[i] = d + i < p.D ? __float_as_uint(src[i]) : 0u;
                    }
                }
                uint32_t* o = tile + rr * S + d;
                o[0] = x[0]; o[1] = x[1]; o[2] = x[2]; o[3] = x[3];
            }
        }
        if (t.cache && h == 0 && t.tr != nullptr && tid < kAttnTile) {
            const int j = j0 + tid, pg = (int)fdiv32((uint32_t)j, ca.fd_page);
            const int page = j < klen ? pages[pg] : -1;
            const uint64_t there = __ballot(page >= 0 && page < ca.num_pages);
            if (tid < kAttnTile / kAttnBlock) ca.mask[r0 / kAttnBlock + tid] = (uint16_t)(there >> (16 * tid));
        }
        __syncthreads();
        if (t.lane != nullptr) {
            Word* dst = t.lane + (int64_t)h * p.D4 * t.Rp;
            for (int i = tid; i < (p.D4 / 4) * kAttnTile; i += kDecodeThreads) {
                const int p4 = i / kAttnTile, rr = i & (kAttnTile - 1);
                uint4* o = reinterpret_cast<uint4*>(dst + ((int64_t)p4 * t.Rp + r0 + rr) * 4);
                Word w[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) w[x] = attn_word(tile[rr * S + p4 * 4 + x], p.M, true, p.elo, p.ehi, lo, hi);
                o[0] = make_uint4(w[0].w, w[0].se, w[1].w, w[1].se);
                o[1] = make_uint4(w[2].w, w[2].se, w[3].w, w[3].se);
            }
        }
        if (t.tr != nullptr) {
            Word* dst = t.tr + ((int64_t)h * t.Rp + r0) * p.D4;
            const int pair = tid & 7;
            for (int blk = 0; blk < kAttnTile / kAttnBlock; ++blk) {
                const int rr = blk * kAttnBlock + pair * 2;
                for (int d = tid >> 3; d < p.D4; d += kDecodeThreads / 8) {
                    const Word a = attn_word(tile[rr * S + d], p.M, false, p.elo, p.ehi, lo, hi);
                    const Word b = attn_word(tile[(rr + 1) * S + d], p.M, false, p.elo, p.ehi, lo, hi);
                    *reinterpret_cast<uint4*>(dst + ((int64_t)blk * p.D4 + d) * kAttnBlock + pair * 2) =
                        make_uint4(a.w, a.se, b.w, b.se);
                }
            }
        }
        if (t.row != nullptr) {
            Word* dst = t.row + (int64_t)h * t.Rp * p.Dp + (int64_t)r0 * CPW;
            for (int i = tid; i < kAttnTile * p.Dp / 2; i += kDecodeThreads) {
                const int g = i / (kAttnTile * 8), rr = (i >> 3) & (kAttnTile - 1), c = (i & 7) * 2, d = g * CPW + c;
                const Word a = attn_word(tile[rr * S + d], p.M, false, p.elo, p.ehi, lo, hi);
                const Word b = attn_word(tile[rr * S + d + 1], p.M, false, p.elo, p.ehi, lo, hi);
                *reinterpret_cast<uint4*>(dst + ((int64_t)g * t.Rp + rr) * CPW + c) = make_uint4(a.w, a.se, b.w, b.se);
            }
        }
        if (p.o != nullptr && blockIdx.y == 1) {
            // D_i = sum_d dO_id o_id, exact products summed in 64 bits, four
            // threads per row, rounded once
            const int rr = tid >> 2, r = r0 + rr;
            double sum = 0.0;
            if (r < t.R) {
                const int tok = (int)fdiv32((uint32_t)r, t.fd_G), hh = h * t.G + (r - tok * t.G);
                const float* o = p.o + (int64_t)tok * p.ldo + (int64_t)hh * p.D;
                for (int d = tid & 3; d < p.D; d += 4) sum += (double)__uint_as_float(tile[rr * S + d]) * (double)o[d];
                sum += __shfl_xor(sum, 1, 64);
                sum += __shfl_xor(sum, 2, 64);
                if ((tid & 3) == 0) {
                    hi = max(hi, (int)((__float_as_uint((float)sum) >> 23) & 0xFFu));
                    p.delta[(int64_t)h * t.Rp + r] = (float)sum;
                    p.rowlse[(int64_t)h * t.Rp + r] = p.lse[(int64_t)tok * (p.K * t.G) + hh];
                }
            }
        }
    }
    for (int off = 32; off > 0; off >>= 1) {
        lo = min(lo, __shfl_xor(lo, off, 64));
        hi = max(hi, __shfl_xor(hi, off, 64));
    }
    if ((tid & 63) == 0) {
        range[2 * (tid >> 6)] = lo;
        range[2 * (tid >> 6) + 1] = hi;
    }
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kDecodeThreads / 64; ++w) {
            lo = min(lo, range[2 * w]);
            hi = max(hi, range[2 * w + 1]);
        }
        p.stats[blockIdx.y * kAttnSlots + blockIdx.x] = (uint32_t)lo | ((uint32_t)hi << 8);
    }
}

// ------------------------------------------------------------------ tiles

// CW sums of a row: scaled into the output (its columns below D), or as a partial.
template <int CW>
__device__ __forceinline__ void store_row(const float (&acc)[1][CW], float scale, float* o, int D, bool vec)
{
#pragma unroll
    for (int d = 0; d < CW; d += 4) {
        if (vec) {
            if (d < D) *reinterpret_cast<float4*>(o + d) = make_float4(acc[0][d] * scale, acc[0][d + 1] * scale, acc[0][d + 2] * scale, acc[0][d + 3] * scale);
        } else {
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (d + x < D) o[d + x] = acc[0][d + x] * scale;
        }
    }
}

__device__ __forceinline__ bool rows_aligned(const float* o, int64_t ld, int D)
{
    return ((ld | D) & 3) == 0 && (reinterpret_cast<uintptr_t>(o) & 15) == 0;
}


// A chunk of a row tile's keys: blocks [b0, b1) of 16 packed keys.
__device__ __forceinline__ void chunk_blocks(int first, int last, int splits, int c, int& b0, int& b1)
{
    const int n = last - first, per = (n + splits - 1) / splits;
    b0 = min(last, first + c * per);
    b1 = min(last, b0 + per);
}

// A lane's row of a tile and the keys [ks, lim) it sees; lim_lo, lim_hi: the
// tile's least and largest limit (rows ascend with the lanes).
struct Row {
    int row, tok, lim, lim_lo, lim_hi;
    int f0, f1, b0, b1;                      // blocks of the tile's range and of this chunk
    bool valid;
};
__device__ __forceinline__ Row tile_row(const AttnParams& p, const Span& sp, int split)
{
    Row r;
    const int rend = (sp.qs + sp.qn) * p.G;
    const int raw = sp.qs * p.G + sp.tile * kAttnTile + (int)(threadIdx.x & 63);
    r.valid = raw < rend;
    r.row = min(raw, rend - 1);
    r.tok = r.row / p.G;
    const int ke = sp.ks + sp.kn;
    r.lim = p.causal ? min(ke, max(sp.ks, sp.ks + sp.kn - sp.qn + (r.tok - sp.qs) + 1)) : ke;
    r.lim_lo = __builtin_amdgcn_readlane(r.lim, 0);
    r.lim_hi = __builtin_amdgcn_readlane(r.lim, 63);
    r.f0 = sp.ks / kAttnBlock;
    r.f1 = r.lim_hi > sp.ks ? (r.lim_hi + kAttnBlock - 1) / kAttnBlock : r.f0;
    chunk_blocks(r.f0, r.f1, p.splits, split, r.b0, r.b1);
    return r;
}

// Which of the block's 16 keys a row sees.
__device__ __forceinline__ uint32_t seen_keys(const AttnParams& p, const Row& r, const Span& sp, int j0)
{
    const uint32_t there = p.k_mask != nullptr ? p.k_mask[j0 / kAttnBlock] : 0xFFFFu;
    if (j0 >= sp.ks && j0 + kAttnBlock <= r.lim_lo) return there;
    const int a = max(0, sp.ks - j0), n = min(max(r.lim - j0, 0), kAttnBlock);
    return ((1u << n) - 1u) & ~((1u << a) - 1u) & there;
}

// CW columns (from CW g on) of a row's result: partial, or o.
template <int CW>
__device__ __forceinline__ void store_fwd(const AttnParams& p, const Row& r, int h, int split, int g, const float (&acc)[1][CW],
                                          double m, double l)
{
    if (!r.valid) return;
    if (p.splits > 1) {
        const int64_t at = ((int64_t)split * p.K + h) * p.RQ + r.row;
        p.part_m[at] = m;
        p.part_l[at] = l;
        if (l != 0.0) store_row(acc, 1.0f, p.part0 + at * p.Dp + g * CW, CW, true);
        return;
    }
    const int hh = h * p.G + (r.row - r.tok * p.G);
    const float inv = l == 0.0 ? 0.0f : (float)(1.0 / l);
    store_row(acc, inv, p.o + (int64_t)r.tok * p.ldo + (int64_t)hh * p.D + g * CW, p.D - g * CW, rows_aligned(p.o, p.ldo, p.D));
    if (p.lse != nullptr)
        p.lse[(int64_t)r.tok * (p.K * p.G) + hh] = l == 0.0 ? -__builtin_inff() : (float)((m + log2(l)) * 0.69314718055994530942);
}

// ------------------------------------------------------------------ workgroups
//
// A tile of 64 rows (or keys) belongs to NW = Dp / 16 waves, which all hold
// the same rows in their lanes. Per step of 16 NW keys, wave w computes the
// scores of 16 of them and their weights, the weights go through LDS to every
// wave, and wave w sums the products with columns 16 w .. 16 w + 15 over all
// the step's keys: D x 16 products for the scores and as many for the sums,
// whatever D is, with 16 sums per lane. (One wave per tile, the first form,
// needed 64 or 128 sums per lane: two waves per SIMD, and a short prompt's
// latency was that of one wave's whole tile. 16 x 512 tokens, 12 heads of 64:
// 1148 us against 529.) A workgroup holds TT tiles; its persistent waves take
// the next TT tiles from a counter, the longest first.

// Exchange of a step's weights: [key / 4][row][4] words of sign | exponent bits
// and row offset (disjoint bits; the floats themselves with the native
// multiplier). At M = 8, whose table leaves no room for that, exponent and
// mantissa index in 16 bits, and the signs of 8 keys in one byte.
template <int TAB>
__host__ __device__ constexpr int exchange_bytes(int NW)
{
    return TAB == AT_LDS8 ? NW * (16 * kAttnTile * 2 + kAttnTile * 2) : NW * 16 * kAttnTile * 4;
}
template <int TAB>
__host__ __device__ constexpr int tile_bytes(int NW, int CW)
{
    return exchange_bytes<TAB>(NW) + NW * (16 / CW) * kAttnTile * 8;        // + a double per row and wave
}

template <int TAB>
struct Exchange {
    unsigned char* buf;
    int NW, lane;

    __device__ __forceinline__ uint8_t* signs() const { return buf + NW * 16 * kAttnTile * 2; }

    // wave w's CW weights of this lane's row
    template <bool SIGNED, int CW>
    __device__ __forceinline__ void put(int w, const float (&x)[CW], int M) const
    {
        if constexpr (TAB == AT_LDS8) {
            uint32_t neg = 0u;
#pragma unroll
            for (int j = 0; j < CW; j += 4) {
                uint32_t h[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t b = __float_as_uint(x[j + i]);
                    h[i] = (b << 1) >> 16;
                    if (SIGNED) neg |= (b >> 31) << (j + i);
                }
                *reinterpret_cast<uint2*>(buf + (((w * CW + j) / 4) * kAttnTile + lane) * 8) = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
            }
            if (SIGNED)
#pragma unroll
                for (int j = 0; j < CW; j += 8) signs()[((w * CW + j) / 8) * kAttnTile + lane] = (uint8_t)(neg >> j);
        } else {
#pragma unroll
            for (int j = 0; j < CW; j += 4) {
                uint32_t v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t b = __float_as_uint(x[j + i]);
                    const uint32_t o = b << 1 == 0u ? (2u << M) : (b >> (22 - M)) & ((2u << M) - 2u);
                    v[i] = TAB == AT_NATIVE ? b : (b & 0xFF800000u) | o;
                }
                *reinterpret_cast<uint4*>(buf + (((w * CW + j) / 4) * kAttnTile + lane) * 16) = make_uint4(v[0], v[1], v[2], v[3]);
            }
        }
    }

    // keys 4 q .. 4 q + 3 of the step as lane operands
    template <bool SIGNED>
    __device__ __forceinline__ void get(int q, uint32_t (&wa)[4], uint32_t (&sa)[4], uint32_t base) const
    {
        if constexpr (TAB == AT_LDS8) {
            const uint2 v = *reinterpret_cast<const uint2*>(buf + (q * kAttnTile + lane) * 8);
            const uint32_t neg = SIGNED ? (uint32_t)signs()[(q >> 1) * kAttnTile + lane] >> ((q & 1) * 4) : 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t d = i < 2 ? v.x : v.y;
                const uint32_t h = i & 1 ? d >> 16 : d & 0xFFFFu;
                wa[i] = base + (h == 0u ? 512u : (h << 1) & 0x1FEu);
                sa[i] = (h << 15) & 0x7F800000u;
                if (SIGNED) sa[i] |= (neg >> i) << 31;
            }
        } else {
            const uint4 v = *reinterpret_cast<const uint4*>(buf + (q * kAttnTile + lane) * 16);
            const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                wa[i] = (x[i] & 0x7FFFFFu) + base;
                sa[i] = TAB == AT_NATIVE ? x[i] : x[i] & 0xFF800000u;
            }
        }
    }
};

// acc[0][c] += sum over the step's first 16 nb rows j of T(weight j, row j's
// column c): `row` points at this wave's columns of their Words [16 nb][16].
template <int TAB, bool SIGNED, int CW>
__device__ __forceinline__ void weigh(const Exchange<TAB>& ex, int nb, const Word* row, float (&acc)[1][CW], const Table& lut)
{
    if (nb <= 0) return;
    uint32_t wa[4], sa[4], q[2][2][CW / 2];
    auto load = [&](int j, int b) {
        load_columns(row + j * 16, q[b][0]);
        load_columns(row + (j + 1) * 16, q[b][1]);
    };
    const int n = nb * 4;
    load(0, 0);
    ex.template get<SIGNED>(0, wa, sa, lut.lds);
#pragma unroll 1
    for (int k = 0; k < n; ++k) {
        uint32_t wn[4], sn[4];
        load(4 * k + 2, 1);
        {
            const uint32_t w2[2] = {wa[0], wa[1]}, s2[2] = {sa[0], sa[1]};
            fold<TAB, 2, 1, CW, CW / 2>(w2, s2, q[0], acc, lut);
        }
        const int next = min(k + 1, n - 1);
        load(4 * next, 0);
        ex.template get<SIGNED>(next, wn, sn, lut.lds);
        {
            const uint32_t w2[2] = {wa[2], wa[3]}, s2[2] = {sa[2], sa[3]};
            fold<TAB, 2, 1, CW, CW / 2>(w2, s2, q[1], acc, lut);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            wa[i] = wn[i];
            sa[i] = sn[i];
        }
    }
}

// This wave's place in its workgroup: wave w of tile tt takes CW keys of a
// step and CW columns: block w CW / 16 of the step's 16-key blocks (and column
// group), from position `off` in it.
template <int TAB, int CW>
struct Place {
    int w, tt, waves, blk, off;
    Exchange<TAB> ex;
    double* each;              // [waves][64]: a value per row and wave of the tile
    Table lut;

    __device__ __forceinline__ Place(const AttnParams& p, unsigned char* lds)
    {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);    // in scalar registers
        waves = p.NW * (16 / CW);
        tt = wave / waves;
        w = wave - tt * waves;
        blk = w * CW / 16;
        off = w * CW % 16;
        unsigned char* at = lds + table_lds<TAB>() + 64 + tt * tile_bytes<TAB>(p.NW, CW);
        ex = Exchange<TAB>{at, p.NW, (int)(threadIdx.x & 63)};
        each = reinterpret_cast<double*>(at + exchange_bytes<TAB>(p.NW));
        lut = stage_table<TAB>(p.lut, p.M, lds);
    }
    // which of this wave's keys (rows) of a block count
    __device__ __forceinline__ uint32_t part(uint32_t seen) const { return (seen >> off) & ((1u << CW) - 1u); }
};

// The workgroup's next TT tiles: an item number from the counter, through LDS.
__device__ __forceinline__ int next_item(int* counter, int* shared)
{
    __syncthreads();                                   // everyone is done with the last item's LDS
    if (threadIdx.x == 0) *shared = atomicAdd(counter, 1);
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(*shared);
}

// The largest number of steps among the workgroup's tiles (shared[tt + 1]).
__device__ __forceinline__ int most_steps(int steps, int tt, int TT, int* shared)
{
    if (TT == 1) return steps;
    if ((threadIdx.x & 63) == 0) shared[1 + tt] = steps;
    __syncthreads();
    int n = 0;
    for (int i = 0; i < TT; ++i) n = max(n, shared[1 + i]);
    return __builtin_amdgcn_readfirstlane(n);
}

// ------------------------------------------------------------------ forward

template <int TAB, int CW>
__device__ __forceinline__ void fwd_tile(const AttnParams& p, const Place<TAB, CW>& at, const Row& r, const Span& sp, bool live, int h,
                                         int split, int steps)
{
    const int lane = threadIdx.x & 63, NW = p.NW;
    const Word* ql = p.q_lane + (int64_t)h * p.D4 * p.RQp + (int64_t)r.row * 4;
    const Word* kt = p.k_tr + (int64_t)h * p.TKp * p.D4 + at.off;
    const Word* vr = p.v_row + ((int64_t)h * NW + at.blk) * p.TKp * 16 + at.off;
    float* tops = reinterpret_cast<float*>(at.each);
    float acc[1][CW];
#pragma unroll
    for (int c = 0; c < CW; ++c) acc[0][c] = 0.0f;
    double m = -__builtin_inf(), l = 0.0;
#pragma unroll 1
    for (int it = 0; it < steps; ++it) {
        const int kb0 = r.b0 + it * NW, kb = kb0 + at.blk;
        const bool mine = live && kb < r.b1;
        float s[1][CW];
        uint32_t seen = 0u;
        float top = -__builtin_inff();
        if (mine) {
            dot_block<TAB, CW>(ql, p.RQp, kt + (int64_t)kb * kAttnBlock * p.D4, p.D4, s, at.lut);
            seen = at.part(seen_keys(p, r, sp, kb * kAttnBlock));
#pragma unroll
            for (int c = 0; c < CW; ++c) top = fmaxf(top, (seen >> c) & 1u ? s[0][c] : -__builtin_inff());
        }
        tops[at.w * kAttnTile + lane] = top;
        __syncthreads();
        for (int x = 0; x < at.waves; ++x) top = fmaxf(top, tops[x * kAttnTile + lane]);
        const double mn = fmax(m, __builtin_ceil((double)top * p.c));
        if (__any(mn > m)) {                 // a power of two: no mantissa changes
            const int d = mn > m ? (int)fmax(m - mn, -4096.0) : 0;
            l = __builtin_ldexp(l, d);
#pragma unroll
            for (int c = 0; c < CW; ++c) acc[0][c] = __builtin_ldexpf(acc[0][c], d);
            m = mn;
        }
        if (mine) {
            each_value(s[0], [&](float v, int c) {
                const float e = exp2_once(__builtin_fma((double)v, p.c, -m));
                const float x = (seen >> c) & 1u ? e : 0.0f;
                l += (double)x;
                return x;
            });
            at.ex.template put<false>(at.w, s[0], p.M);
        }
        __syncthreads();
        if (live) weigh<TAB, false>(at.ex, min(NW, r.b1 - kb0), vr + (int64_t)kb0 * kAttnBlock * 16, acc, at.lut);
    }
    at.each[at.w * kAttnTile + lane] = l;
    __syncthreads();
    l = 0.0;
    for (int x = 0; x < at.waves; ++x) l += at.each[x * kAttnTile + lane];
    if (live) store_fwd(p, r, h, split, at.w, acc, m, l);
}

// The checked path, kept small rather than fast: every wave computes all the
// scores for its own 16 columns. A weight's product may leave the format's
// range here, and whether it does must not depend on the order of the keys:
// the row's maximum over all its keys comes first.
template <int TAB>
__device__ __forceinline__ void fwd_tile_checked(const AttnParams& p, const Row& r, const Span& sp, int h, int split, int g,
                                                 const Table& lut)
{
    const uint32_t quad = threadIdx.x & 3u;
    const Word* ql = p.q_lane + (int64_t)h * p.D4 * p.RQp + (int64_t)r.row * 4;
    const Word* kt = p.k_tr + (int64_t)h * p.TKp * p.D4;
    const Word* vr = p.v_row + ((int64_t)h * p.NW + g) * p.TKp * CPW;
    float top = -__builtin_inff();
    bool bad = false;                        // a seen score is NaN or +Inf
#pragma unroll 1
    for (int kb = r.f0; kb < r.f1; ++kb) {
        float s[CPW];
        dot_block_checked<TAB>(ql, p.RQp, kt + (int64_t)kb * kAttnBlock * p.D4, p.D4, quad, s, lut, p.elo, p.ehi);
        const uint32_t seen = seen_keys(p, r, sp, kb * kAttnBlock);
#pragma unroll
        for (int c = 0; c < CPW; ++c) {
            const float v = (seen >> c) & 1u ? s[c] : -__builtin_inff();
            bad = bad || !(v < __builtin_inff());
            top = fmaxf(top, v);
        }
    }
    const double m = __builtin_ceil((double)top * p.c);
    float acc[1][CPW];
#pragma unroll
    for (int c = 0; c < CPW; ++c) acc[0][c] = 0.0f;
    double l = 0.0;
#pragma unroll 1
    for (int kb = r.b0; kb < r.b1; ++kb) {
        float s[CPW];
        dot_block_checked<TAB>(ql, p.RQp, kt + (int64_t)kb * kAttnBlock * p.D4, p.D4, quad, s, lut, p.elo, p.ehi);
        const uint32_t seen = seen_keys(p, r, sp, kb * kAttnBlock);
#pragma unroll
        for (int c = 0; c < CPW; ++c) {
            const float e = exp2_once(__builtin_fma((double)s[c], p.c, -m));
            s[c] = ((seen >> c) & 1u) && !bad ? e : 0.0f;
            l += (double)s[c];
        }
        weigh_block_checked<TAB>(s, seen, vr + (int64_t)kb * kAttnBlock * CPW, quad, acc[0], lut, p.M, p.elo, p.ehi);
    }
    if (bad) l = __builtin_nan("");
    store_fwd(p, r, h, split, g, acc, m, l);
}

// CW, the keys and columns of a wave: 16, or 8 for calls that leave the GPU
// mostly empty (a lone wave issues one instruction in five or more clocks, so
// twice the waves of half the work end sooner; five prompts of up to 48 tokens: 36 instead of
// 51 us).
// Waves of a workgroup: up to 8; 12 at M = 8, where one workgroup fills a CU's
// LDS; up to 16 with CW = 8 (two per 16 columns).
template <int TAB, int CW>
__host__ __device__ constexpr int max_waves() { return CW == 8 ? 16 : TAB == AT_LDS8 ? 12 : 8; }
template <int TAB, int CW>
__host__ __device__ constexpr int min_waves() { return CW == 16 && TAB == AT_LDS8 ? 3 : 4; }

// Items: TT consecutive tiles (in find_tile's order: those that end their
// sequences, with a causal mask the longest, first) of one kv head and chunk.
template <int TAB, int CW>
__global__ __launch_bounds__((64 * max_waves<TAB, CW>()), (min_waves<TAB, CW>())) void attn_fwd_kernel(AttnParams p)
{
    extern __shared__ __align__(16) unsigned char lds[];
    int* shared = reinterpret_cast<int*>(lds + table_lds<TAB>());
    const Place<TAB, CW> at(p, lds);
    int ql, qh, kl, kh, vl, vh;
    tensor_range(p.stats, 0, ql, qh);
    tensor_range(p.stats, 1, kl, kh);
    tensor_range(p.stats, 2, vl, vh);
    const bool fast = !p.force_checked && p.elo == 1 && range_fast<TAB>(ql, qh) && range_fast<TAB>(kl, kh) &&
                      range_fast<TAB>(vl, vh) && qh + kh <= p.smax;
    const int heads = p.K * p.splits;
    for (;;) {
        const int item = next_item(p.next, shared);
        if (item >= p.items) break;
        const int gt = item / heads, hs = item % heads;
        const int h = hs % p.K, split = hs / p.K;
        const Span sp = find_tile(p.cu_q, p.total_q, p.cu_k, p.total_k, p.nseq, false, p.G, kAttnTile, gt * p.TT + at.tt,
                                  p.k_len, p.k_stride, p.k_most);
        const bool live = sp.tile >= 0;
        const Row r = tile_row(p, sp, split);
        if (!fast) {
            if (live && at.w < p.NW) fwd_tile_checked<TAB>(p, r, sp, h, split, at.w, at.lut);
            continue;
        }
        const int steps = most_steps(live ? (r.b1 - r.b0 + p.NW - 1) / p.NW : 0, at.tt, p.TT, shared);
        fwd_tile<TAB, CW>(p, at, r, sp, live, h, split, steps);
    }
}

// Joins the chunks of every row, L lanes per row: the lanes first hold the
// chunks' maxima and sums, then the columns. L = 64 for more than 16 chunks
// (43 chunks of 512 rows: 178 -> 36 us), else 16 (2 chunks of 98,304 rows: 34
// against 62 us).
template <int L>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnJoinParams p)
{
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) / L;   // kv head * RQ + row
    const int64_t rows = (int64_t)p.K * p.RQ;
    if (at >= rows) return;
    const int lane = threadIdx.x % L;
    const int h = (int)(at / p.RQ), row = (int)(at - (int64_t)h * p.RQ);
    const int tok = row / p.G;
    // rows of no sequence keep what they hold
    int end = 0;
    for (int b = lane; b <= p.nseq; b += L) end = max(end, min(max(p.cu_q[b], 0), p.total_q));
    for (int off = L / 2; off > 0; off >>= 1) end = max(end, __shfl_xor(end, off, L));
    if (tok >= end || tok < max(0, p.cu_q[0])) return;
    double m = -__builtin_inf();
    for (int s = lane; s < p.splits; s += L)
        if (p.part_l[s * rows + at] != 0.0) m = fmax(m, p.part_m[s * rows + at]);
    for (int off = L / 2; off > 0; off >>= 1) m = fmax(m, __shfl_xor(m, off, L));
    double l = 0.0;
    constexpr int N = kAttnMaxDim / L;
    float a[N];
#pragma unroll
    for (int i = 0; i < N; ++i) a[i] = 0.0f;
    for (int s0 = 0; s0 < p.splits; s0 += L) {
        // this lane's chunk: its power of two, or none of it (an empty chunk)
        const int s = s0 + lane;
        const double ls = s < p.splits ? p.part_l[s * rows + at] : 0.0;
        const int shift = ls != 0.0 ? (int)fmax(p.part_m[s * rows + at] - m, -4096.0) : 1;
        double t = ls != 0.0 ? __builtin_ldexp(ls, shift) : 0.0;
        for (int off = L / 2; off > 0; off >>= 1) t += __shfl_xor(t, off, L);
        l += t;
        const int n = min(L, p.splits - s0);
#pragma unroll 4
        for (int j = 0; j < n; ++j) {
            const int d = __shfl(shift, j, L);
            const float* part = p.part + ((s0 + j) * rows + at) * p.Dp;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = lane + L * i;
                const float v = c < p.Dp && d <= 0 ? part[c] : 0.0f;
                a[i] += __builtin_ldexpf(v, d);
            }
        }
    }
    const int hh = h * p.G + (row - tok * p.G);
    const float inv = l == 0.0 ? 0.0f : (float)(1.0 / l);
    float* o = p.o + (int64_t)tok * p.ldo + (int64_t)hh * p.D;
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (lane + L * i < p.D) o[lane + L * i] = a[i] * inv;
    if (p.lse != nullptr && lane == 0)
        p.lse[(int64_t)tok * (p.K * p.G) + hh] = l == 0.0 ? -__builtin_inff() : (float)((m + log2(l)) * 0.69314718055994530942);
}

// ------------------------------------------------------------------ backward

// P = RN32(2^x) and dS = RN32(P (dP - D)), magnitudes below 2^-64 zero.
template <bool CHK>
__device__ __forceinline__ void score_gradient(double x, float lse, float dp, float delta, float& pr, float& ds)
{
    pr = exp2_once(x);
    if (CHK) pr = lse == -__builtin_inff() ? 0.0f : x != x ? __builtin_nanf("") : pr;
    ds = (float)((double)pr * ((double)dp - (double)delta));
    ds = !(__builtin_fabsf(ds) < 0x1p-64f) ? ds : 0.0f;
}

// One row's state of the backward pass.
struct RowState {
    float lse, delta;
    double base;
};
__device__ __forceinline__ RowState row_state(const AttnParams& p, const Row& r, int h)
{
    RowState b;
    b.lse = p.rowlse[(int64_t)h * p.RQp + r.row];
    b.delta = p.delta[(int64_t)h * p.RQp + r.row];
    b.base = (double)b.lse * 1.4426950408889634074;
    return b;
}

template <int CW>
__device__ __forceinline__ void store_dq(const AttnParams& p, const Row& r, int h, int split, int g, const float (&acc)[1][CW])
{
    if (!r.valid) return;
    if (p.splits > 1) {
        store_row(acc, 1.0f, p.part0 + (((int64_t)split * p.K + h) * p.RQ + r.row) * p.Dp + g * CW, CW, true);
    } else {
        float* o = p.dq + (int64_t)r.tok * p.lddq + (int64_t)(h * p.G + (r.row - r.tok * p.G)) * p.D;
        store_row(acc, p.scale, o + g * CW, p.D - g * CW, rows_aligned(p.dq, p.lddq, p.D));
    }
}

// dQ of 64 rows: each wave the scores and dP of CW keys of a step and their
// dS, then CW columns of the sum over the step's keys.
template <int TAB, int CW>
__device__ __forceinline__ void dq_tile(const AttnParams& p, const Place<TAB, CW>& at, const Row& r, const Span& sp, bool live, int h,
                                        int split, int steps)
{
    const int NW = p.NW;
    const int64_t lane_at = (int64_t)h * p.D4 * p.RQp + (int64_t)r.row * 4, tr_at = (int64_t)h * p.TKp * p.D4 + at.off;
    const Word* kr = p.k_row + ((int64_t)h * NW + at.blk) * p.TKp * 16 + at.off;
    RowState b{0.0f, 0.0f, 0.0};
    if (live) b = row_state(p, r, h);
    float acc[1][CW];
#pragma unroll
    for (int c = 0; c < CW; ++c) acc[0][c] = 0.0f;
#pragma unroll 1
    for (int it = 0; it < steps; ++it) {
        const int kb0 = r.b0 + it * NW, kb = kb0 + at.blk;
        float s[1][CW];
        const bool mine = live && kb < r.b1;
        if (mine) {
            float dp[1][CW];
            const int64_t tr = tr_at + (int64_t)kb * kAttnBlock * p.D4;
            dot_block<TAB, CW>(p.q_lane + lane_at, p.RQp, p.k_tr + tr, p.D4, s, at.lut);
            dot_block<TAB, CW>(p.do_lane + lane_at, p.RQp, p.v_tr + tr, p.D4, dp, at.lut);
            const uint32_t seen = at.part(seen_keys(p, r, sp, kb * kAttnBlock));
            each_value(s[0], [&](float v, int c) {
                float pr, ds;
                score_gradient<false>(__builtin_fma((double)v, p.c, -b.base), b.lse, dp[0][0], b.delta, pr, ds);
#pragma unroll
                for (int i = 0; i < CW - 1; ++i) dp[0][i] = dp[0][i + 1];
                return (seen >> c) & 1u ? ds : 0.0f;
            });
        }
        __syncthreads();                     // the last step's weights have been read
        if (mine) at.ex.template put<true>(at.w, s[0], p.M);
        __syncthreads();
        if (live) weigh<TAB, true>(at.ex, min(NW, r.b1 - kb0), kr + (int64_t)kb0 * kAttnBlock * 16, acc, at.lut);
    }
    if (live) store_dq(p, r, h, split, at.w, acc);
}

template <int TAB>
__device__ __forceinline__ void dq_tile_checked(const AttnParams& p, const Row& r, const Span& sp, int h, int split, int g,
                                                const Table& lut)
{
    const uint32_t quad = threadIdx.x & 3u;
    const int64_t lane_at = (int64_t)h * p.D4 * p.RQp + (int64_t)r.row * 4, tr_at = (int64_t)h * p.TKp * p.D4;
    const Word* kr = p.k_row + ((int64_t)h * p.NW + g) * p.TKp * CPW;
    const RowState b = row_state(p, r, h);
    float acc[1][CPW];
#pragma unroll
    for (int c = 0; c < CPW; ++c) acc[0][c] = 0.0f;
#pragma unroll 1
    for (int kb = r.b0; kb < r.b1; ++kb) {
        float s[CPW], dp[CPW];
        const int64_t tr = tr_at + (int64_t)kb * kAttnBlock * p.D4;
        dot_block_checked<TAB>(p.q_lane + lane_at, p.RQp, p.k_tr + tr, p.D4, quad, s, lut, p.elo, p.ehi);
        dot_block_checked<TAB>(p.do_lane + lane_at, p.RQp, p.v_tr + tr, p.D4, quad, dp, lut, p.elo, p.ehi);
        const uint32_t seen = seen_keys(p, r, sp, kb * kAttnBlock);
#pragma unroll
        for (int c = 0; c < CPW; ++c) {
            float pr, ds;
            score_gradient<true>(__builtin_fma((double)s[c], p.c, -b.base), b.lse, dp[c], b.delta, pr, ds);
            s[c] = (seen >> c) & 1u ? ds : 0.0f;
        }
        weigh_block_checked<TAB>(s, seen, kr + (int64_t)kb * kAttnBlock * CPW, quad, acc[0], lut, p.M, p.elo, p.ehi);
    }
    store_dq(p, r, h, split, g, acc);
}

// dK and dV of 64 keys, 16 rows per wave of a step as uniform operands (which
// the products take first: the image with the uniform operand first).
struct Key {
    int key, key_hi, shift, r_lo, r_hi, b0, b1;      // row r sees keys below r / G + shift
    bool valid;
};
__device__ __forceinline__ Key tile_key(const AttnParams& p, const Span& sp, int split)
{
    Key k;
    const int ke = sp.ks + sp.kn, lo = sp.ks + sp.tile * kAttnTile, raw = lo + (int)(threadIdx.x & 63);
    k.valid = raw < ke;
    k.key = min(raw, ke - 1);
    k.key_hi = min(lo + kAttnTile, ke) - 1;
    k.shift = sp.ks + sp.kn - sp.qn - sp.qs + 1;
    const int first = p.causal ? min(sp.qs + sp.qn, max(sp.qs, lo + 1 - k.shift)) : sp.qs;
    k.r_lo = first * p.G;
    k.r_hi = (sp.qs + sp.qn) * p.G;
    chunk_blocks(k.r_lo / kAttnBlock, k.r_hi > k.r_lo ? (k.r_hi + kAttnBlock - 1) / kAttnBlock : k.r_lo / kAttnBlock, p.splits,
                 split, k.b0, k.b1);
    return k;
}

// Which of the block's 16 rows see this lane's key.
__device__ __forceinline__ uint32_t seeing_rows(const AttnParams& p, const Span& sp, const Key& k, int r0)
{
    if (r0 >= k.r_lo && r0 + kAttnBlock <= k.r_hi && (!p.causal || k.key_hi < r0 / p.G + k.shift)) return 0xFFFFu;
    uint32_t seen = 0u;
#pragma unroll
    for (int c = 0; c < kAttnBlock; ++c) {
        const int r = r0 + c;
        const bool in = r >= sp.qs * p.G && r < k.r_hi && (!p.causal || k.key < r / p.G + k.shift);
        seen |= in ? 1u << c : 0u;
    }
    return seen;
}

template <int CW>
__device__ __forceinline__ void store_key(const AttnParams& p, const Key& k, int h, int split, int g, const float (&acc)[1][CW],
                                          float* part, float* out, int64_t ld, float scale)
{
    if (!k.valid) return;
    if (p.splits > 1) store_row(acc, 1.0f, part + (((int64_t)split * p.K + h) * p.total_k + k.key) * p.Dp + g * CW, CW, true);
    else store_row(acc, scale, out + (int64_t)k.key * ld + (int64_t)h * p.D + g * CW, p.D - g * CW, rows_aligned(out, ld, p.D));
}

template <int TAB, int CW>
__device__ __forceinline__ void dkv_tile(const AttnParams& p, const Place<TAB, CW>& at, const Key& k, const Span& sp, bool live, int h,
                                         int split, int steps)
{
    const int NW = p.NW;
    const int64_t lane_at = (int64_t)h * p.D4 * p.TKp + (int64_t)k.key * 4, tr_at = (int64_t)h * p.RQp * p.D4 + at.off;
    const int64_t row_at = ((int64_t)h * NW + at.blk) * p.RQp * 16 + at.off;
    float dv[1][CW], dk[1][CW];
#pragma unroll
    for (int c = 0; c < CW; ++c) dv[0][c] = dk[0][c] = 0.0f;
#pragma unroll 1
    for (int it = 0; it < steps; ++it) {
        const int rb0 = k.b0 + it * NW, rb = rb0 + at.blk;
        float s[1][CW], dp[1][CW];
        const bool mine = live && rb < k.b1;
        if (mine) {
            const int64_t tr = tr_at + (int64_t)rb * kAttnBlock * p.D4;
            dot_block<TAB, CW>(p.k_lane + lane_at, p.TKp, p.q_tr + tr, p.D4, s, at.lut);
            dot_block<TAB, CW>(p.v_lane + lane_at, p.TKp, p.do_tr + tr, p.D4, dp, at.lut);
            const uint32_t seen = at.part(seeing_rows(p, sp, k, rb * kAttnBlock));
            const float* lse_at = p.rowlse + (int64_t)h * p.RQp + rb * kAttnBlock + at.off;
            const float* delta_at = p.delta + (int64_t)h * p.RQp + rb * kAttnBlock + at.off;
            each_value(s[0], [&](float v, int c) {
                const float lse = lse_at[c];
                float pr, ds;
                score_gradient<false>(__builtin_fma((double)v, p.c, -((double)lse * 1.4426950408889634074)), lse, dp[0][0],
                                      delta_at[c], pr, ds);
                const bool in = (seen >> c) & 1u;
#pragma unroll
                for (int i = 0; i < CW - 1; ++i) dp[0][i] = dp[0][i + 1];
                dp[0][CW - 1] = in ? ds : 0.0f;
                return in ? pr : 0.0f;
            });
        }
        const int nb = min(NW, k.b1 - rb0);
        const int64_t first = row_at + (int64_t)rb0 * kAttnBlock * 16;
        __syncthreads();                     // the last step's weights have been read
        if (mine) at.ex.template put<false>(at.w, s[0], p.M);
        __syncthreads();
        if (live) weigh<TAB, false>(at.ex, nb, p.do_row + first, dv, at.lut);
        __syncthreads();
        if (mine) at.ex.template put<true>(at.w, dp[0], p.M);
        __syncthreads();
        if (live) weigh<TAB, true>(at.ex, nb, p.q_row + first, dk, at.lut);
    }
    if (!live) return;
    store_key(p, k, h, split, at.w, dv, p.part0, p.dv, p.lddv, 1.0f);
    store_key(p, k, h, split, at.w, dk, p.part1, p.dk, p.lddk, p.scale);
}

template <int TAB>
__device__ __forceinline__ void dkv_tile_checked(const AttnParams& p, const Key& k, const Span& sp, int h, int split, int g,
                                                 const Table& lut)
{
    const uint32_t quad = threadIdx.x & 3u;
    const int64_t lane_at = (int64_t)h * p.D4 * p.TKp + (int64_t)k.key * 4, tr_at = (int64_t)h * p.RQp * p.D4;
    const int64_t row_at = ((int64_t)h * p.NW + g) * p.RQp * CPW;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {             // dV, dK
        float acc[1][CPW];
#pragma unroll
        for (int c = 0; c < CPW; ++c) acc[0][c] = 0.0f;
#pragma unroll 1
        for (int rb = k.b0; rb < k.b1; ++rb) {
            float s[CPW], dp[CPW];
            const int64_t tr = tr_at + (int64_t)rb * kAttnBlock * p.D4;
            dot_block_checked<TAB>(p.k_lane + lane_at, p.TKp, p.q_tr + tr, p.D4, quad, s, lut, p.elo, p.ehi);
            dot_block_checked<TAB>(p.v_lane + lane_at, p.TKp, p.do_tr + tr, p.D4, quad, dp, lut, p.elo, p.ehi);
            const uint32_t seen = seeing_rows(p, sp, k, rb * kAttnBlock);
            const float* lse_at = p.rowlse + (int64_t)h * p.RQp + rb * kAttnBlock;
            const float* delta_at = p.delta + (int64_t)h * p.RQp + rb * kAttnBlock;
#pragma unroll
            for (int c = 0; c < CPW; ++c) {
                const float lse = lse_at[c];
                float pr, ds;
                score_gradient<true>(__builtin_fma((double)s[c], p.c, -((double)lse * 1.4426950408889634074)), lse, dp[c],
                                     delta_at[c], pr, ds);
                s[c] = (seen >> c) & 1u ? (pass ? ds : pr) : 0.0f;
            }
            weigh_block_checked<TAB>(s, seen, (pass ? p.q_row : p.do_row) + row_at + (int64_t)rb * kAttnBlock * CPW, quad, acc[0],
                                     lut, p.M, p.elo, p.ehi);
        }
        if (pass) store_key(p, k, h, split, g, acc, p.part1, p.dk, p.lddk, p.scale);
        else store_key(p, k, h, split, g, acc, p.part0, p.dv, p.lddv, 1.0f);
    }
}

// KEYS: dK and dV (tiles of keys), else dQ (tiles of rows). Waves of 8 columns
// (run_bwd), whose sums fit the 128 registers of four waves per SIMD; with 16
// columns these spill, and three waves per SIMD are left (8 ragged sequences
// up to 512, 12/4 heads of 64: dQ 301 us, dK and dV 373; with 8 columns 254
// and 338). The forward pass has half the sums and loses by either change (16
// x 512 tokens, 12 heads of 64: 529 -> 560 us with 8 columns; 8 heads of 128,
// 661 -> 850 us with three waves).
template <int TAB, bool KEYS, int CW>
__global__ __launch_bounds__((64 * max_waves<TAB, CW>()), (CW == 16 ? 3 : 4)) void attn_bwd_kernel(AttnParams p)
{
    extern __shared__ __align__(16) unsigned char lds[];
    int* shared = reinterpret_cast<int*>(lds + table_lds<TAB>());
    const Place<TAB, CW> at(p, lds);
    bool fast = !p.force_checked && p.elo == 1;
    int lo[4], hi[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        tensor_range(p.stats, t, lo[t], hi[t]);
        fast = fast && range_fast<TAB>(lo[t], hi[t]);
    }
    fast = fast && hi[0] + hi[2] <= p.smax;
    const int heads = p.K * p.splits;
    for (;;) {
        const int item = next_item(p.next, shared);
        if (item >= p.items) break;
        const int gt = item / heads, hs = item % heads;
        const int h = hs % p.K, split = hs / p.K;
        const Span sp = find_tile(p.cu_q, p.total_q, p.cu_k, p.total_k, p.nseq, KEYS, KEYS ? 1 : p.G, kAttnTile, gt * p.TT + at.tt);
        const bool live = sp.tile >= 0;
        if constexpr (KEYS) {
            const Key k = tile_key(p, sp, split);
            if (!fast) {
                if (live && at.w < p.NW) dkv_tile_checked<TAB>(p, k, sp, h, split, at.w, at.lut);
                continue;
            }
            const int steps = most_steps(live ? (k.b1 - k.b0 + p.NW - 1) / p.NW : 0, at.tt, p.TT, shared);
            dkv_tile<TAB, CW>(p, at, k, sp, live, h, split, steps);
        } else {
            const Row r = tile_row(p, sp, split);
            if (!fast) {
                if (live && at.w < p.NW) dq_tile_checked<TAB>(p, r, sp, h, split, at.w, at.lut);
                continue;
            }
            const int steps = most_steps(live ? (r.b1 - r.b0 + p.NW - 1) / p.NW : 0, at.tt, p.TT, shared);
            dq_tile<TAB, CW>(p, at, r, sp, live, h, split, steps);
        }
    }
}

// out = scale * (sum of the chunks' partials, ascending): 16 lanes per row of
// `rows` per kv head, G rows per token.
struct SumParams {
    const int* cu;
    const float* part;
    float* out;
    int64_t ld;
    int nseq, total, K, G, D, Dp, splits;
    float scale;
};
__global__ __launch_bounds__(256) void attn_sum_kernel(SumParams p)
{
    const int R = p.total * p.G;
    const int64_t at = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4), rows = (int64_t)p.K * R;
    if (at >= rows) return;
    const int h = (int)(at / R), row = (int)(at - (int64_t)h * R), tok = row / p.G;
    int end = 0;
    for (int b = threadIdx.x & 15; b <= p.nseq; b += 16) end = max(end, min(max(p.cu[b], 0), p.total));
    for (int off = 8; off > 0; off >>= 1) end = max(end, __shfl_xor(end, off, 64));
    if (tok >= end || tok < max(0, p.cu[0])) return;
    float* o = p.out + (int64_t)tok * p.ld + (int64_t)(h * p.G + (row - tok * p.G)) * p.D;
    for (int d = threadIdx.x & 15; d < p.D; d += 16) {
        float a = 0.0f;
#pragma unroll 4
        for (int s = 0; s < p.splits; ++s) a += p.part[(s * rows + at) * p.Dp + d];
        o[d] = a * p.scale;
    }
}

// ------------------------------------------------------------------ launchers

hipError_t launch_attn_decode(const AttnDecodeParams& p, hipStream_t s)
{
    attn_decode_kernel<<<dim3(kAttnSlots, p.count), kDecodeThreads, kAttnTile * (p.Dp + 1) * sizeof(uint32_t), s>>>(p);
    return hipGetLastError();
}

hipError_t launch_join(const AttnJoinParams& p, hipStream_t s)
{
    const int64_t rows = (int64_t)p.K * p.RQ;
    if (p.splits > 16) attn_join_kernel<64><<<(unsigned)((rows + 3) / 4), 256, 0, s>>>(p);
    else attn_join_kernel<16><<<(unsigned)((rows + 15) / 16), 256, 0, s>>>(p);
    return hipGetLastError();
}

// Tiles per workgroup: as many as fit its waves and, at M = 8, the LDS.
template <int TAB, int CW>
static int tiles_per_group(int NW)
{
    int n = std::max(1, max_waves<TAB, CW>() / (NW * (16 / CW)));
    if (CW == 8) n = 1;                      // few tiles, or many sums: a workgroup each
    while (n > 1 && table_lds<TAB>() + 64 + n * tile_bytes<TAB>(NW, CW) > kLdsBytes) --n;
    return n;
}

template <int TAB, int CW, typename F>
static hipError_t run(AttnParams p, F* f, Resident& cache, hipStream_t s)
{
    p.TT = tiles_per_group<TAB, CW>(p.NW);
    p.items = (int64_t)((p.tiles + p.TT - 1) / p.TT) * p.K * p.splits;
    const int threads = 64 * p.NW * (16 / CW) * p.TT;
    const size_t lds = table_lds<TAB>() + 64 + (size_t)p.TT * tile_bytes<TAB>(p.NW, CW);
    const int slots = resident(cache, p.NW, reinterpret_cast<const void*>(f), threads, lds);
    if (slots < 1) return hipErrorInvalidValue;
    f<<<(unsigned)std::min<int64_t>(p.items, slots), threads, lds, s>>>(p);
    return hipGetLastError();
}

// Fewer waves of 16 columns than two per SIMD of the GPU's 256 CUs (five
// prompts of up to 48 tokens: 51 us with 16 columns, 36 with 8; 16 x 512
// tokens, 12 heads of 64: 529 and 560).
// APPROX_ATTENTION_COLUMNS=8 or 16 forces a side (for measurements and tests).
static bool few_waves(const AttnParams& p)
{
    const char* force = std::getenv("APPROX_ATTENTION_COLUMNS");
    if (force != nullptr && (force[0] == '8' || force[0] == '1')) return force[0] == '8';
    return (int64_t)p.tiles * p.K * p.splits * p.NW < 2048;
}

template <int TAB>
static hipError_t run_fwd(const AttnParams& p, hipStream_t s)
{
    static Resident narrow, wide;
    return few_waves(p) ? run<TAB, 8>(p, &attn_fwd_kernel<TAB, 8>, narrow, s) : run<TAB, 16>(p, &attn_fwd_kernel<TAB, 16>, wide, s);
}

hipError_t launch_attn_fwd(const AttnParams& p, hipStream_t s)
{
    hipError_t e;
    switch (attn_table_kind(p.M)) {
    case AT_LDS: e = run_fwd<AT_LDS>(p, s); break;
    case AT_LDS8: e = run_fwd<AT_LDS8>(p, s); break;
    case AT_GLOBAL: e = run_fwd<AT_GLOBAL>(p, s); break;
    default: e = run_fwd<AT_NATIVE>(p, s); break;
    }
    if (e != hipSuccess || p.splits == 1) return e;
    return launch_join(AttnJoinParams{p.cu_q, p.nseq, p.K, p.G, p.D, p.Dp, p.total_q, p.RQ, p.splits, p.part0, p.part_m,
                                      p.part_l, p.o, p.ldo, p.lse}, s);
}

// 8 columns per wave: 2 to 24% faster than 16 at M = 4 and 7 (D = 32 to 128,
// calls that fill the GPU and calls that do not), 1 to 11% at M = 10 (2% slower
// at D = 128). At M = 8 one workgroup's table fills a CU, so that a tile of 8
// columns with D up to 32 leaves it at 2 or 4 waves: 8 sequences up to 512, 12/4
// heads of 32: 770 us with 8 columns, 555 with 16 and more tiles.
template <int TAB>
static hipError_t run_bwd(const AttnParams& p, bool keys, hipStream_t s)
{
    static Resident cache[4];
    if constexpr (TAB == AT_LDS8) {
        if (p.NW <= 2 && !few_waves(p))
            return keys ? run<TAB, 16>(p, &attn_bwd_kernel<TAB, true, 16>, cache[2], s)
                        : run<TAB, 16>(p, &attn_bwd_kernel<TAB, false, 16>, cache[3], s);
    }
    return keys ? run<TAB, 8>(p, &attn_bwd_kernel<TAB, true, 8>, cache[0], s)
                : run<TAB, 8>(p, &attn_bwd_kernel<TAB, false, 8>, cache[1], s);
}

static hipError_t launch_sum(const AttnParams& p, bool keys, const float* part, float* out, int64_t ld, float scale, hipStream_t s)
{
    const SumParams q{keys ? p.cu_k : p.cu_q, part, out, ld, p.nseq, keys ? p.total_k : p.total_q, p.K, keys ? 1 : p.G,
                      p.D, p.Dp, p.splits, scale};
    const int64_t rows = (int64_t)q.K * q.total * q.G;
    attn_sum_kernel<<<(unsigned)((rows + 15) / 16), 256, 0, s>>>(q);
    return hipGetLastError();
}

hipError_t launch_attn_bwd(const AttnParams& p, bool keys, hipStream_t s)
{
    hipError_t e;
    switch (attn_table_kind(p.M)) {
    case AT_LDS: e = run_bwd<AT_LDS>(p, keys, s); break;
    case AT_LDS8: e = run_bwd<AT_LDS8>(p, keys, s); break;
    case AT_GLOBAL: e = run_bwd<AT_GLOBAL>(p, keys, s); break;
    default: e = run_bwd<AT_NATIVE>(p, keys, s); break;
    }
    if (e != hipSuccess || p.splits == 1) return e;
    if (!keys) return launch_sum(p, false, p.part0, p.dq, p.lddq, p.scale, s);
    e = launch_sum(p, true, p.part0, p.dv, p.lddv, 1.0f, s);
    return e != hipSuccess ? e : launch_sum(p, true, p.part1, p.dk, p.lddk, p.scale, s);
}

}  // namespace amx
