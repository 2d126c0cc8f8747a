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
// One wave owns 64 rows, one per lane, and takes 16 keys at a time. The keys
// (and then the values' columns) are uniform operands spread over the lanes
// of each quad (product.h); the scores of a block come out in the lanes that
// need them as the lane operand of P V, so they never leave the registers.
// What bounds the loops is the rate of table lookups (one 16-bit LDS read per
// product), as in the GEMM kernel.
#include <algorithm>
#include <atomic>

#include "attention.h"
#include "product.h"

namespace amx {

// ------------------------------------------------------------------ decode

// Word of one operand in the attention image's layout (decode_bits of the
// GEMM path with this image's column stride); folds its exponent into lo/hi.
__device__ __forceinline__ Word attn_word(uint32_t bits, int M, bool lane_role, int elo, int ehi, int& lo, int& hi)
{
    if (M == 0) {
        hi = max(hi, (int)((bits >> 23) & 0xFFu));
        return Word{0u, bits};
    }
    bits = cast_fmt(bits, elo, ehi);
    const uint32_t e = (bits >> 23) & 0xFFu, frac = bits & 0x7FFFFFu;
    const uint32_t idx = frac >> (23 - M);
    Word o;
    if (e == 0u || e == 255u) {
        o.se = e == 0u ? 0u : frac ? 0x7FC00000u : (bits & 0xFF800000u);
        o.w = lane_role ? (2u << M) : 0u;
        if (e == 255u) hi = 255;
    } else {
        o.se = bits & 0xFF800000u;
        o.w = lane_role ? idx * 2u : idx * (uint32_t)attn_col_bytes(M);
        lo = min(lo, (int)e);
        hi = max(hi, (int)e);
    }
    return o;
}

// Decodes 64 rows of one kv head per step through LDS into the panels asked
// for. Bound by HBM: 4 bytes read and 8 written per element and panel.
constexpr int kDecodeThreads = 256;
__global__ __launch_bounds__(kDecodeThreads) void attn_decode_kernel(AttnDecodeParams p)
{
    __shared__ uint32_t tile[kAttnTile * (kAttnMaxDim + 1)];
    __shared__ int range[2 * (kDecodeThreads / 64)];
    const AttnTensor& t = p.t[blockIdx.y];
    const int tid = threadIdx.x, S = p.Dp + 1;
    const int blocks = t.Rp / kAttnTile;
    const bool vec = ((t.ld | p.D) & 3) == 0 && (reinterpret_cast<uintptr_t>(t.src) & 15) == 0;
    int lo = 255, hi = 0;
    for (int64_t item = blockIdx.x; item < (int64_t)blocks * p.K; item += gridDim.x) {
        const int h = (int)(item / blocks), r0 = (int)(item - (int64_t)h * blocks) * kAttnTile;
        __syncthreads();
        if (vec) {
            const int per = p.Dp / 4;
            for (int i = tid; i < kAttnTile * per; i += kDecodeThreads) {
                const int rr = i / per, d = (i - rr * per) * 4, r = r0 + rr;
                uint4 x = make_uint4(0, 0, 0, 0);
                if (r < t.R && d < p.D) {
                    const int tok = r / t.G, hh = h * t.G + (r - tok * t.G);
                    x = *reinterpret_cast<const uint4*>(t.src + (int64_t)tok * t.ld + (int64_t)hh * p.D + d);
                }
                uint32_t* o = tile + rr * S + d;
                o[0] = x.x; o[1] = x.y; o[2] = x.z; o[3] = x.w;
            }
        } else {
            for (int i = tid; i < kAttnTile * p.Dp; i += kDecodeThreads) {
                const int rr = i / p.Dp, d = i - rr * p.Dp, r = r0 + rr;
                uint32_t x = 0;
                if (r < t.R && d < p.D) {
                    const int tok = r / t.G, hh = h * t.G + (r - tok * t.G);
                    x = __float_as_uint(t.src[(int64_t)tok * t.ld + (int64_t)hh * p.D + d]);
                }
                tile[rr * S + d] = x;
            }
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
            for (int i = tid; i < kAttnTile * p.D4 / 2; i += kDecodeThreads) {
                const int pair = i & 7, q = i >> 3, blk = q / p.D4, d = q - blk * p.D4;
                const int rr = blk * kAttnBlock + pair * 2;
                const Word a = attn_word(tile[rr * S + d], p.M, false, p.elo, p.ehi, lo, hi);
                const Word b = attn_word(tile[(rr + 1) * S + d], p.M, false, p.elo, p.ehi, lo, hi);
                *reinterpret_cast<uint4*>(dst + ((int64_t)blk * p.D4 + d) * kAttnBlock + pair * 2) =
                    make_uint4(a.w, a.se, b.w, b.se);
            }
        }
        if (t.row != nullptr) {
            Word* dst = t.row + ((int64_t)h * t.Rp + r0) * p.Dp;
            for (int i = tid; i < kAttnTile * p.Dp / 2; i += kDecodeThreads) {
                const int rr = i / (p.Dp / 2), d = (i - rr * (p.Dp / 2)) * 2;
                const Word a = attn_word(tile[rr * S + d], p.M, false, p.elo, p.ehi, lo, hi);
                const Word b = attn_word(tile[rr * S + d + 1], p.M, false, p.elo, p.ehi, lo, hi);
                *reinterpret_cast<uint4*>(dst + (int64_t)rr * p.Dp + d) = make_uint4(a.w, a.se, b.w, b.se);
            }
        }
        if (t.flat != nullptr) {
            Word* dst = t.flat + (int64_t)h * p.D4 * t.Fp;
            for (int i = tid; i < kAttnTile * p.D4; i += kDecodeThreads) {
                const int d = i / kAttnTile, rr = i & (kAttnTile - 1);
                dst[(int64_t)d * t.Fp + r0 + rr] = attn_word(tile[rr * S + d], p.M, false, p.elo, p.ehi, lo, hi);
            }
        }
        if (p.o != nullptr && blockIdx.y == 1) {
            // D_i = sum_d dO_id o_id, exact products summed in 64 bits, four
            // threads per row, rounded once
            const int rr = tid >> 2, r = r0 + rr;
            double sum = 0.0;
            if (r < t.R) {
                const int tok = r / t.G, hh = h * t.G + (r - tok * t.G);
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

// ------------------------------------------------------------------ ranges and sequences

// Exponent range of one decoded tensor over all its decode workgroups.
__device__ __forceinline__ void tensor_range(const uint32_t* stats, int t, int& lo, int& hi)
{
    lo = 255;
    hi = 0;
    for (int i = threadIdx.x & 63; i < kAttnSlots; i += 64) {
        const uint32_t v = stats[t * kAttnSlots + i];
        lo = min(lo, (int)(v & 0xFFu));
        hi = max(hi, (int)(v >> 8));
    }
    for (int off = 32; off > 0; off >>= 1) {
        lo = min(lo, __shfl_xor(lo, off, 64));
        hi = max(hi, __shfl_xor(hi, off, 64));
    }
    lo = __builtin_amdgcn_readfirstlane(lo);
    hi = __builtin_amdgcn_readfirstlane(hi);
}

// The fast path (no product leaves the normal range, and the lane operands'
// scaled significands stay normal): every operand's exponent within
// [kFastLo, kFastHi] (|x| in [2^-62, 2^41)), so products of two operands
// reach at least 2^-124 and products with a weight (at least 2^-64) at least
// 2^-126; the sum of q's and k's largest exponents bounded so that |c s| stays
// below 2^40 (its fraction is then still exact to 2^-12 ulp of a numerator).
// The native multiplier has no lower bound (its products may be subnormal).
constexpr int kFastLo = 65, kFastHi = 167;
template <int TAB>
__device__ __forceinline__ bool range_fast(int lo, int hi)
{
    return hi <= kFastHi && (TAB == AT_NATIVE || lo >= kFastLo);
}

// One sequence's rows and keys as absolute packed positions.
struct Span {
    int qs, qn, ks, kn;
    int seq;
    int tile;              // tile within the sequence; -1: no such tile
};

__device__ __forceinline__ uint32_t fdiv32(uint32_t n, const FastDiv& f) { return (__umulhi(n, f.m) + n) >> f.l; }

// Prefix maximum over the wave (lane i: the maximum of lanes 0..i).
__device__ __forceinline__ int wave_prefix_max(int v)
{
    const int lane = threadIdx.x & 63;
    for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(v, off, 64);
        if (lane >= off) v = max(v, o);
    }
    return v;
}

__device__ __forceinline__ int wave_prefix_sum(int v)
{
    const int lane = threadIdx.x & 63;
    for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(v, off, 64);
        if (lane >= off) v += o;
    }
    return v;
}

// Sequence and tile of tile number t when every sequence's `units` rows
// (queries: tokens * mult; keys: tokens) are cut into tiles of `size`.
// Offsets are clamped to the tensors and to their running maximum, so
// whatever they hold, sequences stay inside and do not overlap.
__device__ __forceinline__ Span find_tile(const int* cu_q, int total_q, const int* cu_k, int total_k, int nseq,
                                          bool by_key, int mult, int size, int t)
{
    const int lane = threadIdx.x & 63;
    int cq = 0, ck = 0, base = 0;
    Span sp;
    sp.tile = -1;
    sp.qs = sp.qn = sp.ks = sp.kn = sp.seq = 0;
    for (int b0 = 0; b0 < nseq; b0 += 64) {
        const int b = b0 + lane;
        const int bq = min(b, nseq), b1 = min(b + 1, nseq);
        const int qs = max(cq, wave_prefix_max(min(max(cu_q[bq], 0), total_q)));
        const int qe = max(qs, min(max(cu_q[b1], 0), total_q));
        const int ks = max(ck, wave_prefix_max(min(max(cu_k[bq], 0), total_k)));
        const int ke = max(ks, min(max(cu_k[b1], 0), total_k));
        const int n = by_key ? ke - ks : qe - qs;
        const int tiles = b < nseq ? (n * mult + size - 1) / size : 0;
        const int incl = base + wave_prefix_sum(tiles);
        const uint64_t found = __ballot(incl > t);
        if (found) {
            const int l = __builtin_ctzll(found);
            sp.seq = b0 + l;
            sp.qs = __shfl(qs, l, 64);
            sp.qn = __shfl(qe, l, 64) - sp.qs;
            sp.ks = __shfl(ks, l, 64);
            sp.kn = __shfl(ke, l, 64) - sp.ks;
            sp.tile = t - (__shfl(incl, l, 64) - __shfl(tiles, l, 64));
            break;
        }
        cq = __shfl(qe, 63, 64);
        ck = __shfl(ke, 63, 64);
        base = __shfl(incl, 63, 64);
    }
    sp.qs = __builtin_amdgcn_readfirstlane(sp.qs);
    sp.qn = __builtin_amdgcn_readfirstlane(sp.qn);
    sp.ks = __builtin_amdgcn_readfirstlane(sp.ks);
    sp.kn = __builtin_amdgcn_readfirstlane(sp.kn);
    sp.tile = __builtin_amdgcn_readfirstlane(sp.tile);
    return sp;
}

// ------------------------------------------------------------------ products

template <int TAB>
__device__ __forceinline__ uint32_t table_at(const unsigned char* lut, uint32_t off)
{
    if constexpr (TAB == AT_GLOBAL)
        return *reinterpret_cast<const uint16_t __attribute__((address_space(1)))*>(
            (const unsigned char __attribute__((address_space(1)))*)lut + off);
    else return *reinterpret_cast<const uint16_t*>(lut + off);
}

// Column c's w (h = 0) or se (h = 1) in every lane (col_word for any number of
// loaded columns).
template <int NQ>
__device__ __forceinline__ uint32_t uniform_word(const uint32_t (&q)[NQ], int c, int h)
{
    return quad_bcast(q[4 * (c >> 3) + 2 * (c & 1) + h], (c >> 1) & 3);
}

// Products of NI reduction steps with NC uniform columns each (NQ registers of
// each step's words): step i's lane operand (wa, sa) times the columns of
// q[i], folded into acc[i % GR], on the fast path. The lookups run kAhead
// products ahead of the folds (the LDS wait counter holds 15).
constexpr int kAhead = 12;
template <int TAB, int NI, int GR, int NC = CPW, int NQ = UQ>
__device__ __forceinline__ void fold(const uint32_t (&wa)[NI], const uint32_t (&sa)[NI], const uint32_t (&q)[NI][NQ],
                                     float (&acc)[GR][NC], const unsigned char* lut)
{
    if constexpr (TAB == AT_NATIVE) {
#pragma unroll
        for (int s = 0; s < NI * NC; ++s) {
            const int i = s / NC, c = s % NC;
            fmac_quad(acc[i % GR][c], q[i][4 * (c >> 3) + 2 * (c & 1) + 1], __uint_as_float(sa[i]), (c >> 1) & 3);
        }
    } else {
        uint32_t e[kAhead + 1];
#pragma unroll
        for (int s = 0; s < kAhead && s < NI * NC; ++s) e[s] = table_at<TAB>(lut, wa[s / NC] + uniform_word(q[s / NC], s % NC, 0));
#pragma unroll
        for (int s = 0; s < NI * NC; ++s) {
            const int n = s + kAhead, i = s / NC, c = s % NC;
            if (n < NI * NC) e[n % (kAhead + 1)] = table_at<TAB>(lut, wa[n / NC] + uniform_word(q[n / NC], n % NC, 0));
            fmac_quad(acc[i % GR][c], q[i][4 * (c >> 3) + 2 * (c & 1) + 1],
                      __uint_as_float((e[s % (kAhead + 1)] << 8) + sa[i]), (c >> 1) & 3);
            if ((s & 3) == 3) __builtin_amdgcn_sched_barrier(0);
        }
    }
}

// The same for one step on the checked path: Algorithm 2 with every special
// case, one product at a time; where `keep` is false (per lane) or bit c of
// `cols` is clear, the sum stays as it is.
template <int TAB, int NC, int NQ>
__device__ __forceinline__ void fold_checked(uint32_t wa, uint32_t sa, const uint32_t (&q)[NQ], float (&acc)[NC],
                                             const unsigned char* lut, int elo, int ehi, bool keep, uint32_t cols = 0xFFFFu)
{
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const uint32_t sb = uniform_word(q, c, 1);
        float v;
        if constexpr (TAB == AT_NATIVE) v = fmaf(__uint_as_float(sa), __uint_as_float(sb), acc[c]);
        else v = checked_product_acc(acc[c], table_at<TAB>(lut, wa + uniform_word(q, c, 0)), sa, sb, elo, ehi);
        acc[c] = keep && ((cols >> c) & 1u) ? v : acc[c];
        asm volatile("" : "+v"(acc[c]));
    }
}

// acc[c] = FP32 sums, ascending over d, of T(row d, column c's d): the lane
// panel's row at `lane` (Words at [D4 / 4][Rp][4]), 16 uniform columns at `tr`
// ([D4][16]). Two steps at a time, their words requested two steps ahead.
template <int TAB>
__device__ __forceinline__ void dot_block(const Word* lane, int64_t Rp, const Word* tr, int D4, uint32_t quad,
                                          float (&acc)[1][CPW], const unsigned char* lut)
{
    uint32_t wa[2][2], sa[2][2], q[2][2][UQ];
    auto load = [&](int s, int b) {
        const uint4 w = *reinterpret_cast<const uint4*>(lane + (int64_t)(s >> 1) * Rp * 4 + (s & 1) * 2);
        wa[b][0] = w.x; sa[b][0] = w.y; wa[b][1] = w.z; sa[b][1] = w.w;
        load_uniform(tr + s * 32, quad, q[b][0]);
        load_uniform(tr + s * 32 + 16, quad, q[b][1]);
    };
    const int steps = D4 / 2;                 // even
#pragma unroll
    for (int c = 0; c < CPW; ++c) acc[0][c] = 0.0f;
    load(0, 0);
#pragma unroll 1
    for (int s = 0; s < steps; s += 2) {
        load(s + 1, 1);
        fold<TAB, 2, 1>(wa[0], sa[0], q[0], acc, lut);
        load(min(s + 2, steps - 1), 0);
        fold<TAB, 2, 1>(wa[1], sa[1], q[1], acc, lut);
    }
}

template <int TAB>
__device__ __forceinline__ void dot_block_checked(const Word* lane, int64_t Rp, const Word* tr, int D4, uint32_t quad,
                                                  float (&acc)[CPW], const unsigned char* lut, int elo, int ehi)
{
#pragma unroll
    for (int c = 0; c < CPW; ++c) acc[c] = 0.0f;
#pragma unroll 1
    for (int d = 0; d < D4; ++d) {
        const uint2 w = *reinterpret_cast<const uint2*>(lane + (int64_t)(d >> 2) * Rp * 4 + (d & 3));
        uint32_t q[UQ];
        load_uniform(tr + d * CPW, quad, q);
        fold_checked<TAB>(w.x, w.y, q, acc, lut, elo, ehi, true);
    }
}

// Lane operand of a weight (a numerator, probability or score gradient).
template <int TAB>
__device__ __forceinline__ void weight_word(float x, int M, uint32_t& w, uint32_t& se)
{
    const uint32_t bits = __float_as_uint(x);
    if constexpr (TAB == AT_NATIVE) {
        w = 0u;
        se = bits;
    } else {
        w = bits << 1 == 0u ? (2u << M) : (bits >> (22 - M)) & ((2u << M) - 2u);
        se = bits & 0xFF800000u;
    }
}

// acc[g][c] += sum over the block's 16 rows j of T(x[j], row j's column):
// `row` points at the block's Words [16][16 DC]. A masked weight is zero and
// its lookup reads the pad. x is consumed (rotated in registers).
template <int TAB, int DC>
__device__ __forceinline__ void weigh_block(float (&x)[CPW], const Word* row, uint32_t quad, float (&acc)[DC][CPW],
                                            const unsigned char* lut, int M)
{
    static_assert(DC % 2 == 0, "two column groups per step");
    constexpr int H = DC / 2;                 // steps per row
    uint32_t q[2][2][UQ];
    auto load = [&](int s, int b) {
        load_uniform(row + s * 32, quad, q[b][0]);
        load_uniform(row + s * 32 + 16, quad, q[b][1]);
    };
    load(0, 0);
#pragma unroll 1
    for (int j4 = 0; j4 < CPW; j4 += 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t w[2], se[2];
            weight_word<TAB>(x[j], M, w[0], se[0]);
            w[1] = w[0];
            se[1] = se[0];
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const int local = j * H + h;
                load(min(j4 * H + local + 1, CPW * H - 1), (local + 1) & 1);
                float(&a)[2][CPW] = *reinterpret_cast<float(*)[2][CPW]>(&acc[2 * h]);
                fold<TAB, 2, 2>(w, se, q[local & 1], a, lut);
            }
        }
#pragma unroll
        for (int j = 0; j < CPW - 4; ++j) x[j] = x[j + 4];
    }
}

// One group of 16 columns on the checked path (`row`: the group's Words of the
// block's first row, rows Dp apart). seen: bit j, whether row j counts.
template <int TAB>
__device__ __forceinline__ void weigh_block_checked(float (&x)[CPW], uint32_t seen, const Word* row, int Dp, uint32_t quad,
                                                    float (&acc)[CPW], const unsigned char* lut, int M, int elo, int ehi)
{
#pragma unroll 1
    for (int j = 0; j < CPW; ++j) {
        int lo = 0, hi = 0;
        const Word w = attn_word(__float_as_uint(x[0]), M, true, elo, ehi, lo, hi);
        uint32_t q[UQ];
        load_uniform(row + (int64_t)j * Dp, quad, q);
        fold_checked<TAB>(w.w, w.se, q, acc, lut, elo, ehi, (seen >> j) & 1u);
#pragma unroll
        for (int i = 0; i < CPW - 1; ++i) x[i] = x[i + 1];
    }
}

// RN32(2^x), zero below 2^-64. The fraction's power is a polynomial in 64
// bits (the exponential series of f ln 2, |f| <= 1/2: remainder below 2^-41).
__device__ __forceinline__ float exp2_once(double x)
{
    const double n = __builtin_rint(x), f = x - n;
    double r = 7.0549116208011233e-09;                  // ln2^10 / 10!
    r = __builtin_fma(r, f, 1.0178086009239699e-07);
    r = __builtin_fma(r, f, 1.3215486790144307e-06);
    r = __builtin_fma(r, f, 1.5252733804059841e-05);
    r = __builtin_fma(r, f, 1.5403530393381609e-04);
    r = __builtin_fma(r, f, 1.3333558146428443e-03);
    r = __builtin_fma(r, f, 9.6181291076284772e-03);
    r = __builtin_fma(r, f, 5.5504108664821580e-02);
    r = __builtin_fma(r, f, 2.4022650695910071e-01);
    r = __builtin_fma(r, f, 6.9314718055994531e-01);
    r = __builtin_fma(r, f, 1.0);
    const float v = __builtin_ldexpf((float)r, (int)n);
    return x >= -64.0 ? v : 0.0f;
}

// The table copy, and the lookups' base.
template <int TAB>
__device__ __forceinline__ const unsigned char* stage_table(const uint16_t* lut, int M, unsigned char* lds)
{
    if constexpr (TAB == AT_LDS || TAB == AT_LDS8) {
        const uint4* src = reinterpret_cast<const uint4*>(lut);
        uint4* dst = reinterpret_cast<uint4*>(lds);
        const int n16 = attn_image_bytes(M) >> 4;
        for (int t = threadIdx.x; t < n16; t += blockDim.x) dst[t] = src[t];
        __syncthreads();
        return lds;
    }
    return reinterpret_cast<const unsigned char*>(lut);
}

template <int TAB>
constexpr int table_lds()
{
    return TAB == AT_LDS ? 33280 : TAB == AT_LDS8 ? 132096 : 16;
}
template <int TAB>
constexpr int attn_threads()
{
    return TAB == AT_LDS8 ? 512 : 256;        // at M = 8 one workgroup's table fills a CU's LDS
}

// ------------------------------------------------------------------ forward

// One row of 16 DC sums: scaled into the output, or as a partial.
template <int DC>
__device__ __forceinline__ void store_row(const float (&acc)[DC][CPW], float scale, float* o, int D, bool vec)
{
#pragma unroll
    for (int g = 0; g < DC; ++g)
#pragma unroll
        for (int c = 0; c < CPW; c += 4) {
            const int d = g * CPW + c;
            if (vec) {
                if (d < D) *reinterpret_cast<float4*>(o + d) = make_float4(acc[g][c] * scale, acc[g][c + 1] * scale, acc[g][c + 2] * scale, acc[g][c + 3] * scale);
            } else {
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    if (d + x < D) o[d + x] = acc[g][c + x] * scale;
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
__device__ __forceinline__ uint32_t seen_keys(const Row& r, const Span& sp, int j0)
{
    if (j0 >= sp.ks && j0 + kAttnBlock <= r.lim_lo) return 0xFFFFu;
    const int a = max(0, sp.ks - j0), n = min(max(r.lim - j0, 0), kAttnBlock);
    return ((1u << n) - 1u) & ~((1u << a) - 1u);
}

// NG groups of 16 columns (from group g0) of a row's result: partial, or o.
template <int NG>
__device__ __forceinline__ void store_fwd(const AttnParams& p, const Row& r, int h, int split, int g0,
                                          const float (&acc)[NG][CPW], double m, double l)
{
    if (!r.valid) return;
    if (p.splits > 1) {
        const int64_t at = ((int64_t)split * p.K + h) * p.RQ + r.row;
        p.part_m[at] = m;
        p.part_l[at] = l;
        if (l != 0.0) store_row<NG>(acc, 1.0f, p.part0 + at * p.Dp + g0 * CPW, p.Dp - g0 * CPW, true);
        return;
    }
    const int hh = h * p.G + (r.row - r.tok * p.G);
    const float inv = l == 0.0 ? 0.0f : (float)(1.0 / l);
    store_row<NG>(acc, inv, p.o + (int64_t)r.tok * p.ldo + (int64_t)hh * p.D + g0 * CPW, p.D - g0 * CPW,
                  rows_aligned(p.o, p.ldo, p.D));
    if (p.lse != nullptr)
        p.lse[(int64_t)r.tok * (p.K * p.G) + hh] = l == 0.0 ? -__builtin_inff() : (float)((m + log2(l)) * 0.69314718055994530942);
}

template <int TAB, int DC>
__device__ __forceinline__ void fwd_item(const AttnParams& p, const Span& sp, int h, int split, const unsigned char* lut)
{
    const uint32_t quad = threadIdx.x & 3u;
    const Row r = tile_row(p, sp, split);
    const Word* ql = p.q_lane + (int64_t)h * p.D4 * p.RQp + (int64_t)r.row * 4;
    const Word* kt = p.k_tr + (int64_t)h * p.TKp * p.D4;
    const Word* vr = p.v_row + (int64_t)h * p.TKp * p.Dp;
    float acc[DC][CPW];
#pragma unroll
    for (int g = 0; g < DC; ++g)
#pragma unroll
        for (int c = 0; c < CPW; ++c) acc[g][c] = 0.0f;
    double m = -__builtin_inf(), l = 0.0;
#pragma unroll 1
    for (int kb = r.b0; kb < r.b1; ++kb) {
        float s[1][CPW];
        dot_block<TAB>(ql, p.RQp, kt + (int64_t)kb * kAttnBlock * p.D4, p.D4, quad, s, lut);
        const uint32_t seen = seen_keys(r, sp, kb * kAttnBlock);
        float top = -__builtin_inff();
#pragma unroll
        for (int c = 0; c < CPW; ++c) top = fmaxf(top, (seen >> c) & 1u ? s[0][c] : -__builtin_inff());
        const double mn = fmax(m, __builtin_ceil((double)top * p.c));
        if (__any(mn > m)) {                 // a power of two: no mantissa changes
            const int d = mn > m ? (int)fmax(m - mn, -4096.0) : 0;
            l = __builtin_ldexp(l, d);
#pragma unroll
            for (int g = 0; g < DC; ++g)
#pragma unroll
                for (int c = 0; c < CPW; ++c) acc[g][c] = __builtin_ldexpf(acc[g][c], d);
            m = mn;
        }
#pragma unroll
        for (int c = 0; c < CPW; ++c) {
            const float e = exp2_once(__builtin_fma((double)s[0][c], p.c, -m));
            s[0][c] = (seen >> c) & 1u ? e : 0.0f;
            l += (double)s[0][c];
            if (c & 1) __builtin_amdgcn_sched_barrier(0);    // few temporaries at a time
        }
        weigh_block<TAB, DC>(s[0], vr + (int64_t)kb * kAttnBlock * p.Dp, quad, acc, lut, p.M);
    }
    store_fwd<DC>(p, r, h, split, 0, acc, m, l);
}

// The same on the checked path, kept small rather than fast: 16 columns of
// the values at a time, the scores computed again for each. A weight's
// product may leave the format's range here, and whether it does must not
// depend on the order of the keys: the row's maximum over all its keys comes
// first.
template <int TAB>
__device__ __forceinline__ void fwd_item_checked(const AttnParams& p, const Span& sp, int h, int split, const unsigned char* lut)
{
    const uint32_t quad = threadIdx.x & 3u;
    const Row r = tile_row(p, sp, split);
    const Word* ql = p.q_lane + (int64_t)h * p.D4 * p.RQp + (int64_t)r.row * 4;
    const Word* kt = p.k_tr + (int64_t)h * p.TKp * p.D4;
    float top = -__builtin_inff();
    bool bad = false;                        // a seen score is NaN or +Inf
#pragma unroll 1
    for (int kb = r.f0; kb < r.f1; ++kb) {
        float s[CPW];
        dot_block_checked<TAB>(ql, p.RQp, kt + (int64_t)kb * kAttnBlock * p.D4, p.D4, quad, s, lut, p.elo, p.ehi);
        const uint32_t seen = seen_keys(r, sp, kb * kAttnBlock);
#pragma unroll
        for (int c = 0; c < CPW; ++c) {
            const float v = (seen >> c) & 1u ? s[c] : -__builtin_inff();
            bad = bad || !(v < __builtin_inff());
            top = fmaxf(top, v);
        }
    }
    const double m = __builtin_ceil((double)top * p.c);
#pragma unroll 1
    for (int g = 0; g < p.Dp / CPW; ++g) {
        float acc[1][CPW];
#pragma unroll
        for (int c = 0; c < CPW; ++c) acc[0][c] = 0.0f;
        double l = 0.0;
#pragma unroll 1
        for (int kb = r.b0; kb < r.b1; ++kb) {
            float s[CPW];
            dot_block_checked<TAB>(ql, p.RQp, kt + (int64_t)kb * kAttnBlock * p.D4, p.D4, quad, s, lut, p.elo, p.ehi);
            const uint32_t seen = seen_keys(r, sp, kb * kAttnBlock);
#pragma unroll
            for (int c = 0; c < CPW; ++c) {
                const float e = exp2_once(__builtin_fma((double)s[c], p.c, -m));
                s[c] = ((seen >> c) & 1u) && !bad ? e : 0.0f;
                l += (double)s[c];
            }
            weigh_block_checked<TAB>(s, seen, p.v_row + ((int64_t)h * p.TKp + kb * kAttnBlock) * p.Dp + g * CPW, p.Dp, quad, acc[0],
                                     lut, p.M, p.elo, p.ehi);
        }
        if (bad) l = __builtin_nan("");
        store_fwd<1>(p, r, h, split, g, acc, m, l);
    }
}

// Persistent; one item per wave: a tile of 64 rows of one kv head and a chunk
// of its keys. Item order: heads outermost (the waves of a workgroup stream
// the same keys through one L1), then chunks, then tiles from the last (with
// a causal mask the longest first).
template <int TAB, int DC>
__global__ __launch_bounds__(attn_threads<TAB>(), 2) void attn_fwd_kernel(AttnParams p)
{
    __shared__ __align__(16) unsigned char lds[table_lds<TAB>()];
    const unsigned char* lut = stage_table<TAB>(p.lut, p.M, lds);
    int ql, qh, kl, kh, vl, vh;
    tensor_range(p.stats, 0, ql, qh);
    tensor_range(p.stats, 1, kl, kh);
    tensor_range(p.stats, 2, vl, vh);
    const bool fast = !p.force_checked && p.elo == 1 && range_fast<TAB>(ql, qh) && range_fast<TAB>(kl, kh) &&
                      range_fast<TAB>(vl, vh) && qh + kh <= p.smax;
    constexpr int W = attn_threads<TAB>() / 64;
    for (int64_t it = (int64_t)blockIdx.x * W + (threadIdx.x >> 6); it < p.items; it += (int64_t)gridDim.x * W) {
        const int item = __builtin_amdgcn_readfirstlane((int)it);
        const int t = p.tiles - 1 - item % p.tiles, r = item / p.tiles;
        const int split = r % p.splits, h = r / p.splits;
        const Span sp = find_tile(p.cu_q, p.total_q, p.cu_k, p.total_k, p.nseq, false, p.G, kAttnTile, t);
        if (sp.tile < 0) continue;
        if (fast) fwd_item<TAB, DC>(p, sp, h, split, lut);
        else fwd_item_checked<TAB>(p, sp, h, split, lut);
    }
}

// Joins the chunks of every row: 16 lanes per row.
__global__ __launch_bounds__(256) void attn_join_kernel(AttnJoinParams p)
{
    const int64_t at = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);   // kv head * RQ + row
    const int64_t rows = (int64_t)p.K * p.RQ;
    if (at >= rows) return;
    const int h = (int)(at / p.RQ), row = (int)(at - (int64_t)h * p.RQ);
    const int tok = row / p.G;
    // rows of no sequence keep what they hold
    int end = 0;
    for (int b = threadIdx.x & 15; b <= p.nseq; b += 16) end = max(end, min(max(p.cu_q[b], 0), p.total_q));
    for (int off = 8; off > 0; off >>= 1) end = max(end, __shfl_xor(end, off, 64));
    if (tok >= end || tok < max(0, p.cu_q[0])) return;
    double m = -__builtin_inf(), l = 0.0;
    for (int s = 0; s < p.splits; ++s)
        if (p.part_l[s * rows + at] != 0.0) m = fmax(m, p.part_m[s * rows + at]);
    for (int s = 0; s < p.splits; ++s) {
        const double ls = p.part_l[s * rows + at];
        if (ls != 0.0) l += __builtin_ldexp(ls, (int)fmax(p.part_m[s * rows + at] - m, -4096.0));
    }
    const int hh = h * p.G + (row - tok * p.G);
    const float inv = l == 0.0 ? 0.0f : (float)(1.0 / l);
    float* o = p.o + (int64_t)tok * p.ldo + (int64_t)hh * p.D;
    for (int d = threadIdx.x & 15; d < p.D; d += 16) {
        float a = 0.0f;
        for (int s = 0; s < p.splits; ++s)
            if (p.part_l[s * rows + at] != 0.0)
                a += __builtin_ldexpf(p.part[(s * rows + at) * p.Dp + d], (int)fmax(p.part_m[s * rows + at] - m, -4096.0));
        o[d] = a * inv;
    }
    if (p.lse != nullptr && (threadIdx.x & 15) == 0)
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

// dQ of 64 rows over a chunk of their keys: the scores and dP of 16 keys,
// then dS (in the lanes that hold it) times the keys' rows.
struct Backward {
    int64_t lane_at, tr_at, row_at;
    float lse, delta;
    double base;
};
__device__ __forceinline__ Backward row_state(const AttnParams& p, const Row& r, int h)
{
    Backward b;
    b.lane_at = (int64_t)h * p.D4 * p.RQp + (int64_t)r.row * 4;
    b.tr_at = (int64_t)h * p.TKp * p.D4;
    b.row_at = (int64_t)h * p.TKp * p.Dp;
    b.lse = p.rowlse[(int64_t)h * p.RQp + r.row];
    b.delta = p.delta[(int64_t)h * p.RQp + r.row];
    b.base = (double)b.lse * 1.4426950408889634074;
    return b;
}

template <int NG>
__device__ __forceinline__ void store_dq(const AttnParams& p, const Row& r, int h, int split, int g0, const float (&acc)[NG][CPW])
{
    if (!r.valid) return;
    if (p.splits > 1) {
        store_row<NG>(acc, 1.0f, p.part0 + (((int64_t)split * p.K + h) * p.RQ + r.row) * p.Dp + g0 * CPW, p.Dp - g0 * CPW, true);
    } else {
        float* o = p.dq + (int64_t)r.tok * p.lddq + (int64_t)(h * p.G + (r.row - r.tok * p.G)) * p.D;
        store_row<NG>(acc, p.scale, o + g0 * CPW, p.D - g0 * CPW, rows_aligned(p.dq, p.lddq, p.D));
    }
}

template <int TAB, int DC>
__device__ __forceinline__ void dq_item(const AttnParams& p, const Span& sp, int h, int split, const unsigned char* lut)
{
    const uint32_t quad = threadIdx.x & 3u;
    const Row r = tile_row(p, sp, split);
    const Backward b = row_state(p, r, h);
    float acc[DC][CPW];
#pragma unroll
    for (int g = 0; g < DC; ++g)
#pragma unroll
        for (int c = 0; c < CPW; ++c) acc[g][c] = 0.0f;
#pragma unroll 1
    for (int kb = r.b0; kb < r.b1; ++kb) {
        float s[1][CPW], dp[1][CPW];
        const int64_t at = b.tr_at + (int64_t)kb * kAttnBlock * p.D4;
        dot_block<TAB>(p.q_lane + b.lane_at, p.RQp, p.k_tr + at, p.D4, quad, s, lut);
        dot_block<TAB>(p.do_lane + b.lane_at, p.RQp, p.v_tr + at, p.D4, quad, dp, lut);
        const uint32_t seen = seen_keys(r, sp, kb * kAttnBlock);
#pragma unroll
        for (int c = 0; c < CPW; ++c) {
            float pr, ds;
            score_gradient<false>(__builtin_fma((double)s[0][c], p.c, -b.base), b.lse, dp[0][c], b.delta, pr, ds);
            s[0][c] = (seen >> c) & 1u ? ds : 0.0f;
            if (c & 1) __builtin_amdgcn_sched_barrier(0);    // few temporaries at a time
        }
        weigh_block<TAB, DC>(s[0], p.k_row + b.row_at + (int64_t)kb * kAttnBlock * p.Dp, quad, acc, lut, p.M);
    }
    store_dq<DC>(p, r, h, split, 0, acc);
}

template <int TAB>
__device__ __forceinline__ void dq_item_checked(const AttnParams& p, const Span& sp, int h, int split, const unsigned char* lut)
{
    const uint32_t quad = threadIdx.x & 3u;
    const Row r = tile_row(p, sp, split);
    const Backward b = row_state(p, r, h);
#pragma unroll 1
    for (int g = 0; g < p.Dp / CPW; ++g) {
        float acc[1][CPW];
#pragma unroll
        for (int c = 0; c < CPW; ++c) acc[0][c] = 0.0f;
#pragma unroll 1
        for (int kb = r.b0; kb < r.b1; ++kb) {
            float s[CPW], dp[CPW];
            const int64_t at = b.tr_at + (int64_t)kb * kAttnBlock * p.D4;
            dot_block_checked<TAB>(p.q_lane + b.lane_at, p.RQp, p.k_tr + at, p.D4, quad, s, lut, p.elo, p.ehi);
            dot_block_checked<TAB>(p.do_lane + b.lane_at, p.RQp, p.v_tr + at, p.D4, quad, dp, lut, p.elo, p.ehi);
            const uint32_t seen = seen_keys(r, sp, kb * kAttnBlock);
#pragma unroll
            for (int c = 0; c < CPW; ++c) {
                float pr, ds;
                score_gradient<true>(__builtin_fma((double)s[c], p.c, -b.base), b.lse, dp[c], b.delta, pr, ds);
                s[c] = (seen >> c) & 1u ? ds : 0.0f;
            }
            weigh_block_checked<TAB>(s, seen, p.k_row + b.row_at + (int64_t)kb * kAttnBlock * p.Dp + g * CPW, p.Dp, quad, acc[0],
                                     lut, p.M, p.elo, p.ehi);
        }
        store_dq<1>(p, r, h, split, g, acc);
    }
}

// dK and dV of 64 keys over a chunk of the rows that see them, 16 rows at a
// time as uniform operands (which the products take first: the image with the
// uniform operand first). MODE: bit 0 dV, bit 1 dK.
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

template <int NG>
__device__ __forceinline__ void store_key(const AttnParams& p, const Key& k, int h, int split, int g0, const float (&acc)[NG][CPW],
                                          float* part, float* out, int64_t ld, float scale)
{
    if (!k.valid) return;
    if (p.splits > 1)
        store_row<NG>(acc, 1.0f, part + (((int64_t)split * p.K + h) * p.total_k + k.key) * p.Dp + g0 * CPW, p.Dp - g0 * CPW, true);
    else
        store_row<NG>(acc, scale, out + (int64_t)k.key * ld + (int64_t)h * p.D + g0 * CPW, p.D - g0 * CPW, rows_aligned(out, ld, p.D));
}

template <int TAB, int DC, int MODE>
__device__ __forceinline__ void dkv_item(const AttnParams& p, const Span& sp, int h, int split, const unsigned char* lut)
{
    const uint32_t quad = threadIdx.x & 3u;
    const Key k = tile_key(p, sp, split);
    const int64_t lane_at = (int64_t)h * p.D4 * p.TKp + (int64_t)k.key * 4;
    const int64_t tr_at = (int64_t)h * p.RQp * p.D4, row_at = (int64_t)h * p.RQp * p.Dp;
    constexpr int DV = (MODE & 1) ? DC : 1, DK = (MODE & 2) ? DC : 1;
    float dv[DV][CPW], dk[DK][CPW];
#pragma unroll
    for (int g = 0; g < DV; ++g)
#pragma unroll
        for (int c = 0; c < CPW; ++c) dv[g][c] = 0.0f;
#pragma unroll
    for (int g = 0; g < DK; ++g)
#pragma unroll
        for (int c = 0; c < CPW; ++c) dk[g][c] = 0.0f;
#pragma unroll 1
    for (int rb = k.b0; rb < k.b1; ++rb) {
        float s[1][CPW], dp[1][CPW];
        const int64_t at = tr_at + (int64_t)rb * kAttnBlock * p.D4;
        dot_block<TAB>(p.k_lane + lane_at, p.TKp, p.q_tr + at, p.D4, quad, s, lut);
        if constexpr (MODE & 2) dot_block<TAB>(p.v_lane + lane_at, p.TKp, p.do_tr + at, p.D4, quad, dp, lut);
        const int r0 = rb * kAttnBlock;
        const uint32_t seen = seeing_rows(p, sp, k, r0);
        const float* lse_at = p.rowlse + (int64_t)h * p.RQp + r0;
        const float* delta_at = p.delta + (int64_t)h * p.RQp + r0;
#pragma unroll
        for (int c = 0; c < CPW; ++c) {
            const float lse = lse_at[c];
            float pr, ds;
            score_gradient<false>(__builtin_fma((double)s[0][c], p.c, -((double)lse * 1.4426950408889634074)), lse,
                                  (MODE & 2) ? dp[0][c] : 0.0f, (MODE & 2) ? delta_at[c] : 0.0f, pr, ds);
            const bool in = (seen >> c) & 1u;
            s[0][c] = in ? pr : 0.0f;
            dp[0][c] = in ? ds : 0.0f;
            if (c & 1) __builtin_amdgcn_sched_barrier(0);    // few temporaries at a time
        }
        const int64_t rat = row_at + (int64_t)rb * kAttnBlock * p.Dp;
        if constexpr (MODE & 1) weigh_block<TAB, DC>(s[0], p.do_row + rat, quad, dv, lut, p.M);
        if constexpr (MODE & 2) weigh_block<TAB, DC>(dp[0], p.q_row + rat, quad, dk, lut, p.M);
    }
    if constexpr (MODE & 1) store_key<DC>(p, k, h, split, 0, dv, p.part0, p.dv, p.lddv, 1.0f);
    if constexpr (MODE & 2) store_key<DC>(p, k, h, split, 0, dk, p.part1, p.dk, p.lddk, p.scale);
}

template <int TAB, int MODE>
__device__ __forceinline__ void dkv_item_checked(const AttnParams& p, const Span& sp, int h, int split, const unsigned char* lut)
{
    const uint32_t quad = threadIdx.x & 3u;
    const Key k = tile_key(p, sp, split);
    const int64_t lane_at = (int64_t)h * p.D4 * p.TKp + (int64_t)k.key * 4;
    const int64_t tr_at = (int64_t)h * p.RQp * p.D4, row_at = (int64_t)h * p.RQp * p.Dp;
    // the column groups of dV (even passes) and dK (odd)
#pragma unroll 1
    for (int gg = 0; gg < 2 * (p.Dp / CPW); ++gg) {
        const bool want_dk = gg & 1;
        if (!(MODE & (want_dk ? 2 : 1))) continue;
        const int g = gg >> 1;
        float acc[1][CPW];
#pragma unroll
        for (int c = 0; c < CPW; ++c) acc[0][c] = 0.0f;
#pragma unroll 1
        for (int rb = k.b0; rb < k.b1; ++rb) {
            float s[CPW], dp[CPW];
            const int64_t at = tr_at + (int64_t)rb * kAttnBlock * p.D4;
            dot_block_checked<TAB>(p.k_lane + lane_at, p.TKp, p.q_tr + at, p.D4, quad, s, lut, p.elo, p.ehi);
            dot_block_checked<TAB>(p.v_lane + lane_at, p.TKp, p.do_tr + at, p.D4, quad, dp, lut, p.elo, p.ehi);
            const int r0 = rb * kAttnBlock;
            const uint32_t seen = seeing_rows(p, sp, k, r0);
            const float* lse_at = p.rowlse + (int64_t)h * p.RQp + r0;
            const float* delta_at = p.delta + (int64_t)h * p.RQp + r0;
#pragma unroll
            for (int c = 0; c < CPW; ++c) {
                const float lse = lse_at[c];
                float pr, ds;
                score_gradient<true>(__builtin_fma((double)s[c], p.c, -((double)lse * 1.4426950408889634074)), lse, dp[c],
                                     delta_at[c], pr, ds);
                s[c] = (seen >> c) & 1u ? (want_dk ? ds : pr) : 0.0f;
            }
            const Word* row = (want_dk ? p.q_row : p.do_row) + row_at + (int64_t)rb * kAttnBlock * p.Dp + g * CPW;
            weigh_block_checked<TAB>(s, seen, row, p.Dp, quad, acc[0], lut, p.M, p.elo, p.ehi);
        }
        if (want_dk) store_key<1>(p, k, h, split, g, acc, p.part1, p.dk, p.lddk, p.scale);
        else store_key<1>(p, k, h, split, g, acc, p.part0, p.dv, p.lddv, 1.0f);
    }
}

// MODE 0: dQ; else dkv_item's.
template <int TAB, int DC, int MODE>
__global__ __launch_bounds__(attn_threads<TAB>(), 2) void attn_bwd_kernel(AttnParams p)
{
    __shared__ __align__(16) unsigned char lds[table_lds<TAB>()];
    const unsigned char* lut = stage_table<TAB>(p.lut, p.M, lds);
    bool fast = !p.force_checked && p.elo == 1;
    int lo[4], hi[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        tensor_range(p.stats, t, lo[t], hi[t]);
        fast = fast && range_fast<TAB>(lo[t], hi[t]);
    }
    fast = fast && hi[0] + hi[2] <= p.smax;
    constexpr int W = attn_threads<TAB>() / 64;
    for (int64_t it = (int64_t)blockIdx.x * W + (threadIdx.x >> 6); it < p.items; it += (int64_t)gridDim.x * W) {
        const int item = __builtin_amdgcn_readfirstlane((int)it);
        const int tt = item % p.tiles, r = item / p.tiles;
        const int t = MODE == 0 ? p.tiles - 1 - tt : tt;       // with a causal mask the longest first
        const int split = r % p.splits, h = r / p.splits;
        const Span sp = find_tile(p.cu_q, p.total_q, p.cu_k, p.total_k, p.nseq, MODE != 0, MODE == 0 ? p.G : 1, kAttnTile, t);
        if (sp.tile < 0) continue;
        if constexpr (MODE == 0) {
            if (fast) dq_item<TAB, DC>(p, sp, h, split, lut);
            else dq_item_checked<TAB>(p, sp, h, split, lut);
        } else {
            if (fast) dkv_item<TAB, DC, MODE>(p, sp, h, split, lut);
            else dkv_item_checked<TAB, MODE>(p, sp, h, split, lut);
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

// ------------------------------------------------------------------ paged cache

// Few rows over many keys, read from the cache as it lies: a wave takes a
// block of NR rows (uniform operands, the products' first) and a chunk of
// keys, 64 at a time. Scores: one key per lane, its elements decoded as they
// are read. The numerators then go through LDS as Words, 16 keys at a time,
// and become the uniform operand of P V, whose lanes are the value's columns.
// Each key and value element is read once per row block and serves NR
// products; for a token or two the cache's bytes bound the kernel, for more
// rows the table lookups.
constexpr int kPagedKeys = 64;

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
__global__ __launch_bounds__(attn_threads<TAB>(), 2) void attn_paged_kernel(PagedParams p)
{
    constexpr int W = attn_threads<TAB>() / 64;
    __shared__ __align__(16) unsigned char lds[table_lds<TAB>()];
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
        uint32_t* buf = words[threadIdx.x >> 6];
        if (!q_fast || !paged_item<TAB, NR, VC>(p, b, split, lut, buf, q_hi)) paged_item_checked<TAB, NR>(p, b, split, lut, buf);
    }
}

// ------------------------------------------------------------------ launchers

hipError_t launch_attn_decode(const AttnDecodeParams& p, hipStream_t s)
{
    attn_decode_kernel<<<dim3(kAttnSlots, p.count), kDecodeThreads, 0, s>>>(p);
    return hipGetLastError();
}

// Resident workgroups of a kernel on the current device (queried once per
// device and kernel).
constexpr int kMaxGpus = 64;
static int resident(std::atomic<int>* cache, const void* f, int threads)
{
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxGpus) return 256;
    int n = cache[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        int cus = 0, per = 0;
        if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus < 1) cus = 1;
        if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&per, f, threads, 0) != hipSuccess || per < 1) per = 1;
        n = cus * per;
        cache[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

static hipError_t launch_join(const AttnJoinParams& p, hipStream_t s)
{
    attn_join_kernel<<<(unsigned)(((int64_t)p.K * p.RQ + 15) / 16), 256, 0, s>>>(p);
    return hipGetLastError();
}

template <int TAB, int DC>
static hipError_t run_fwd(const AttnParams& p, hipStream_t s)
{
    static std::atomic<int> cache[kMaxGpus];
    constexpr int NT = attn_threads<TAB>();
    const int64_t want = (p.items + NT / 64 - 1) / (NT / 64);
    const int grid = (int)std::min<int64_t>(want, resident(cache, reinterpret_cast<const void*>(&attn_fwd_kernel<TAB, DC>), NT));
    attn_fwd_kernel<TAB, DC><<<grid, NT, 0, s>>>(p);
    return hipGetLastError();
}

template <int TAB>
static hipError_t run_fwd_dim(const AttnParams& p, hipStream_t s)
{
    return p.Dp <= 64 ? run_fwd<TAB, 4>(p, s) : run_fwd<TAB, 8>(p, s);
}

hipError_t launch_attn_fwd(const AttnParams& p, hipStream_t s)
{
    hipError_t e;
    switch (attn_table_kind(p.M)) {
    case AT_LDS: e = run_fwd_dim<AT_LDS>(p, s); break;
    case AT_LDS8: e = run_fwd_dim<AT_LDS8>(p, s); break;
    case AT_GLOBAL: e = run_fwd_dim<AT_GLOBAL>(p, s); break;
    default: e = run_fwd_dim<AT_NATIVE>(p, s); break;
    }
    if (e != hipSuccess || p.splits == 1) return e;
    return launch_join(AttnJoinParams{p.cu_q, p.nseq, p.K, p.G, p.D, p.Dp, p.total_q, p.RQ, p.splits, p.part0, p.part_m,
                                      p.part_l, p.o, p.ldo, p.lse}, s);
}

template <int TAB, int DC, int MODE>
static hipError_t run_bwd(const AttnParams& p, hipStream_t s)
{
    static std::atomic<int> cache[kMaxGpus];
    constexpr int NT = attn_threads<TAB>();
    const int64_t want = (p.items + NT / 64 - 1) / (NT / 64);
    const int grid = (int)std::min<int64_t>(want, resident(cache, reinterpret_cast<const void*>(&attn_bwd_kernel<TAB, DC, MODE>), NT));
    attn_bwd_kernel<TAB, DC, MODE><<<grid, NT, 0, s>>>(p);
    return hipGetLastError();
}

template <int TAB>
static hipError_t run_bwd_dim(const AttnParams& p, bool keys, hipStream_t s)
{
    if (!keys) return p.Dp <= 64 ? run_bwd<TAB, 4, 0>(p, s) : run_bwd<TAB, 8, 0>(p, s);
    if (p.Dp <= 64) return run_bwd<TAB, 4, 3>(p, s);
    // 256 accumulators per lane do not fit: dV and dK in a launch each
    const hipError_t e = run_bwd<TAB, 8, 1>(p, s);
    return e != hipSuccess ? e : run_bwd<TAB, 8, 2>(p, s);
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
    case AT_LDS: e = run_bwd_dim<AT_LDS>(p, keys, s); break;
    case AT_LDS8: e = run_bwd_dim<AT_LDS8>(p, keys, s); break;
    case AT_GLOBAL: e = run_bwd_dim<AT_GLOBAL>(p, keys, s); break;
    default: e = run_bwd_dim<AT_NATIVE>(p, keys, s); break;
    }
    if (e != hipSuccess || p.splits == 1) return e;
    if (!keys) return launch_sum(p, false, p.part0, p.dq, p.lddq, p.scale, s);
    e = launch_sum(p, true, p.part0, p.dv, p.lddv, 1.0f, s);
    return e != hipSuccess ? e : launch_sum(p, true, p.part1, p.dk, p.lddk, p.scale, s);
}

template <int TAB, int NR, int VC>
static hipError_t run_paged(const PagedParams& p, hipStream_t s)
{
    static std::atomic<int> cache[kMaxGpus];
    constexpr int NT = attn_threads<TAB>();
    const int64_t want = (p.items + NT / 64 - 1) / (NT / 64);
    const int grid = (int)std::min<int64_t>(want, resident(cache, reinterpret_cast<const void*>(&attn_paged_kernel<TAB, NR, VC>), NT));
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
