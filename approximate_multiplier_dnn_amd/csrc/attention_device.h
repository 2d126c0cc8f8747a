// attention_device.h -- device code shared by the attention kernels
// (attention.hip: packed prompts; paged.hip: a paged cache): operand words,
// exponent ranges, sequences, products on the fast and the checked path, and
// the softmax's exponential.
#pragma once
#include <algorithm>
#include <atomic>

#include "attention.h"
#include "product.h"

namespace amx {

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
// (queries: tokens * mult; keys: tokens) are cut into tiles of `size`. Up to
// 64 sequences: tiles are numbered by their rank in the sequence, rows from
// the last tile and keys from the first (with a causal mask the longest), so
// that the longest tiles come first and short ones end the launch; more
// sequences: one after the other.
// Offsets are clamped to the tensors and to their running maximum, so
// whatever they hold, sequences stay inside and do not overlap.
__device__ __forceinline__ Span find_tile(const int* cu_q, int total_q, const int* cu_k, int total_k, int nseq,
                                          bool by_key, int mult, int size, int t, const int* k_len = nullptr, int k_stride = 0,
                                          int k_most = 0)
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
        int ks, ke;
        if (k_len != nullptr) {                         // fixed places, a length each
            ks = bq * k_stride;
            ke = ks + (b < nseq ? min(max(k_len[b], 0), k_most) : 0);
        } else {
            ks = max(ck, wave_prefix_max(min(max(cu_k[bq], 0), total_k)));
            ke = max(ks, min(max(cu_k[b1], 0), total_k));
        }
        const int n = by_key ? ke - ks : qe - qs;
        const int tiles = b < nseq ? (n * mult + size - 1) / size : 0;
        int l = -1;
        if (nseq <= 64) {
            // ranks 0, 1, ... of the sequences that have so many tiles
            int left = t, rank = 0;
            for (;; ++rank) {
                const uint64_t have = __ballot(tiles > rank);
                const int count = __builtin_popcountll(have);
                if (count == 0) break;
                if (count == 1) {                       // one sequence: its other tiles in a step
                    const int only = __builtin_ctzll(have);
                    rank += left;
                    l = rank < __shfl(tiles, only, 64) ? only : -1;
                    break;
                }
                if (left < count) {                     // the left-th of these sequences
                    uint64_t rest = have;
                    for (int i = 0; i < left; ++i) rest &= rest - 1;
                    l = __builtin_ctzll(rest);
                    break;
                }
                left -= count;
            }
            if (l < 0) break;
            sp.tile = by_key ? rank : __shfl(tiles, l, 64) - 1 - rank;
        } else {
            const int incl = base + wave_prefix_sum(tiles);
            const uint64_t found = __ballot(incl > t);
            if (found) {
                l = __builtin_ctzll(found);
                sp.tile = t - (__shfl(incl, l, 64) - __shfl(tiles, l, 64));
            }
            base = __shfl(incl, 63, 64);
        }
        if (l >= 0) {
            sp.seq = b0 + l;
            sp.qs = __shfl(qs, l, 64);
            sp.qn = __shfl(qe, l, 64) - sp.qs;
            sp.ks = __shfl(ks, l, 64);
            sp.kn = __shfl(ke, l, 64) - sp.ks;
            break;
        }
        cq = __shfl(qe, 63, 64);
        ck = __shfl(ke, 63, 64);
    }
    sp.qs = __builtin_amdgcn_readfirstlane(sp.qs);
    sp.qn = __builtin_amdgcn_readfirstlane(sp.qn);
    sp.ks = __builtin_amdgcn_readfirstlane(sp.ks);
    sp.kn = __builtin_amdgcn_readfirstlane(sp.kn);
    sp.seq = __builtin_amdgcn_readfirstlane(sp.seq);
    sp.tile = __builtin_amdgcn_readfirstlane(sp.tile);
    return sp;
}

// ------------------------------------------------------------------ products

// Where the lookups read: the table's address in LDS, or its place in global
// memory. Lane operands carry `lds` in their offsets (one addition per operand
// instead of one per lookup), so a lookup adds only the uniform's offset, in
// the instruction that broadcasts it.
struct Table {
    const unsigned char* global;
    uint32_t lds;
};

template <int TAB>
__device__ __forceinline__ uint32_t table_at(const Table& t, uint32_t off)
{
    if constexpr (TAB == AT_GLOBAL)
        return *reinterpret_cast<const uint16_t __attribute__((address_space(1)))*>(
            (const unsigned char __attribute__((address_space(1)))*)t.global + off);
    else return *(const uint16_t __attribute__((address_space(3)))*)(uintptr_t)off;
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
                                     float (&acc)[GR][NC], const Table& lut)
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
                                             const Table& lut, int elo, int ehi, bool keep, uint32_t cols = 0xFFFFu)
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

// Uniform words of one step in NQ registers: 8 (NQ = 4) or 16 (NQ = 8) columns.
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

// acc[c] = FP32 sums, ascending over d, of T(row d, column c's d): the lane
// panel's row at `lane` (Words at [D4 / 4][Rp][4]), CW uniform columns at `tr`
// (of [D4][16]). Two steps at a time, their words requested two steps ahead.
template <int TAB, int CW>
__device__ __forceinline__ void dot_block(const Word* lane, int64_t Rp, const Word* tr, int D4, float (&acc)[1][CW], const Table& lut)
{
    uint32_t wa[2][2], sa[2][2], q[2][2][CW / 2];
    auto load = [&](int s, int b) {
        const uint4 w = *reinterpret_cast<const uint4*>(lane + (int64_t)(s >> 1) * Rp * 4 + (s & 1) * 2);
        wa[b][0] = w.x + lut.lds; sa[b][0] = w.y; wa[b][1] = w.z + lut.lds; sa[b][1] = w.w;
        load_columns(tr + s * 32, q[b][0]);
        load_columns(tr + s * 32 + 16, q[b][1]);
    };
    const int steps = D4 / 2;                 // even
#pragma unroll
    for (int c = 0; c < CW; ++c) acc[0][c] = 0.0f;
    load(0, 0);
#pragma unroll 1
    for (int s = 0; s < steps; s += 2) {
        load(s + 1, 1);
        fold<TAB, 2, 1, CW, CW / 2>(wa[0], sa[0], q[0], acc, lut);
        load(min(s + 2, steps - 1), 0);
        fold<TAB, 2, 1, CW, CW / 2>(wa[1], sa[1], q[1], acc, lut);
    }
}

template <int TAB>
__device__ __forceinline__ void dot_block_checked(const Word* lane, int64_t Rp, const Word* tr, int D4, uint32_t quad,
                                                  float (&acc)[CPW], const Table& lut, int elo, int ehi)
{
#pragma unroll
    for (int c = 0; c < CPW; ++c) acc[c] = 0.0f;
#pragma unroll 1
    for (int d = 0; d < D4; ++d) {
        const uint2 w = *reinterpret_cast<const uint2*>(lane + (int64_t)(d >> 2) * Rp * 4 + (d & 3));
        uint32_t q[UQ];
        load_uniform(tr + d * CPW, quad, q);
        fold_checked<TAB>(w.x + lut.lds, w.y, q, acc, lut, elo, ehi, true);
    }
}

// One group of 16 columns on the checked path (`row`: the group's Words
// [16][16] of the block's rows). seen: bit j, whether row j counts.
template <int TAB>
__device__ __forceinline__ void weigh_block_checked(float (&x)[CPW], uint32_t seen, const Word* row, uint32_t quad,
                                                    float (&acc)[CPW], const Table& lut, int M, int elo, int ehi)
{
#pragma unroll 1
    for (int j = 0; j < CPW; ++j) {
        int lo = 0, hi = 0;
        const Word w = attn_word(__float_as_uint(x[0]), M, true, elo, ehi, lo, hi);
        uint32_t q[UQ];
        load_uniform(row + j * CPW, quad, q);
        fold_checked<TAB>(w.w + lut.lds, w.se, q, acc, lut, elo, ehi, (seen >> j) & 1u);
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

// f(element, its place) over a block's CW values, in a loop of four (rotating
// the registers): few temporaries at a time.
template <int CW, typename F>
__device__ __forceinline__ void each_value(float (&x)[CW], F f)
{
#pragma unroll 1
    for (int g = 0; g < CW; g += 4) {
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = f(x[i], g + i);
#pragma unroll
        for (int i = 0; i < CW - 4; ++i) x[i] = x[i + 4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[CW - 4 + i] = y[i];
    }
}

// The table copy, and where the lookups read it.
template <int TAB>
__device__ __forceinline__ Table stage_table(const uint16_t* lut, int M, unsigned char* lds)
{
    Table t{reinterpret_cast<const unsigned char*>(lut), 0u};
    if constexpr (TAB == AT_LDS || TAB == AT_LDS8) {
        const uint4* src = reinterpret_cast<const uint4*>(lut);
        uint4* dst = reinterpret_cast<uint4*>(lds);
        const int n16 = attn_image_bytes(M) >> 4;
        for (int i = threadIdx.x; i < n16; i += blockDim.x) dst[i] = src[i];
        __syncthreads();
        t.lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)lds;
        asm("" : "+s"(t.lds));               // kept out of the lookups' address arithmetic
    }
    return t;
}

template <int TAB>
constexpr int table_lds()
{
    return TAB == AT_LDS ? 33280 : TAB == AT_LDS8 ? 132096 : 0;
}

// Resident workgroups of a kernel on the current device (queried once per
// device, kernel and configuration `slot`), after allowing it all of a CU's
// LDS as dynamic LDS.
constexpr int kLdsBytes = 163840;
constexpr int kMaxGpus = 64;
constexpr int kMaxConfigs = 16;
struct Resident {
    std::atomic<int> n[kMaxGpus][kMaxConfigs];
};
inline int resident(Resident& cache, int slot, const void* f, int threads, size_t lds)
{
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxGpus) return 0;
    int n = cache.n[dev][slot].load(std::memory_order_relaxed);
    if (n == 0) {
        int cus = 0, per = 0;
        if (lds > 0 && hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, kLdsBytes) != hipSuccess) return 0;
        if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus < 1) return 0;
        if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&per, f, threads, lds) != hipSuccess || per < 1) return 0;
        n = cus * per;
        cache.n[dev][slot].store(n, std::memory_order_relaxed);
    }
    return n;
}

hipError_t launch_join(const AttnJoinParams& p, hipStream_t s);

}  // namespace amx
