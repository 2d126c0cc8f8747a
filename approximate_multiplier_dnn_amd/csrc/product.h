// product.h -- device code of one approximate product and of its operands'
// delivery, shared by the GEMM kernels (kernels.hip) and the attention
// kernels (attention.hip).
#pragma once
#include "internal.h"

namespace amx {

// Output columns per wave (uniform operands of one reduction index).
constexpr int CPW = kColsPerWave;

// Exponent cast of an FP32 operand to the multiplier's format (1, E, M)
// (ApproxTrain Section V: exponent widths below 8 with a casting function):
// a normal value whose biased exponent lies below elo becomes a signed zero,
// above ehi a signed infinity; zero, subnormal, Inf and NaN are kept. The
// identity for FP32's own range (elo = 1, ehi = 254).
__device__ __forceinline__ uint32_t cast_fmt(uint32_t bits, int elo, int ehi)
{
    const int e = (int)((bits >> 23) & 0xFFu);
    const uint32_t sign = bits & 0x80000000u;
    bits = (e != 0 && e != 255 && e < elo) ? sign : bits;
    bits = (e != 0 && e != 255 && e > ehi) ? (sign | 0x7F800000u) : bits;
    return bits;
}

// M = 0 selects the native multiplier: the Word carries the operand's own
// bits (se) and no table offset, and the exponent range is not gathered (nor
// is the operand cast: the native multiplier is FP32).
__device__ __forceinline__ Word decode_bits(uint32_t bits, int M, int lane_role, int& emin, int& emax, int elo,
                                            int ehi)
{
    if (M == 0) return Word{0u, bits};
    bits = cast_fmt(bits, elo, ehi);
    const uint32_t e = (bits >> 23) & 0xFFu;
    const uint32_t frac = bits & 0x7FFFFFu;
    const uint32_t idx = frac >> (23 - M);
    const uint32_t pad = (1u << M) * 2u;            // zero entry after the column's 2^M entries
    const uint32_t colb = (uint32_t)lut_col_bytes(M);   // column stride in bytes
    Word o;
    if (e == 0u) {                                  // zero or subnormal (counts as zero)
        o.se = 0u;
        o.w = lane_role ? pad : 0u;
    } else if (e == 255u) {                         // Inf or NaN
        o.se = frac ? 0x7FC00000u : (bits & 0xFF800000u);
        o.w = lane_role ? pad : 0u;
    } else {
        o.se = bits & 0xFF800000u;
        o.w = lane_role ? idx * 2u : idx * colb;
        emin = min(emin, (int)e);
        emax = max(emax, (int)e);
    }
    return o;
}

// Checked path: Algorithm 2 with every special case, as selects (no
// divergence), then acc + product. seA, seB: operands already cast to the
// format; elo..ehi: the format's normal range of biased exponents.
__device__ __forceinline__ float checked_product_acc(float acc, uint32_t e, uint32_t seA, uint32_t seB, int elo,
                                                     int ehi)
{
    const uint32_t ea = (seA >> 23) & 0xFFu, eb = (seB >> 23) & 0xFFu;
    const uint32_t sign = (seA ^ seB) & 0x80000000u;
    const int ex = (int)ea + (int)eb - 127 + (int)(e >> 15);
    uint32_t bits = sign | ((uint32_t)(ex & 0xFF) << 23) | ((e & 0x7FFFu) << 8);
    bits = ex > ehi ? (sign | 0x7F800000u) : bits;             // overflow -> signed Inf
    bits = ex < elo ? sign : bits;                             // underflow -> signed zero
    const bool zero = ea == 0u || eb == 0u;                    // zero or subnormal operand
    const bool a_inf = ea == 255u && (seA & 0x7FFFFFu) == 0u;
    const bool b_inf = eb == 255u && (seB & 0x7FFFFFu) == 0u;
    const bool nan = (ea == 255u && (seA & 0x7FFFFFu) != 0u) || (eb == 255u && (seB & 0x7FFFFFu) != 0u);
    bits = zero ? sign : bits;
    bits = (a_inf || b_inf) ? (zero ? 0x7FC00000u : (sign | 0x7F800000u)) : bits;
    bits = nan ? 0x7FC00000u : bits;
    return acc + __uint_as_float(bits);
}


// Uniform words of one reduction index for this wave's 16 columns, spread
// over the 4 lanes of each quad: lane i of a quad holds, in register
// 4j + t, dword 16j + 4i + t of the 32 dwords {w0, se0, w1, se1, ...}.
// 8 VGPRs per index instead of 32 (a quarter of the vector-memory return
// traffic of a full broadcast); a consumer reads column c's value with a
// quad_perm DPP broadcast of lane (c >> 1) & 3, folded into its own
// instruction (v_add_u32_dpp, v_fmac_f32_dpp).
constexpr int UQ = 8;

__device__ __forceinline__ void load_uniform(const Word* row, uint32_t quad, uint32_t (&q)[UQ])
{
    const uint4* src = reinterpret_cast<const uint4*>(row) + quad;
    const uint4 a = src[0], b = src[4];
    q[0] = a.x; q[1] = a.y; q[2] = a.z; q[3] = a.w;
    q[4] = b.x; q[5] = b.y; q[6] = b.z; q[7] = b.w;
}

// Lane i of every quad, broadcast to the quad (quad_perm:[i,i,i,i]). i is a
// constant once the callers' loops are unrolled.
__device__ __forceinline__ uint32_t quad_bcast(uint32_t v, int i)
{
    switch (i) {
    case 0: return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x00, 0xF, 0xF, true);
    case 1: return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x55, 0xF, 0xF, true);
    case 2: return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xAA, 0xF, 0xF, true);
    default: return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xFF, 0xF, 0xF, true);
    }
}

// acc += (lane i of this lane's quad in q) * x, one v_fmac_f32 with a DPP
// broadcast operand (the compiler does not fold a DPP move into an FMA on
// this target). The asm statement also keeps each fold in place in the
// schedule. q comes straight from vector-memory loads, so no VALU write
// precedes its DPP read.
__device__ __forceinline__ void fmac_quad(float& acc, uint32_t q, float x, int i)
{
#define AMX_FMAC_DPP(I)                                                                                  \
    asm volatile("v_fmac_f32_dpp %0, %1, %2 quad_perm:[" #I "," #I "," #I "," #I "] row_mask:0xf bank_mask:0xf" \
                 : "+v"(acc) : "v"(q), "v"(x))
    switch (i) {
    case 0: AMX_FMAC_DPP(0); break;
    case 1: AMX_FMAC_DPP(1); break;
    case 2: AMX_FMAC_DPP(2); break;
    default: AMX_FMAC_DPP(3); break;
    }
#undef AMX_FMAC_DPP
}

// Column c's w (h = 0) or se (h = 1), in every lane.
__device__ __forceinline__ uint32_t col_word(const uint32_t (&q)[UQ], int c, int h)
{
    return quad_bcast(q[4 * (c >> 3) + 2 * (c & 1) + h], (c >> 1) & 3);
}

}  // namespace amx
