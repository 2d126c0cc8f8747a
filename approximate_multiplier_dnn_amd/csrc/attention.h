// attention.h -- parameter blocks and launchers of the attention and
// dense-layer kernels (attention.hip, dense.hip), shared with their host API
// (layers.cpp). Not part of the C ABI.
#pragma once
#include "internal.h"

namespace amx {

// The table image the attention kernels stage: 2^M columns of 2^M entries and
// two zero entries (the pad), one column per uniform operand's mantissa, rows
// by the lane operand's. Unlike the GEMM kernel's M = 8 image it holds no
// second copies: 132,096 bytes leave LDS for the kernels' own use.
__host__ __device__ inline int attn_col_bytes(int M) { return ((1 << M) + 2) * 2; }
__host__ __device__ inline int attn_image_bytes(int M) { return M ? (1 << M) * attn_col_bytes(M) : 0; }

// Where the table is read: staged in LDS (M <= 7, M = 8), from global memory
// (M = 9..11), or the native multiplier.
enum AttnTable : int { AT_LDS = 0, AT_LDS8, AT_GLOBAL, AT_NATIVE, AT_COUNT };
inline int attn_table_kind(int M) { return M == 0 ? AT_NATIVE : M <= 7 ? AT_LDS : M == 8 ? AT_LDS8 : AT_GLOBAL; }

constexpr int kAttnTile = 64;       // rows (one per lane) of a wave's item
constexpr int kAttnBlock = 16;      // columns a wave takes at a time (uniform operands)
constexpr int kAttnSlots = 512;     // decode workgroups per tensor, each with its exponent range
constexpr int kAttnMaxDim = 128;
constexpr int kAttnMaxSplits = 32;

// One decoded tensor, rows x D per kv head: row r of kv head h is token
// r / G, head h * G + r % G (G = 1 for keys and values). The panels
// of 8-byte Words:
//   lane: [K][D4 / 4][Rp][4]  rows across the lanes, reduction over D
//   tr:   [K][Rp / 16][D4][16]  16 rows as uniform columns, reduction over D
//   row:  [K][Dp / 16][Rp][16]  16 columns uniform, reduction over the rows
// with Rp the rows rounded up to 64, D4 and Dp the dimension rounded up to 4
// and 16; the padding holds zero operands.
struct AttnTensor {
    const float* src;
    int64_t ld;          // floats between tokens
    int R, G, Rp;
    FastDiv fd_G;
    int cache;           // 1: rows are keys in a paged cache, src its pages (AttnCache)
    Word* lane;
    Word* tr;
    Word* row;
};

// Keys of a paged cache laid out as packed keys: key j of sequence b is row
// b * stride + j (stride a multiple of 64), and bit i of mask[row / 16] says
// whether key 16 * (row / 16) + i has a page. Blocks of 64 rows past a
// sequence's keys are left out.
struct AttnCache {
    const int* k_len;
    const int* table;
    int table_ld, page, num_pages, stride;
    FastDiv fd_page, fd_stride;
    uint16_t* mask;
};

struct AttnDecodeParams {
    AttnTensor t[4];
    AttnCache cache;
    int count;
    int K, D, D4, Dp, M, elo, ehi;
    uint32_t* stats;     // [4][kAttnSlots]: min exponent | max exponent << 8 (255 for Inf and NaN)
    // backward: the tensors are q, dO, k, v (forward: q, k, v); delta[h][r] = RN32(sum_d dO o) and lse as [h][r]
    const float* o;
    int64_t ldo;
    const float* lse;    // [tokens][heads]
    float* delta;
    float* rowlse;
    int* next;           // two item counters to clear, or null
};

// Attention of packed sequences. cu_q / cu_k: device offsets (nseq + 1).
struct AttnParams {
    const int* cu_q;
    const int* cu_k;          // null: sequence b's keys are k_len[b] rows from b * k_stride on (AttnCache)
    const int* k_len;
    int k_stride, k_most;     // k_most: largest length
    const uint16_t* k_mask;   // or null
    int nseq, K, G, D, D4, Dp;
    int NW, TT;               // waves of a tile (Dp / 16); tiles of a workgroup (set by the launcher)
    int total_q, total_k, RQ, RQp, TKp;
    int causal;
    double c;                 // scale * log2(e)
    float scale;
    int M, elo, ehi, smax;    // smax: largest sum of q's and k's biased exponents of the fast path
    int force_checked;
    const uint16_t* lut;      // image of the kernel's operand order
    const uint32_t* stats;
    const Word *q_lane, *k_lane, *v_lane, *do_lane;
    const Word *q_tr, *k_tr, *v_tr, *do_tr;
    const Word *q_row, *k_row, *v_row, *do_row;
    const float* delta;
    const float* rowlse;
    int tiles, splits;        // row tiles (upper bound) per kv head; chunks of each tile's range
    int64_t items;            // set by the launcher
    int* next;                // item counter, cleared by the decode launch
    // outputs (token-major, ld floats between tokens)
    float *o, *lse, *dq, *dk, *dv;
    int64_t ldo, lddq, lddk, lddv;
    // partials (splits > 1)
    float* part0;             // [split][K][R][Dp]
    float* part1;
    double* part_m;           // [split][K][R]
    double* part_l;
};

// Chunks of rows to be joined (forward and paged).
struct AttnJoinParams {
    const int* cu_q;
    int nseq, K, G, D, Dp, total_q, RQ, splits;
    const float* part;        // [split][K][RQ][Dp]
    const double* part_m;     // [split][K][RQ]
    const double* part_l;
    float* o;
    int64_t ldo;
    float* lse;
};

// A chunk of new tokens per sequence over a paged cache.
struct PagedParams {
    const int* cu_q;
    const int* k_len;
    const int* table;         // [nseq][table_ld] page numbers
    const float* kp;          // [num_pages][page][K][D]
    const float* vp;
    const float* q;
    int64_t ldq;
    int nseq, K, G, D, D4, Dp, total_q, RQ;
    int page, num_pages, table_ld;
    FastDiv fd_page;
    int causal, vec;          // vec: 16-byte loads of the keys
    double c;
    int M, elo, ehi, smax;
    int force_checked;
    const uint16_t* lut;      // uniform operand first
    int NR;                   // rows of a block (4, 8 or 16)
    int blocks, splits, chunk;   // row blocks (upper bound) per kv head; chunks of `chunk` keys
    float *o, *lse;
    int64_t ldo;
    float* part0;
    double* part_m;
    double* part_l;
};

hipError_t launch_attn_decode(const AttnDecodeParams& p, hipStream_t s);
hipError_t launch_attn_fwd(const AttnParams& p, hipStream_t s);
// dQ, or (keys) dK and dV; p's tiles, splits, items, image and partials are
// those of that pass.
hipError_t launch_attn_bwd(const AttnParams& p, bool keys, hipStream_t s);
hipError_t launch_attn_paged(const PagedParams& p, hipStream_t s);

}  // namespace amx
