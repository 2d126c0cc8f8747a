// dense.h -- parameter blocks and launchers of the dense layer's elementwise
// kernels (dense.hip). Not part of the C ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace amx {

enum Activation : int { ACT_NONE = 0, ACT_RELU, ACT_GELU, ACT_SILU, ACT_COUNT };

struct EpilogueParams {
    const float* sums;        // X W; may be z or y
    const float* bias;        // or null
    const float* residual;    // or null
    float* z;                 // or null
    float* y;
    int64_t lds, ldr, ldz, ldy;
    int m, n, act;
    int vec;                  // n and every leading dimension multiples of 4, every pointer 16-byte aligned
};
hipError_t launch_epilogue(const EpilogueParams& p, hipStream_t s);
// The reduction of a GEMM's chunk partials (launch_reduce; batch 1) that ends
// in the epilogue (`sums` is not read).
struct ReduceParams;
hipError_t launch_reduce_epilogue(const ReduceParams& p, const EpilogueParams& e, hipStream_t s);

struct DzParams {
    const float* dy;
    const float* z;           // null: dz = dy
    float* dz;                // [m][n], or null
    double* part;             // [chunks][n], or null
    int64_t lddy, ldz;
    int m, n, act;
    int rows;                 // rows per chunk
};
// dz, and (db not null) the bias gradient from its partials.
hipError_t launch_dz(const DzParams& p, float* db, hipStream_t s);

}  // namespace amx
