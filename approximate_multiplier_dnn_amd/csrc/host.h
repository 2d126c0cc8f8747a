// host.h -- the per-device and per-stream host state of api.cpp that the
// calls of layers.cpp share.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace amx {

// The multiplier selected on the current device.
struct HostTable {
    int dev = 0;
    int M = 0;                                 // 0: the native multiplier
    const uint16_t* lane_first = nullptr;      // attention images (attention.h)
    const uint16_t* uniform_first = nullptr;
    int elo = 1, ehi = 254;
    int force_checked = 0;
};

// APPROX_OK, or APPROX_ENOLUT / APPROX_EHIP.
int host_table(HostTable* t);

// The stream's scratch arena (after its statistics region).
int host_scratch(int dev, hipStream_t stream, size_t bytes, char** out);

// The stream's second scratch block, which GEMM calls leave alone.
int host_kept(int dev, hipStream_t stream, size_t bytes, char** out);

struct EpilogueParams;

// sums = X W as approx_gemm; *fused: the reduction ended in the epilogue
// (which is then done, and sums is not written).
int host_dense(int m, int n, int k, const float* X, int ldx, const float* W, int ldw, float* sums, int lds,
               const EpilogueParams& e, bool* fused, hipStream_t stream);

}  // namespace amx
