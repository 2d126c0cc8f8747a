// dense_device.h -- the dense layer's epilogue, shared by its own kernel
// (dense.hip) and the reductions that end in it (kernels.hip).
#pragma once
#include "dense.h"

namespace amx {

// Activations on FP32 (forward): Phi(z) = erfc(-z / sqrt 2) / 2 keeps its
// relative accuracy for negative z, where 1 + erf cancels.
__device__ __forceinline__ float activate(float z, int act)
{
    switch (act) {
    case ACT_RELU: return z < 0.0f ? 0.0f : z;                  // NaN stays
    case ACT_GELU: return 0.5f * z * erfcf(z * -0.70710678118654752f);
    case ACT_SILU: return z / (1.0f + expf(-z));
    default: return z;
    }
}

// Output (i, j) from its sum: bias, activation, residual.
__device__ __forceinline__ void finish_output(const EpilogueParams& p, int64_t i, int64_t j, float z)
{
    if (p.bias != nullptr) z += p.bias[j];
    if (p.z != nullptr) p.z[i * p.ldz + j] = z;
    z = activate(z, p.act);
    if (p.residual != nullptr) z += p.residual[i * p.ldr + j];
    p.y[i * p.ldy + j] = z;
}

}  // namespace amx
