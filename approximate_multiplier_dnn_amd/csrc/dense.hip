// dense.hip -- elementwise kernels of the dense layer: the forward epilogue
// (bias, activation, residual) and the backward pass's dz = dy act'(z) with
// the bias gradient. The products run in kernels.hip.
#include <algorithm>

#include "dense_device.h"

namespace amx {

// Derivatives in 64 bits: dz enters the multiplier's table, which cuts it at M
// bits, so it is rounded once (an error of one last place next to such a
// border would move its products by 2^-M).
__device__ __forceinline__ double slope(double z, int act)
{
    switch (act) {
    case ACT_RELU: return z > 0.0 ? 1.0 : 0.0;
    case ACT_GELU: return 0.5 * erfc(z * -0.70710678118654752440) + z * exp(-0.5 * z * z) * 0.39894228040143267794;
    case ACT_SILU: {
        const double s = 1.0 / (1.0 + exp(-z));
        return s * (1.0 + z * (1.0 - s));
    }
    default: return 1.0;
    }
}

// z = sums + bias; y = act(z) + residual, four columns per thread where rows
// are 16-byte aligned. Bound by HBM.
__global__ __launch_bounds__(256) void epilogue_kernel(EpilogueParams p)
{
    const int per = p.vec ? p.n / 4 : p.n;
    const int64_t total = (int64_t)p.m * per;
    for (int64_t g = blockIdx.x * 256LL + threadIdx.x; g < total; g += (int64_t)gridDim.x * 256) {
        const int64_t i = g / per;
        const int j = (int)(g - i * per);
        if (p.vec) {
            float4 z = reinterpret_cast<const float4*>(p.sums + i * p.lds)[j];
            if (p.bias != nullptr) {
                const float4 b = reinterpret_cast<const float4*>(p.bias)[j];
                z.x += b.x; z.y += b.y; z.z += b.z; z.w += b.w;
            }
            if (p.z != nullptr) reinterpret_cast<float4*>(p.z + i * p.ldz)[j] = z;
            z.x = activate(z.x, p.act); z.y = activate(z.y, p.act); z.z = activate(z.z, p.act); z.w = activate(z.w, p.act);
            if (p.residual != nullptr) {
                const float4 r = reinterpret_cast<const float4*>(p.residual + i * p.ldr)[j];
                z.x += r.x; z.y += r.y; z.z += r.z; z.w += r.w;
            }
            reinterpret_cast<float4*>(p.y + i * p.ldy)[j] = z;
        } else {
            finish_output(p, i, j, p.sums[i * p.lds + j]);
        }
    }
}

// dz = RN32(dy act'(z)) for a block of 64 columns and a chunk of rows, four
// rows of threads; the bias gradient's part of the chunk is summed in 64 bits
// and left in part[chunk][n] (a second launch adds the chunks in order).
__global__ __launch_bounds__(256) void dz_kernel(DzParams p)
{
    __shared__ double sums[3][64];
    const int c = threadIdx.x & 63, w = threadIdx.x >> 6, j = blockIdx.x * 64 + c;
    const int i0 = blockIdx.y * p.rows, i1 = min(p.m, i0 + p.rows);
    double sum = 0.0;
    if (j < p.n)
        for (int i = i0 + w; i < i1; i += 4) {
            const float dy = p.dy[(int64_t)i * p.lddy + j];
            const float dz = p.z == nullptr ? dy : (float)((double)dy * slope((double)p.z[(int64_t)i * p.ldz + j], p.act));
            if (p.dz != nullptr) p.dz[(int64_t)i * p.n + j] = dz;
            sum += (double)dz;
        }
    if (p.part == nullptr) return;
    if (w > 0) sums[w - 1][c] = sum;
    __syncthreads();
    if (w == 0 && j < p.n) p.part[(int64_t)blockIdx.y * p.n + j] = sum + sums[0][c] + sums[1][c] + sums[2][c];
}

__global__ __launch_bounds__(64) void db_kernel(const double* part, float* db, int n, int chunks)
{
    const int j = blockIdx.x * 64 + threadIdx.x;
    if (j >= n) return;
    double sum = 0.0;
#pragma unroll 8
    for (int c = 0; c < chunks; ++c) sum += part[(int64_t)c * n + j];
    db[j] = (float)sum;
}

hipError_t launch_epilogue(const EpilogueParams& p, hipStream_t s)
{
    const int64_t total = (int64_t)p.m * (p.vec ? p.n / 4 : p.n);
    epilogue_kernel<<<(unsigned)std::min<int64_t>((total + 255) / 256, 256 * 16), 256, 0, s>>>(p);
    return hipGetLastError();
}

hipError_t launch_dz(const DzParams& p, float* db, hipStream_t s)
{
    const int chunks = std::max(1, (p.m + p.rows - 1) / p.rows);      // no row: db = 0
    dz_kernel<<<dim3((p.n + 63) / 64, chunks), 256, 0, s>>>(p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || db == nullptr) return e;
    db_kernel<<<(p.n + 63) / 64, 64, 0, s>>>(p.part, db, p.n, chunks);
    return hipGetLastError();
}

}  // namespace amx
