// Norm over many gradient tensors, and their scaling to a given largest norm.  Simplest
// form: one launch per tensor and phase; every workgroup adds its fp64 sum of squares
// into its own place, and the scaling workgroups add the places in order.
#include <stdint.h>

#include <algorithm>

#include "device_common.h"
#include "block_launch.h"

namespace ttt {
namespace {

constexpr int kParts = 1024;   // workgroups of a launch, and partial sums

__device__ __forceinline__ double block_sum(double x, double* lds)
{
    for (int o = 32; o; o >>= 1) x += __shfl_xor(x, o);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    return lds[0] + lds[1] + lds[2] + lds[3];
}

__global__ __launch_bounds__(256) void clip_clear_kernel(double* part)
{
    part[blockIdx.x * 256 + threadIdx.x] = 0.0;
}

template <typename TIO>
__global__ __launch_bounds__(256) void clip_square_kernel(const TIO* __restrict__ g, long long n,
                                                          double* part)
{
    __shared__ double lds[4];
    double s = 0.0;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += 256ll * gridDim.x) {
        const double v = io<TIO>::load(g, i);
        s = fma(v, v, s);
    }
    s = block_sum(s, lds);
    if (threadIdx.x == 0) part[blockIdx.x] += s;
}

__device__ __forceinline__ double total(const double* part, double* lds)
{
    double s = 0.0;
    for (int i = threadIdx.x; i < kParts; i += 256) s += part[i];
    return block_sum(s, lds);
}

__global__ __launch_bounds__(256) void clip_norm_kernel(const double* __restrict__ part,
                                                        float* __restrict__ norm)
{
    __shared__ double lds[4];
    const double t = total(part, lds);
    if (threadIdx.x == 0) *norm = (float)sqrt(t);
}

template <typename TIO>
__global__ __launch_bounds__(256) void clip_scale_kernel(const TIO* g, TIO* out, long long n,
                                                         const double* __restrict__ part,
                                                         float max_norm, float eps)
{
    __shared__ double lds[4];
    const double norm = sqrt(total(part, lds));
    const double q = (double)max_norm / (norm + (double)eps);
    const float f = q > 1.0 ? 1.f : (float)q;   // NaN stays one
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += 256ll * gridDim.x)
        io<TIO>::store(out, i, io<TIO>::load(g, i) * f);
}

unsigned grid_of(long long n) { return (unsigned)std::min<long long>(kParts, (n + 255) / 256); }

}  // namespace

size_t clip_workspace() { return kParts * sizeof(double); }

hipError_t launch_clip(const ClipArgs& a, hipStream_t s)
{
    double* part = (double*)a.workspace;
    const dim3 block(256);
    hipLaunchKernelGGL(clip_clear_kernel, dim3(kParts / 256), block, 0, s, part);
    for (int i = 0; i < a.n; ++i) {
        const long long n = a.sizes[i];
        if (!n) continue;
        if (a.dtypes[i])
            hipLaunchKernelGGL(clip_square_kernel<uint16_t>, dim3(grid_of(n)), block, 0, s,
                               (const uint16_t*)a.grads[i], n, part);
        else
            hipLaunchKernelGGL(clip_square_kernel<float>, dim3(grid_of(n)), block, 0, s,
                               (const float*)a.grads[i], n, part);
    }
    hipLaunchKernelGGL(clip_norm_kernel, dim3(1), block, 0, s, part, a.norm);
    for (int i = 0; a.outs && i < a.n; ++i) {
        const long long n = a.sizes[i];
        if (!n) continue;
        if (a.dtypes[i])
            hipLaunchKernelGGL(clip_scale_kernel<uint16_t>, dim3(grid_of(n)), block, 0, s,
                               (const uint16_t*)a.grads[i], (uint16_t*)a.outs[i], n, part,
                               a.max_norm, a.eps);
        else
            hipLaunchKernelGGL(clip_scale_kernel<float>, dim3(grid_of(n)), block, 0, s,
                               (const float*)a.grads[i], (float*)a.outs[i], n, part, a.max_norm,
                               a.eps);
    }
    return hipGetLastError();
}

}  // namespace ttt
