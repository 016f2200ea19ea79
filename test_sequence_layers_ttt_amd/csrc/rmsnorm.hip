// Root-mean-square norm with the residual's addition: forward in the I/O type or in
// e4m3 with one scale per row, and the backward pass.  Simplest form: one workgroup per
// row, the row read again for each pass over it.
#include <stdint.h>

#include "device_common.h"
#include "block_launch.h"

namespace ttt {
namespace {

constexpr float kE4m3Max = 448.f;

// sum over the 256 threads, the same bits in every thread
__device__ __forceinline__ float block_sum(float x, float* lds)
{
    for (int o = 32; o; o >>= 1) x += __shfl_xor(x, o);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    return lds[0] + lds[1] + lds[2] + lds[3];
}

// max with NaN winning
__device__ __forceinline__ float nan_max(float a, float b) { return a != a ? a : b != b ? b : fmaxf(a, b); }

__device__ __forceinline__ float block_max(float x, float* lds)
{
    for (int o = 32; o; o >>= 1) x = nan_max(x, __shfl_xor(x, o));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    return nan_max(nan_max(lds[0], lds[1]), nan_max(lds[2], lds[3]));
}

// y / scale as e4m3: a zero scale (a row of zeros) gives 0, a NaN stays one
__device__ __forceinline__ uint8_t to_e4m3(float y, float scale)
{
    float v = scale == 0.f ? 0.f : y / scale;
    v = v > kE4m3Max ? kE4m3Max : v < -kE4m3Max ? -kE4m3Max : v;
    return (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(v, v, 0, false);
}

template <typename TIO, bool Q8>
__global__ __launch_bounds__(256) void rms_fwd_kernel(const TIO* X, const TIO* residual,
                                                      const float* __restrict__ weight, float eps,
                                                      void* Y, float* scale, TIO* R, int D)
{
    __shared__ float lds[4];
    const size_t base = (size_t)blockIdx.x * D;
    auto r_at = [&](int i) {
        return io<TIO>::load(X, base + i) + (residual ? io<TIO>::load(residual, base + i) : 0.f);
    };
    float ss = 0.f;
    for (int i = threadIdx.x; i < D; i += 256) {
        const float r = r_at(i);
        ss = fmaf(r, r, ss);
    }
    const float k = rsqrtf(block_sum(ss, lds) / D + eps);
    float sc = 0.f;
    if constexpr (Q8) {
        float m = 0.f;
        for (int i = threadIdx.x; i < D; i += 256)
            m = nan_max(m, fabsf(r_at(i) * k * (weight ? weight[i] : 1.f)));
        sc = block_max(m, lds) / kE4m3Max;
        if (threadIdx.x == 0) scale[blockIdx.x] = sc;
    }
    for (int i = threadIdx.x; i < D; i += 256) {
        const float r = r_at(i);
        const float y = r * k * (weight ? weight[i] : 1.f);
        if constexpr (Q8) ((uint8_t*)Y)[base + i] = to_e4m3(y, sc);
        else io<TIO>::store((TIO*)Y, base + i, y);
        if (R) io<TIO>::store(R, base + i, r);
    }
}

template <typename TIO>
__global__ __launch_bounds__(256) void rms_bwd_kernel(const TIO* __restrict__ R,
                                                      const float* __restrict__ weight,
                                                      const TIO* dY, const TIO* dR, float eps,
                                                      TIO* dX, int D)
{
    __shared__ float lds[4];
    const size_t base = (size_t)blockIdx.x * D;
    float ss = 0.f, su = 0.f;
    for (int i = threadIdx.x; i < D; i += 256) {
        const float r = io<TIO>::load(R, base + i);
        ss = fmaf(r, r, ss);
        su = fmaf(io<TIO>::load(dY, base + i) * (weight ? weight[i] : 1.f), r, su);
    }
    const float k = rsqrtf(block_sum(ss, lds) / D + eps);
    const float m = block_sum(su, lds) * k / D;
    for (int i = threadIdx.x; i < D; i += 256) {
        const float n = io<TIO>::load(R, base + i) * k;
        const float u = io<TIO>::load(dY, base + i) * (weight ? weight[i] : 1.f);
        io<TIO>::store(dX, base + i, k * (u - n * m) + (dR ? io<TIO>::load(dR, base + i) : 0.f));
    }
}

// row rates 1 / sqrt(mean(r^2) + eps), for the columns' sums
template <typename TIO>
__global__ __launch_bounds__(256) void rms_rate_kernel(const TIO* __restrict__ R, float eps,
                                                       float* __restrict__ rate, int D)
{
    __shared__ float lds[4];
    const size_t base = (size_t)blockIdx.x * D;
    float ss = 0.f;
    for (int i = threadIdx.x; i < D; i += 256) {
        const float r = io<TIO>::load(R, base + i);
        ss = fmaf(r, r, ss);
    }
    const float k = rsqrtf(block_sum(ss, lds) / D + eps);
    if (threadIdx.x == 0) rate[blockIdx.x] = k;
}

template <typename TIO>
__global__ __launch_bounds__(256) void rms_dw_kernel(const TIO* __restrict__ R,
                                                     const TIO* __restrict__ dY,
                                                     const float* __restrict__ rate,
                                                     float* __restrict__ dweight, long long rows,
                                                     int D)
{
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= D) return;
    float s = 0.f;
    for (long long r = 0; r < rows; ++r)
        s = fmaf(io<TIO>::load(dY, r * D + i), io<TIO>::load(R, r * D + i) * rate[r], s);
    dweight[i] = s;
}

template <typename TIO>
hipError_t fwd_typed(const RmsArgs& a, hipStream_t s)
{
    const dim3 grid((unsigned)a.rows), block(256);
    if (a.scale)
        hipLaunchKernelGGL((rms_fwd_kernel<TIO, true>), grid, block, 0, s, (const TIO*)a.X,
                           (const TIO*)a.residual, a.weight, a.eps, a.Y, a.scale, (TIO*)a.R, a.D);
    else
        hipLaunchKernelGGL((rms_fwd_kernel<TIO, false>), grid, block, 0, s, (const TIO*)a.X,
                           (const TIO*)a.residual, a.weight, a.eps, a.Y, a.scale, (TIO*)a.R, a.D);
    return hipGetLastError();
}

template <typename TIO>
hipError_t bwd_typed(const RmsBwdArgs& a, hipStream_t s)
{
    const dim3 grid((unsigned)a.rows), block(256);
    const TIO *R = (const TIO*)a.R, *dY = (const TIO*)a.dY;
    float* rate = (float*)a.workspace;
    if (a.dweight) {   // first: dX may stand at dY's place
        if (a.rows)
            hipLaunchKernelGGL(rms_rate_kernel<TIO>, grid, block, 0, s, R, a.eps, rate, a.D);
        hipLaunchKernelGGL(rms_dw_kernel<TIO>, dim3((a.D + 255) / 256), block, 0, s, R, dY, rate,
                           a.dweight, a.rows, a.D);
    }
    if (a.rows)
        hipLaunchKernelGGL(rms_bwd_kernel<TIO>, grid, block, 0, s, R, a.weight, dY,
                           (const TIO*)a.dR, a.eps, (TIO*)a.dX, a.D);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm_fwd(const RmsArgs& a, hipStream_t s)
{
    return a.bf16 ? fwd_typed<uint16_t>(a, s) : fwd_typed<float>(a, s);
}

size_t rmsnorm_bwd_workspace(long long rows, int, bool) { return (size_t)rows * 4; }

hipError_t launch_rmsnorm_bwd(const RmsBwdArgs& a, hipStream_t s)
{
    return a.bf16 ? bwd_typed<uint16_t>(a, s) : bwd_typed<float>(a, s);
}

}  // namespace ttt
