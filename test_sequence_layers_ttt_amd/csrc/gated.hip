// Gated linear recurrence: h_t = exp(g_t) h_{t-1} + x_t per channel, and its backward
// pass.  Simplest form: one thread per (row, feature), serial over the tokens.
#include <stdint.h>

#include <cmath>

#include "device_common.h"
#include "block_launch.h"

namespace ttt {
namespace {

// exp(g) h, with a gate of -inf passing nothing on (infinities and NaN included)
__device__ __forceinline__ float decay(float g, float h)
{
    return g == -INFINITY ? 0.f : expf(g) * h;
}

template <typename TIO>
__global__ __launch_bounds__(256) void gated_fwd_kernel(const TIO* __restrict__ X,
                                                        const TIO* __restrict__ G, const float* h0,
                                                        TIO* __restrict__ Z, float* h_out,
                                                        long long channels, int T, int d)
{
    const long long c = (long long)blockIdx.x * 256 + threadIdx.x;
    if (c >= channels) return;
    const size_t row = c / d, f = c - row * d;
    float h = h0 ? h0[c] : 0.f;
    size_t i = row * T * d + f;
    for (int t = 0; t < T; ++t, i += d) {
        h = decay(io<TIO>::load(G, i), h) + io<TIO>::load(X, i);
        io<TIO>::store(Z, i, h);
    }
    if (h_out) h_out[c] = h;
}

template <typename TIO>
__global__ __launch_bounds__(256) void gated_bwd_kernel(
    const TIO* __restrict__ G, const TIO* __restrict__ Z, const float* __restrict__ h0,
    const TIO* __restrict__ dZ, const float* __restrict__ dh_T, TIO* __restrict__ dX,
    TIO* __restrict__ dG, float* __restrict__ dh0, long long channels, int T, int d)
{
    const long long c = (long long)blockIdx.x * 256 + threadIdx.x;
    if (c >= channels) return;
    const size_t row = c / d, f = c - row * d, base = row * T * d + f;
    float carry = dh_T ? dh_T[c] : 0.f;   // exp(g_{t+1}) lambda_{t+1}
    for (int t = T - 1; t >= 0; --t) {
        const size_t i = base + (size_t)t * d;
        const float lam = io<TIO>::load(dZ, i) + carry;
        const float before = t > 0 ? io<TIO>::load(Z, i - d) : (h0 ? h0[c] : 0.f);
        const float g = io<TIO>::load(G, i);
        carry = decay(g, lam);
        io<TIO>::store(dX, i, lam);
        io<TIO>::store(dG, i, g == -INFINITY ? 0.f : carry * before);
    }
    if (dh0) dh0[c] = carry;
}

unsigned blocks(long long channels) { return (unsigned)((channels + 255) / 256); }

}  // namespace

size_t gated_workspace(int, int, int, bool) { return 0; }

hipError_t launch_gated_fwd(const GatedArgs& a, hipStream_t s)
{
    const long long n = (long long)a.BH * a.d;
    if (a.bf16)
        hipLaunchKernelGGL(gated_fwd_kernel<uint16_t>, dim3(blocks(n)), dim3(256), 0, s,
                           (const uint16_t*)a.X, (const uint16_t*)a.G, a.h0, (uint16_t*)a.Z,
                           a.h_out, n, a.T, a.d);
    else
        hipLaunchKernelGGL(gated_fwd_kernel<float>, dim3(blocks(n)), dim3(256), 0, s,
                           (const float*)a.X, (const float*)a.G, a.h0, (float*)a.Z, a.h_out, n,
                           a.T, a.d);
    return hipGetLastError();
}

hipError_t launch_gated_step(const GatedArgs& a, hipStream_t s) { return launch_gated_fwd(a, s); }

hipError_t launch_gated_bwd(const GatedBwdArgs& a, hipStream_t s)
{
    const long long n = (long long)a.BH * a.d;
    if (a.bf16)
        hipLaunchKernelGGL(gated_bwd_kernel<uint16_t>, dim3(blocks(n)), dim3(256), 0, s,
                           (const uint16_t*)a.G, (const uint16_t*)a.Z, a.h0,
                           (const uint16_t*)a.dZ, a.dh_T, (uint16_t*)a.dX, (uint16_t*)a.dG, a.dh0,
                           n, a.T, a.d);
    else
        hipLaunchKernelGGL(gated_bwd_kernel<float>, dim3(blocks(n)), dim3(256), 0, s,
                           (const float*)a.G, (const float*)a.Z, a.h0, (const float*)a.dZ, a.dh_T,
                           (float*)a.dX, (float*)a.dG, a.dh0, n, a.T, a.d);
    return hipGetLastError();
}

}  // namespace ttt
