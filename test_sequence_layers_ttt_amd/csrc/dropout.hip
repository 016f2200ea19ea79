// Dropout with the residual's addition: y = keep ? x * scale : 0, plus the residual.
//
// The generator is Philox 4x32 of 10 rounds (Salmon, Moraes, Dror, Shaw: Parallel Random
// Numbers: As Easy as 1, 2, 3; 2011): element i takes word i % 4 of the block whose counter
// is first + i / 4 and whose key is the seed, so the backward pass makes the same numbers
// again and no mask is kept.  Seed and counter are read from the device, so a captured
// graph draws anew when they change between its replays.  HBM bounds it: 33.5 M bf16 elements with
// the residual 36 us for 201 MB, 5.6 TB/s.
#include <algorithm>

#include "block_launch.h"
#include "device_common.h"
#include "mfma_common.h"

namespace ttt {
namespace {

typedef uint32_t quad __attribute__((ext_vector_type(4)));

__device__ __forceinline__ quad philox(uint64_t counter, uint32_t k0, uint32_t k1)
{
    uint32_t c0 = (uint32_t)counter, c1 = (uint32_t)(counter >> 32), c2 = 0u, c3 = 0u;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)0xD2511F53u * c0, b = (uint64_t)0xCD9E8D57u * c2;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
        c1 = (uint32_t)b;
        c3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return quad{c0, c1, c2, c3};
}

// 16 bytes a thread: two blocks of numbers for eight bf16 elements, one for four fp32
template <typename TIO, bool RES>
__global__ void __launch_bounds__(256) dropout_kernel(const TIO* X, const TIO* R, TIO* Y, long long n,
                                                      const long long* rng, uint32_t threshold, float scale)
{
    constexpr int V = 16 / (int)sizeof(TIO);
    const uint64_t seed = (uint64_t)rng[0], first = (uint64_t)rng[1];
    const uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
    const long long step = (long long)gridDim.x * 256, vectors = (n + V - 1) / V;
    for (long long v = (long long)blockIdx.x * 256 + threadIdx.x; v < vectors; v += step) {
        quad q[V / 4];
#pragma unroll
        for (int i = 0; i < V / 4; ++i) q[i] = philox(first + (uint64_t)v * (V / 4) + i, k0, k1);
        const long long at = v * V;
        if (at + V <= n) {
            const quad x = *reinterpret_cast<const quad*>(X + at);
            quad r = {0u, 0u, 0u, 0u}, y;
            if constexpr (RES) r = *reinterpret_cast<const quad*>(R + at);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(TIO) == 4) {
                    float f = q[0][i] >= threshold ? __uint_as_float(x[i]) * scale : 0.f;
                    if constexpr (RES) f += __uint_as_float(r[i]);
                    y[i] = __float_as_uint(f);
                } else {
                    float a = q[i / 2][2 * (i & 1)] >= threshold ? __uint_as_float(x[i] << 16) * scale : 0.f;
                    float b = q[i / 2][2 * (i & 1) + 1] >= threshold
                                  ? __uint_as_float(x[i] & 0xffff0000u) * scale : 0.f;
                    if constexpr (RES) {
                        a += __uint_as_float(r[i] << 16);
                        b += __uint_as_float(r[i] & 0xffff0000u);
                    }
                    y[i] = pack_bf16x2(a, b);
                }
            }
            *reinterpret_cast<quad*>(Y + at) = y;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (at + i < n) {
                    float f = q[i / 4][i & 3] >= threshold ? io<TIO>::load(X, at + i) * scale : 0.f;
                    if constexpr (RES) f += io<TIO>::load(R, at + i);
                    io<TIO>::store(Y, at + i, f);
                }
        }
    }
}

template <typename TIO>
hipError_t dropout_as(const DropoutArgs& a, hipStream_t s)
{
    constexpr int V = 16 / (int)sizeof(TIO);
    const long long blocks = ((a.n + V - 1) / V + 255) / 256;
    const unsigned grid = (unsigned)std::min<long long>(blocks, 1 << 20);
    if (a.residual)
        dropout_kernel<TIO, true><<<grid, 256, 0, s>>>((const TIO*)a.X, (const TIO*)a.residual, (TIO*)a.Y, a.n,
                                                      a.rng, a.threshold, a.scale);
    else
        dropout_kernel<TIO, false><<<grid, 256, 0, s>>>((const TIO*)a.X, nullptr, (TIO*)a.Y, a.n, a.rng,
                                                       a.threshold, a.scale);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs& a, hipStream_t s)
{
    return a.bf16 ? dropout_as<uint16_t>(a, s) : dropout_as<float>(a, s);
}

}  // namespace ttt
