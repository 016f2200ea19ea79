// Root-mean-square norm with the residual's addition: forward in the I/O type or in e4m3
// with one scale per row, and the backward pass.
//
// A row of D features is held in registers by TPR threads, K vectors of 16 bytes each, so
// every input is read once and every output written once: HBM bounds it (32768 x 2048
// bf16 backward 99 us for 537 MB, 5.4 TB/s; 16384 x 2048 to e4m3 43 us for 235 MB; a
// device copy reaches 5.2 TB/s).  Rows of up to 128 vectors stay within one wave (sums by
// lane exchanges, no LDS, no barrier); longer ones take a workgroup: 256 threads with one
// vector each beat one wave with four (16384 x 2048 to e4m3: 45 and 92 us), which had too
// few loads under way.  A last vector that would pass the row's end starts early enough
// to be whole: what it shares with the one before is left out of the sums and written
// twice, with the same bits.  (All of a row's loads come before its first store, so
// outputs may stand at their inputs' places.)
//
// dweight sums over the rows: each thread adds up its own columns over its workgroup's
// rows, a wave's threads of one column are added by lane exchanges and the waves in LDS,
// and a second kernel (4.7 us for 1024 planes of 2048) adds the workgroups' planes, all in
// a fixed order.
#include <stdint.h>

#include <algorithm>

#include "block_launch.h"
#include "device_common.h"
#include "mfma_common.h"

namespace ttt {
namespace {

constexpr float kE4m3Max = 448.f;

typedef uint32_t quad __attribute__((ext_vector_type(4)));
typedef quad quad_any __attribute__((aligned(2)));

template <typename TIO> constexpr int kVec = 16 / (int)sizeof(TIO);

// 16 bytes of the I/O type at any element-aligned address; with the streaming policy where rows are
// whole cache lines (LINES: 8192 x 4096 fp32 backward 96 us, against 106 without), without it where a
// line takes several accesses, which then meet in the caches (200000 x 50 bf16 forward 8.7 us,
// against 13.2)
template <bool LINES, typename TIO>
__device__ __forceinline__ quad load16(const TIO* p)
{
    auto from = reinterpret_cast<const quad_any*>(p);
    return LINES ? __builtin_nontemporal_load(from) : *from;
}

template <bool LINES, typename TIO>
__device__ __forceinline__ void store16(TIO* p, quad q)
{
    auto to = reinterpret_cast<quad_any*>(p);
    if constexpr (LINES) __builtin_nontemporal_store(q, to);
    else *to = q;
}

template <typename TIO>
__device__ __forceinline__ void widen(quad q, float (&v)[kVec<TIO>])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(TIO) == 4) {
            v[i] = __uint_as_float(q[i]);
        } else {
            v[2 * i] = __uint_as_float(q[i] << 16);
            v[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
        }
    }
}

template <typename TIO>
__device__ __forceinline__ quad narrow(const float (&v)[kVec<TIO>])
{
    quad q;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(TIO) == 4) q[i] = __float_as_uint(v[i]);
        else q[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    }
    return q;
}

// what lane ^ (16 or 32) has, next to the lane's own, as (lower half's, upper half's)
template <int O>
__device__ __forceinline__ void halves(unsigned x, unsigned& lo, unsigned& hi)
{
    static_assert(O == 16 || O == 32, "");
    if constexpr (O == 16) {
        const auto p = __builtin_amdgcn_permlane16_swap(x, x, false, false);
        lo = p[0];
        hi = p[1];
    } else {
        const auto p = __builtin_amdgcn_permlane32_swap(x, x, false, false);
        lo = p[0];
        hi = p[1];
    }
}

template <int CTRL>
__device__ __forceinline__ unsigned moved(unsigned x)
{
    return (unsigned)__builtin_amdgcn_mov_dpp((int)x, CTRL, 0xF, 0xF, false);
}

// reduction over W <= 64 neighbouring lanes, the same bits in each: `f` is symmetric
template <int W, typename F>
__device__ __forceinline__ unsigned over_lanes(unsigned x, F&& f)
{
    if constexpr (W > 1) x = f(x, moved<kDppQuadXor1>(x));
    if constexpr (W > 2) x = f(x, moved<kDppQuadXor2>(x));
    if constexpr (W > 4) x = f(x, moved<kDppRowHalfMirror>(x));
    if constexpr (W > 8) x = f(x, moved<kDppRowMirror>(x));
    unsigned lo, hi;
    if constexpr (W > 16) {
        halves<16>(x, lo, hi);
        x = f(lo, hi);
    }
    if constexpr (W > 32) {
        halves<32>(x, lo, hi);
        x = f(lo, hi);
    }
    return x;
}

__device__ __forceinline__ unsigned add_bits(unsigned a, unsigned b)
{
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
}

// magnitudes compared as their bits: a NaN is above everything
__device__ __forceinline__ unsigned max_bits(unsigned a, unsigned b) { return a > b ? a : b; }

// N sums (or maxima of magnitudes) over the TPR threads of a row, the same bits in each; `lds`
// holds N words per wave where a row takes several
template <int TPR, int N, bool MAX>
__device__ __forceinline__ void over_row(unsigned (&x)[N], unsigned* lds)
{
    constexpr int W = TPR < 64 ? TPR : 64, WAVES = TPR / 64;
#pragma unroll
    for (int n = 0; n < N; ++n) x[n] = over_lanes<W>(x[n], MAX ? max_bits : add_bits);
    if constexpr (TPR > 64) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int n = 0; n < N; ++n) lds[n * WAVES + (threadIdx.x >> 6)] = x[n];
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            x[n] = lds[n * WAVES];
#pragma unroll
            for (int i = 1; i < WAVES; ++i)
                x[n] = (MAX ? max_bits : add_bits)(x[n], lds[n * WAVES + i]);
        }
    }
}

template <int TPR>
__device__ __forceinline__ float row_sum(float x, unsigned* lds)
{
    unsigned b[1] = {__float_as_uint(x)};
    over_row<TPR, 1, false>(b, lds);
    return __uint_as_float(b[0]);
}

template <int TPR>
__device__ __forceinline__ float row_max(unsigned x, unsigned* lds)
{
    unsigned b[1] = {x};
    over_row<TPR, 1, true>(b, lds);
    return __uint_as_float(b[0]);
}

__device__ __forceinline__ unsigned magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// four values as e4m3, rounded to nearest even (up to 464 in magnitude that is 448; NaN stays)
__device__ __forceinline__ unsigned pack_e4m3(float a, float b, float c, float d)
{
    const int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}

// A row's e4m3 values.  y / scale is t / (max|t| / 448) with t = r * weight * (the rate's power of
// two, which is exact): the rest of the rate cancels, and with it its error; the quotient's remainder
// is put right, so that what e4m3 rounds is off by little more than t's own rounding (at most 448 and
// a rounding of that).  Where the divisor or its reciprocal would leave fp32's range both are scaled by
// a power of two first; a scale of 0 (a row of zeros) gives 0; a NaN or an infinity in the row makes
// it NaN throughout.
struct Row8 {
    float scale, top, inv, by;
    bool rare;
    // the power of two in a rate (1 for a rate of 0, as of a row whose squares leave fp32's range)
    __device__ __forceinline__ static float power(float rate)
    {
        return rate == 0.f ? 1.f : __uint_as_float(__float_as_uint(rate) & 0x7f800000u);
    }
    __device__ __forceinline__ Row8(float most, float rate)
    {
        scale = most * (rate / power(rate)) / kE4m3Max;
        by = scale == 0.f ? 0.f : most < 1e-30f ? 0x1p80f : most > 1e30f ? 0x1p-80f : 1.f;
        rare = by != 1.f;
        top = scale == 0.f ? 1.f : most * by / kE4m3Max;
        inv = 1.f / top;
    }
    template <int V>
    __device__ __forceinline__ void apply(float (&t)[V]) const
    {
        if (rare)
#pragma unroll
            for (int i = 0; i < V; ++i) t[i] *= by;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float q = t[i] * inv;
            t[i] = fmaf(fmaf(-q, top, t[i]), inv, q);
        }
    }
};

// threads of a workgroup
template <int TPR> constexpr int kBlock = TPR < 256 ? 256 : TPR;
// rows a thread has under way at once
template <int TPR, int K> constexpr int kRows = TPR <= 64 && K == 1 ? 2 : 1;

template <typename TIO, int TPR, int K, bool Q8, bool LINES>
__global__ __launch_bounds__(kBlock<TPR>) void rms_fwd_kernel(
    const TIO* X, const TIO* residual, const float* __restrict__ weight, float eps, void* Y,
    float* scale, TIO* R, long long rows, int D)
{
    constexpr int V = kVec<TIO>, U = kRows<TPR, K>, GROUPS = kBlock<TPR> / TPR;
    __shared__ unsigned lds[TPR > 64 ? TPR / 64 : 1];
    const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR;
    const int vectors = (D + V - 1) / V;
    int col[K], dup[K];        // first column of each vector, and how many the one before has
    float w[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int v = lane + k * TPR;
        col[k] = min(v * V, D - V);
        dup[k] = v < vectors ? v * V - col[k] : V;
#pragma unroll
        for (int i = 0; i < V; ++i) w[k][i] = weight && dup[k] < V ? weight[col[k] + i] : 1.f;
    }
    const float inv_d = 1.f / D;
    for (long long r0 = ((long long)blockIdx.x * GROUPS + group) * U; r0 - group * U < rows;
         r0 += (long long)gridDim.x * GROUPS * U) {
        quad x[U][K], z[U][K];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < K; ++k) {
                x[u][k] = z[u][k] = quad{0, 0, 0, 0};
                if (r0 + u < rows && dup[k] < V) {
                    const size_t at = (size_t)(r0 + u) * D + col[k];
                    x[u][k] = load16<LINES>(X + at);
                    if (residual) z[u][k] = load16<LINES>(residual + at);
                }
            }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float r[K][V], ss = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float a[V];
                widen<TIO>(x[u][k], r[k]);
                if (residual) {
                    widen<TIO>(z[u][k], a);
#pragma unroll
                    for (int i = 0; i < V; ++i) r[k][i] += a[i];
                }
                if (dup[k] == 0) {
#pragma unroll
                    for (int i = 0; i < V; ++i) ss = fmaf(r[k][i], r[k][i], ss);
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i) ss = i >= dup[k] ? fmaf(r[k][i], r[k][i], ss) : ss;
                }
            }
            const float rate = rsqrtf(row_sum<TPR>(ss, lds) * inv_d + eps);
            const float by = Q8 ? Row8::power(rate) : rate;
            const bool live = r0 + u < rows;
            unsigned m = 0;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const bool mine = live && dup[k] < V;
                const size_t at = (size_t)(r0 + u) * D + col[k];
                if (R && mine) store16<LINES>(R + at, narrow<TIO>(r[k]));
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    r[k][i] *= by * w[k][i];
                    if constexpr (Q8) m = max_bits(m, magnitude(r[k][i]));
                }
                if constexpr (!Q8)
                    if (mine) store16<LINES>((TIO*)Y + at, narrow<TIO>(r[k]));
            }
            if constexpr (Q8) {
                const Row8 row(row_max<TPR>(m, lds), rate);
                if (live && lane == 0) scale[r0 + u] = row.scale;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    if (!live || dup[k] == V) continue;
                    row.apply(r[k]);
                    unsigned q[V / 4];
#pragma unroll
                    for (int i = 0; i < V / 4; ++i)
                        q[i] = pack_e4m3(r[k][4 * i], r[k][4 * i + 1], r[k][4 * i + 2], r[k][4 * i + 3]);
                    __builtin_memcpy((uint8_t*)Y + (size_t)(r0 + u) * D + col[k], q, V);
                }
            }
        }
    }
}

// Rows too long (or too short) for the registers' layout: a workgroup per row, the row read again
// for every pass.
template <typename TIO, bool Q8>
__global__ __launch_bounds__(256) void rms_fwd_loop_kernel(const TIO* X, const TIO* residual,
                                                           const float* __restrict__ weight,
                                                           float eps, void* Y, float* scale, TIO* R,
                                                           long long rows, int D)
{
    __shared__ unsigned lds[4];
    for (long long row = blockIdx.x; row < rows; row += gridDim.x) {
        const size_t base = (size_t)row * D;
        auto r_at = [&](int i) {
            const float x = io<TIO>::load(X, base + i);
            return residual ? x + io<TIO>::load(residual, base + i) : x;
        };
        float ss = 0.f;
        for (int i = threadIdx.x; i < D; i += 256) {
            const float r = r_at(i);
            ss = fmaf(r, r, ss);
        }
        const float rate = rsqrtf(row_sum<256>(ss, lds) / D + eps);
        const float by = Q8 ? Row8::power(rate) : rate;
        float most = 0.f;
        if constexpr (Q8) {
            unsigned m = 0;
            for (int i = threadIdx.x; i < D; i += 256)
                m = max_bits(m, magnitude(r_at(i) * (by * (weight ? weight[i] : 1.f))));
            most = row_max<256>(m, lds);
        }
        const Row8 row8(most, rate);
        if (Q8 && threadIdx.x == 0) scale[row] = row8.scale;
        for (int i = threadIdx.x; i < D; i += 256) {
            const float r = r_at(i), y = r * (by * (weight ? weight[i] : 1.f));
            if constexpr (Q8) {
                float t[1] = {y};
                row8.apply(t);
                ((uint8_t*)Y)[base + i] = (uint8_t)pack_e4m3(t[0], 0.f, 0.f, 0.f);
            } else
                io<TIO>::store((TIO*)Y, base + i, y);
            if (R) io<TIO>::store(R, base + i, r);
        }
    }
}

template <typename TIO, int TPR, int K, bool LINES>
__global__ __launch_bounds__(kBlock<TPR>) void rms_bwd_kernel(
    const TIO* __restrict__ R, const float* __restrict__ weight, const TIO* dY, const TIO* dR,
    float eps, TIO* dX, float* __restrict__ plane, long long rows, int D)
{
    constexpr int V = kVec<TIO>, GROUPS = kBlock<TPR> / TPR;
    __shared__ unsigned lds[TPR > 64 ? 2 * (TPR / 64) : 1];
    const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR;
    const int vectors = (D + V - 1) / V;
    int col[K], dup[K];
    float w[K][V], dw[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int v = lane + k * TPR;
        col[k] = min(v * V, D - V);
        dup[k] = v < vectors ? v * V - col[k] : V;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            w[k][i] = weight && dup[k] < V ? weight[col[k] + i] : 1.f;
            dw[k][i] = 0.f;
        }
    }
    const float inv_d = 1.f / D;
    for (long long row = (long long)blockIdx.x * GROUPS + group; row - group < rows;
         row += (long long)gridDim.x * GROUPS) {
        const bool live = row < rows;
        quad r[K], y[K], e[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            r[k] = y[k] = e[k] = quad{0, 0, 0, 0};
            if (live && dup[k] < V) {
                const size_t at = (size_t)row * D + col[k];
                r[k] = load16<LINES>(R + at);
                y[k] = load16<LINES>(dY + at);
                if (dR) e[k] = load16<LINES>(dR + at);
            }
        }
        float ss = 0.f, su = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float rv[V], yv[V];
            widen<TIO>(r[k], rv);
            widen<TIO>(y[k], yv);
            if (dup[k] == 0) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    ss = fmaf(rv[i], rv[i], ss);
                    su = fmaf(yv[i] * w[k][i], rv[i], su);
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    ss = i >= dup[k] ? fmaf(rv[i], rv[i], ss) : ss;
                    su = i >= dup[k] ? fmaf(yv[i] * w[k][i], rv[i], su) : su;
                }
            }
        }
        unsigned both[2] = {__float_as_uint(ss), __float_as_uint(su)};
        over_row<TPR, 2, false>(both, lds);
        const float rate = rsqrtf(__uint_as_float(both[0]) * inv_d + eps);
        const float m = __uint_as_float(both[1]) * rate * inv_d;   // mean(u n)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            // (widened again from the words: the first pass's values would take as many
            // registers as all the rest)
            asm volatile("" : "+v"(r[k]), "+v"(y[k]));
            float rv[V], yv[V], ev[V];
            widen<TIO>(r[k], rv);
            widen<TIO>(y[k], yv);
            widen<TIO>(e[k], ev);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float n = rv[i] * rate;
                dw[k][i] = live ? fmaf(yv[i], n, dw[k][i]) : dw[k][i];
                rv[i] = fmaf(rate, yv[i] * w[k][i] - n * m, ev[i]);
            }
            if (live && dup[k] < V) store16<LINES>(dX + (size_t)row * D + col[k], narrow<TIO>(rv));
        }
    }
    if (!plane) return;
    float* out = plane + (size_t)blockIdx.x * D;
    if constexpr (GROUPS > 1) {
        // each column slot over the wave's groups, then over the waves
        constexpr int SLOTS = TPR * K * V, WAVES = kBlock<TPR> / 64;
        __shared__ float part[WAVES * SLOTS];
        const int wave = threadIdx.x >> 6;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) {
#pragma unroll
                for (int o = TPR; o < 64; o <<= 1) dw[k][i] += __shfl_xor(dw[k][i], o);
                if ((threadIdx.x & 63) < TPR) part[wave * SLOTS + (k * TPR + lane) * V + i] = dw[k][i];
            }
        __syncthreads();
        for (int c = threadIdx.x; c < SLOTS; c += kBlock<TPR>) {
            const int v = c / V, i = c % V, c0 = min(v * V, D - V);
            if (v >= vectors || i < v * V - c0) continue;
            float sum = part[c];
#pragma unroll
            for (int g = 1; g < WAVES; ++g) sum += part[g * SLOTS + c];
            out[c0 + i] = sum;
        }
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i >= dup[k]) out[col[k] + i] = dw[k][i];
    }
}

// the same, a workgroup per row at a time, for the rows of rms_fwd_loop_kernel: each thread keeps
// its columns' sums in the plane
template <typename TIO>
__global__ __launch_bounds__(256) void rms_bwd_loop_kernel(
    const TIO* __restrict__ R, const float* __restrict__ weight, const TIO* dY, const TIO* dR,
    float eps, TIO* dX, float* __restrict__ plane, long long rows, int D)
{
    __shared__ unsigned lds[4];
    if (plane)
        for (int i = threadIdx.x; i < D; i += 256) plane[(size_t)blockIdx.x * D + i] = 0.f;
    for (long long row = blockIdx.x; row < rows; row += gridDim.x) {
        const size_t base = (size_t)row * D;
        float ss = 0.f, su = 0.f;
        for (int i = threadIdx.x; i < D; i += 256) {
            const float r = io<TIO>::load(R, base + i);
            ss = fmaf(r, r, ss);
            su = fmaf(io<TIO>::load(dY, base + i) * (weight ? weight[i] : 1.f), r, su);
        }
        const float rate = rsqrtf(row_sum<256>(ss, lds) / D + eps);
        const float m = row_sum<256>(su, lds) * rate / D;
        for (int i = threadIdx.x; i < D; i += 256) {
            const float n = io<TIO>::load(R, base + i) * rate, dy = io<TIO>::load(dY, base + i);
            if (plane) plane[(size_t)blockIdx.x * D + i] += dy * n;
            const float u = dy * (weight ? weight[i] : 1.f);
            io<TIO>::store(dX, base + i,
                           fmaf(rate, u - n * m, dR ? io<TIO>::load(dR, base + i) : 0.f));
        }
    }
}

// dweight: 32 columns a workgroup, the planes dealt out to 32 threads of each column
__global__ __launch_bounds__(1024) void rms_planes_kernel(const float* __restrict__ plane,
                                                          float* __restrict__ dweight, int planes,
                                                          int D)
{
    __shared__ float part[32][33];
    const int c = threadIdx.x & 31, p = threadIdx.x >> 5, i = blockIdx.x * 32 + c;
    float s = 0.f;
    if (i < D) {
#pragma unroll 8
        for (int k = p; k < planes; k += 32) s += plane[(size_t)k * D + i];
    }
    part[p][c] = s;
    __syncthreads();
    if (p == 0 && i < D) {
#pragma unroll
        for (int k = 1; k < 32; ++k) s += part[k][c];
        dweight[i] = s;
    }
}

// how a row lies in registers: threads and vectors of each; 0 threads: not at all
struct Shape { int tpr, k; };

Shape shape_of(int D, int vec)
{
    const int n = (D + vec - 1) / vec;
    if (D < vec || n > 4096) return {0, 0};
    if (n <= 64) return {n <= 2 ? 2 : n <= 4 ? 4 : n <= 8 ? 8 : n <= 16 ? 16 : n <= 32 ? 32 : 64, 1};
    if (n <= 128) return {64, 2};
    if (n <= 1024) return {256, n <= 256 ? 1 : n <= 512 ? 2 : 4};
    return {n <= 2048 ? 512 : 1024, 4};
}

// Workgroups of a launch: 1024 threads a compute unit, each with many rows, as each loads the weight
// (16384 x 2048 bf16 to e4m3: 45.0 us with twice as many, 41.2 with these).
template <int TPR> constexpr long long kMostBlocks = 256 * (1024 / kBlock<TPR>);

// The backward pass holds weight and dweight in fp32 next to three inputs: past 2048 vectors there
// are no registers for that.
Shape bwd_shape_of(int D, int vec)
{
    const Shape s = shape_of(D, vec);
    return s.tpr == 1024 ? Shape{0, 0} : s;
}

// Its workgroups, each with a plane of dweight: half of what the forward pass has where a thread
// holds several vectors, as planes cost twice their size (8192 x 4096 bf16: 52.7 us, 60.5 with all;
// 200000 x 100: 35.8 with half, 34.3 with all).
int planes_of(long long rows, int D, int vec)
{
    const Shape s = bwd_shape_of(D, vec);
    const int block = std::max(256, s.tpr), groups = s.tpr ? block / s.tpr : 1;
    const long long most = 256 * (1024 / block) / (s.k > 1 ? 2 : 1);
    return (int)std::max(1ll, std::min<long long>((rows + groups - 1) / groups, most));
}

template <typename TIO, int TPR, int K, bool LINES>
void fwd_launch(const RmsArgs& a, hipStream_t s)
{
    constexpr int PER = kBlock<TPR> / TPR * kRows<TPR, K>;
    const dim3 grid((unsigned)std::min(kMostBlocks<TPR>, (a.rows + PER - 1) / PER)), block(kBlock<TPR>);
    auto kernel = a.scale ? rms_fwd_kernel<TIO, TPR, K, true, LINES>
                          : rms_fwd_kernel<TIO, TPR, K, false, LINES>;
    hipLaunchKernelGGL(kernel, grid, block, 0, s, (const TIO*)a.X, (const TIO*)a.residual, a.weight,
                       a.eps, a.Y, a.scale, (TIO*)a.R, a.rows, a.D);
}

template <typename TIO, int TPR, int K, bool LINES>
void bwd_launch(const RmsBwdArgs& a, int planes, hipStream_t s)
{
    hipLaunchKernelGGL((rms_bwd_kernel<TIO, TPR, K, LINES>), dim3(planes), dim3(kBlock<TPR>), 0, s,
                       (const TIO*)a.R, a.weight, (const TIO*)a.dY, (const TIO*)a.dR, a.eps,
                       (TIO*)a.dX, a.dweight ? (float*)a.workspace : nullptr, a.rows, a.D);
}

// a case of the switches over shapes
#define RMS_SHAPE(f, TPR, K, ...)                                                       \
    case TPR * 8 + K:                                                                   \
        if (a.D * sizeof(TIO) % 128) f<TIO, TPR, K, false>(__VA_ARGS__);                \
        else f<TIO, TPR, K, true>(__VA_ARGS__);                                         \
        break;

template <typename TIO>
hipError_t fwd_typed(const RmsArgs& a, hipStream_t s)
{
    const Shape shape = shape_of(a.D, kVec<TIO>);
    if (shape.tpr) {
        switch (shape.tpr * 8 + shape.k) {
            RMS_SHAPE(fwd_launch, 2, 1, a, s)
            RMS_SHAPE(fwd_launch, 4, 1, a, s)
            RMS_SHAPE(fwd_launch, 8, 1, a, s)
            RMS_SHAPE(fwd_launch, 16, 1, a, s)
            RMS_SHAPE(fwd_launch, 32, 1, a, s)
            RMS_SHAPE(fwd_launch, 64, 1, a, s)
            RMS_SHAPE(fwd_launch, 64, 2, a, s)
            RMS_SHAPE(fwd_launch, 256, 1, a, s)
            RMS_SHAPE(fwd_launch, 256, 2, a, s)
            RMS_SHAPE(fwd_launch, 256, 4, a, s)
            RMS_SHAPE(fwd_launch, 512, 4, a, s)
            RMS_SHAPE(fwd_launch, 1024, 4, a, s)
        default: return hipErrorInvalidValue;
        }
        return hipGetLastError();
    }
    const dim3 grid((unsigned)std::min(kMostBlocks<256>, a.rows)), block(256);
    if (a.scale)
        hipLaunchKernelGGL((rms_fwd_loop_kernel<TIO, true>), grid, block, 0, s, (const TIO*)a.X,
                           (const TIO*)a.residual, a.weight, a.eps, a.Y, a.scale, (TIO*)a.R, a.rows,
                           a.D);
    else
        hipLaunchKernelGGL((rms_fwd_loop_kernel<TIO, false>), grid, block, 0, s, (const TIO*)a.X,
                           (const TIO*)a.residual, a.weight, a.eps, a.Y, a.scale, (TIO*)a.R, a.rows,
                           a.D);
    return hipGetLastError();
}

template <typename TIO>
hipError_t bwd_typed(const RmsBwdArgs& a, hipStream_t s)
{
    const Shape shape = bwd_shape_of(a.D, kVec<TIO>);
    const int planes = planes_of(a.rows, a.D, kVec<TIO>);
    if (shape.tpr) {
        switch (shape.tpr * 8 + shape.k) {
            RMS_SHAPE(bwd_launch, 2, 1, a, planes, s)
            RMS_SHAPE(bwd_launch, 4, 1, a, planes, s)
            RMS_SHAPE(bwd_launch, 8, 1, a, planes, s)
            RMS_SHAPE(bwd_launch, 16, 1, a, planes, s)
            RMS_SHAPE(bwd_launch, 32, 1, a, planes, s)
            RMS_SHAPE(bwd_launch, 64, 1, a, planes, s)
            RMS_SHAPE(bwd_launch, 64, 2, a, planes, s)
            RMS_SHAPE(bwd_launch, 256, 1, a, planes, s)
            RMS_SHAPE(bwd_launch, 256, 2, a, planes, s)
            RMS_SHAPE(bwd_launch, 256, 4, a, planes, s)
            RMS_SHAPE(bwd_launch, 512, 4, a, planes, s)
        default: return hipErrorInvalidValue;
        }
    } else {
        hipLaunchKernelGGL(rms_bwd_loop_kernel<TIO>, dim3(planes), dim3(256), 0, s,
                           (const TIO*)a.R, a.weight, (const TIO*)a.dY, (const TIO*)a.dR, a.eps,
                           (TIO*)a.dX, a.dweight ? (float*)a.workspace : nullptr, a.rows, a.D);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.dweight) return e;
    hipLaunchKernelGGL(rms_planes_kernel, dim3((a.D + 31) / 32), dim3(1024), 0, s,
                       (const float*)a.workspace, a.dweight, planes, a.D);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm_fwd(const RmsArgs& a, hipStream_t s)
{
    return a.bf16 ? fwd_typed<uint16_t>(a, s) : fwd_typed<float>(a, s);
}

size_t rmsnorm_bwd_workspace(long long rows, int D, bool bf16)
{
    return (size_t)planes_of(rows, D, bf16 ? 8 : 4) * D * 4;
}

hipError_t launch_rmsnorm_bwd(const RmsBwdArgs& a, hipStream_t s)
{
    return a.bf16 ? bwd_typed<uint16_t>(a, s) : bwd_typed<float>(a, s);
}

}  // namespace ttt
