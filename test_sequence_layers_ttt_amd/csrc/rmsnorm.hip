// Root-mean-square norm with the residual's addition: forward in the I/O type or in e4m3
// with one scale per row, and the backward pass.
//
// A row of D features is held in registers by TPR threads, K vectors of 16 bytes each, so
// every input is read once and every output written once: HBM bounds it (32768 x 2048
// bf16 backward 99 us for 537 MB, 5.4 TB/s; 16384 x 2048 to e4m3 42 us for 235 MB; a
// device copy reaches 5.2 TB/s).  Rows of up to 128 vectors stay within one wave (sums by
// lane exchanges, no LDS, no barrier); longer ones take a workgroup: 256 threads with one
// vector each beat one wave with four (16384 x 2048 to e4m3: 46 and 53 us), which has too
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

typedef unsigned long long word64;
typedef uint32_t quad __attribute__((ext_vector_type(4)));
typedef quad quad_any __attribute__((aligned(2)));

template <typename TIO> constexpr int kVec = 16 / (int)sizeof(TIO);
// -0, which any value plus is that value
template <typename TIO>
constexpr quad kNoResidual = sizeof(TIO) == 4
    ? quad{0x80000000u, 0x80000000u, 0x80000000u, 0x80000000u}
    : quad{0x80008000u, 0x80008000u, 0x80008000u, 0x80008000u};

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

// the same of 64-bit words
template <int O>
__device__ __forceinline__ void halves(word64 x, word64& lo, word64& hi)
{
    unsigned l[2], h[2];
    halves<O>((unsigned)x, l[0], h[0]);
    halves<O>((unsigned)(x >> 32), l[1], h[1]);
    lo = (word64)l[1] << 32 | l[0];
    hi = (word64)h[1] << 32 | h[0];
}

template <int CTRL>
__device__ __forceinline__ word64 moved(word64 x)
{
    return (word64)moved<CTRL>((unsigned)(x >> 32)) << 32 | moved<CTRL>((unsigned)x);
}

// reduction over W <= 64 neighbouring lanes, the same bits in each: `f` is symmetric
template <int W, typename T, typename F>
__device__ __forceinline__ T over_lanes(T x, F&& f)
{
    if constexpr (W > 1) x = f(x, moved<kDppQuadXor1>(x));
    if constexpr (W > 2) x = f(x, moved<kDppQuadXor2>(x));
    if constexpr (W > 4) x = f(x, moved<kDppRowHalfMirror>(x));
    if constexpr (W > 8) x = f(x, moved<kDppRowMirror>(x));
    T lo, hi;
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
template <typename T>
__device__ __forceinline__ T max_bits(T a, T b) { return a > b ? a : b; }

// N values of the TPR threads of a row reduced by `f`, the same bits in each; `lds` holds N of
// them per wave where a row takes several
template <int TPR, int N, typename T, typename F>
__device__ __forceinline__ void over_row(T (&x)[N], T* lds, F&& f)
{
    constexpr int W = TPR < 64 ? TPR : 64, WAVES = TPR / 64;
#pragma unroll
    for (int n = 0; n < N; ++n) x[n] = over_lanes<W>(x[n], f);
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
            for (int i = 1; i < WAVES; ++i) x[n] = f(x[n], lds[n * WAVES + i]);
        }
    }
}

template <int TPR>
__device__ __forceinline__ float row_sum(float x, void* lds)
{
    unsigned b[1] = {__float_as_uint(x)};
    over_row<TPR>(b, (unsigned*)lds, add_bits);
    return __uint_as_float(b[0]);
}

// a row's sum and its largest magnitude at once
template <int TPR>
__device__ __forceinline__ void sum_and_max(unsigned (&x)[2], unsigned* lds)
{
    constexpr int W = TPR < 64 ? TPR : 64, WAVES = TPR / 64;
    x[0] = over_lanes<W>(x[0], add_bits);
    x[1] = over_lanes<W>(x[1], max_bits<unsigned>);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) {
            lds[2 * (threadIdx.x >> 6)] = x[0];
            lds[2 * (threadIdx.x >> 6) + 1] = x[1];
        }
        __syncthreads();
        x[0] = lds[0];
        x[1] = lds[1];
#pragma unroll
        for (int i = 1; i < WAVES; ++i) {
            x[0] = add_bits(x[0], lds[2 * i]);
            x[1] = max_bits(x[1], lds[2 * i + 1]);
        }
    }
}

// the row's largest: `x` has the bits of a magnitude
template <int TPR, typename T>
__device__ __forceinline__ T row_max(T x, void* lds)
{
    T b[1] = {x};
    over_row<TPR>(b, (T*)lds, [](T a, T c) { return max_bits(a, c); });
    return b[0];
}

// four values as e4m3, rounded to nearest even (up to 464 in magnitude that is 448; NaN stays)
__device__ __forceinline__ unsigned pack_e4m3(float a, float b, float c, float d)
{
    const int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}

// A row's e4m3 values: y / (max|y| / 448) is t / (max|t| / 448) with t = r * weight, as the rate
// cancels.  The fp32 quotient is off by up to 7 roundings (two of t, two of the largest t, and one each
// of 448 / top, of the factors below and of the product): where t times 448 / top (1 + 2^-21) and t times
// 448 / top (1 - 2^-21) give the same e4m3 values, it is theirs.  Where they do not (one value in 10^5),
// and in rows whose fp32 values leave the range in which those are relative errors, the quotient is
// formed in fp64.  (fp64 throughout: 16384 x 2048 bf16 59 us, against 47.)
struct Row8 {
    float hi, lo;        // 0 where the scale is 0
    bool plain;          // the row's fp32 values are in range
    __device__ __forceinline__ Row8(float top, float rate)
    {
        plain = top >= 0x1p-100f && top <= 0x1p100f && rate > 0.f;
        const float inv = scale_of(top, rate) == 0.f ? 0.f : kE4m3Max / top;
        hi = inv * (1.f + 0x1p-21f);
        lo = inv * (1.f - 0x1p-21f);
    }
    // whether a thread whose largest fp32 |t| is m may have the row's largest in fp64
    __device__ __forceinline__ bool may_have(float m, float top) const
    {
        return !plain || m >= top * (1.f - 0x1p-21f);
    }
    // max|y| / 448
    __device__ __forceinline__ static float scale_of(double most, float rate)
    {
        return (float)(most * rate * (1.0 / kE4m3Max));
    }
    // four values, and whether they are certain
    __device__ __forceinline__ unsigned four(const float* t, bool& sure) const
    {
        const unsigned a = pack_e4m3(t[0] * hi, t[1] * hi, t[2] * hi, t[3] * hi);
        sure = sure && a == pack_e4m3(t[0] * lo, t[1] * lo, t[2] * lo, t[3] * lo);
        return a;
    }
};

// The same in fp64, the quotient's remainder put right, so that what is rounded is the formula's value
// to 2^-52 and a tie is a tie.  A scale of 0 (a row of zeros) gives 0; a NaN or an infinity in the row
// makes it NaN throughout.
struct Row64 {
    double most, inv;
    __device__ __forceinline__ Row64(double m, float scale)
    {
        most = m;
        inv = scale == 0.f ? 0.0 : 1.0 / m;
    }
    // the quotient, in fp32 to the side of every e4m3 value and tie that it is on: 20 bits, the last
    // one set where what is cut off is not 0
    __device__ __forceinline__ float operator()(double t) const
    {
        const double n = t * (double)kE4m3Max, q = n * inv;
        const word64 b = (word64)__double_as_longlong(fma(fma(-q, most, n), inv, q));
        return (float)__longlong_as_double((long long)((b >> 32 | (unsigned)((unsigned)b != 0)) << 32));
    }
};

// the larger of two magnitudes as fp64 bits, where a NaN is above everything
__device__ __forceinline__ word64 larger(word64 a, double t)
{
    return max_bits(a, (word64)__double_as_longlong(fabs(t)));
}

// the squares of a vector's elements that the one before does not have
template <int V>
__device__ __forceinline__ void add_squares(const float (&r)[V], int dup, float& ss)
{
    if (dup == 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) ss = fmaf(r[i], r[i], ss);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) ss = i >= dup ? fmaf(r[i], r[i], ss) : ss;
    }
}

// threads of a workgroup
template <int TPR> constexpr int kBlock = TPR < 256 ? 256 : TPR;
// rows a thread has under way at once
template <int TPR, int K> constexpr int kRows = TPR <= 64 && K == 1 ? 2 : 1;

template <typename TIO, int TPR, int K, bool LINES>
__global__ __launch_bounds__(kBlock<TPR>) void rms_fwd_kernel(
    const TIO* X, const TIO* residual, const float* __restrict__ weight, float eps, TIO* Y, TIO* R,
    long long rows, int D)
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
                add_squares<V>(r[k], dup[k], ss);
            }
            const float rate = rsqrtf(row_sum<TPR>(ss, lds) * inv_d + eps);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (r0 + u >= rows || dup[k] == V) continue;
                const size_t at = (size_t)(r0 + u) * D + col[k];
                if (R) store16<LINES>(R + at, narrow<TIO>(r[k]));
#pragma unroll
                for (int i = 0; i < V; ++i) r[k][i] *= rate * w[k][i];
                store16<LINES>(Y + at, narrow<TIO>(r[k]));
            }
        }
    }
}

// The same to e4m3.
template <typename TIO, int TPR, int K, bool LINES>
__global__ __launch_bounds__(kBlock<TPR>) void rms_q8_kernel(
    const TIO* X, const TIO* residual, const float* __restrict__ weight, float eps, uint8_t* Y,
    float* scale, TIO* R, long long rows, int D)
{
    constexpr int V = kVec<TIO>, U = kRows<TPR, K>, GROUPS = kBlock<TPR> / TPR;
    __shared__ unsigned lds[TPR > 64 ? 2 * (TPR / 64) : 1];
    __shared__ word64 lds64[TPR > 64 ? TPR / 64 : 1];
    __shared__ bool doubt;             // of a row that takes several waves
    const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR;
    const int vectors = (D + V - 1) / V;
    int col[K], dup[K];
    float w[K][V], from = 0.f;         // from: inf where a weight is not finite, which fp64 has to see
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int v = lane + k * TPR;
        col[k] = min(v * V, D - V);
        dup[k] = v < vectors ? v * V - col[k] : V;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            w[k][i] = weight && dup[k] < V ? weight[col[k] + i] : 1.f;
            if (!isfinite(w[k][i])) from = __builtin_inff();
        }
    }
    const float inv_d = 1.f / D;
    for (long long r0 = ((long long)blockIdx.x * GROUPS + group) * U; r0 - group * U < rows;
         r0 += (long long)gridDim.x * GROUPS * U) {
        quad x[U][K], z[U][K];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < K; ++k) {
                x[u][k] = quad{0, 0, 0, 0};
                z[u][k] = kNoResidual<TIO>;
                if (r0 + u < rows && dup[k] < V) {
                    const size_t at = (size_t)(r0 + u) * D + col[k];
                    x[u][k] = load16<LINES>(X + at);
                    if (residual) z[u][k] = load16<LINES>(residual + at);
                }
            }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool live = r0 + u < rows;
            // r of vector k, widened again from its words each time: fp64 may need the words, and there
            // are no registers for both
            auto values = [&](int k, float (&r)[V]) {
                if constexpr (K > 1) asm volatile("" : "+v"(x[u][k]), "+v"(z[u][k]));
                float a[V];
                widen<TIO>(x[u][k], r);
                widen<TIO>(z[u][k], a);
#pragma unroll
                for (int i = 0; i < V; ++i) r[i] += a[i];
            };
            // t of vector k in fp64
            auto exact = [&](int k, double (&t)[V]) {
                asm volatile("" : "+v"(x[u][k]), "+v"(z[u][k]));
                float b[V], a[V];
                widen<TIO>(x[u][k], b);
                widen<TIO>(z[u][k], a);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float by = w[k][i];
                    asm volatile("" : "+v"(by));
                    t[i] = ((double)b[i] + a[i]) * by;
                }
            };
            auto exact_most = [&]() {
                word64 most = 0;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    double t[V];
                    exact(k, t);
#pragma unroll
                    for (int i = 0; i < V; ++i) most = larger(most, t[i]);
                }
                return most;
            };
            float ss = 0.f, m = from;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float r[V];
                values(k, r);
                add_squares<V>(r, dup[k], ss);
#pragma unroll
                for (int i = 0; i < V; ++i) m = fmaxf(m, fabsf(r[i] * w[k][i]));
            }
            if constexpr (TPR > 64) {
                __syncthreads();       // the row before has read what is in LDS
                if (threadIdx.x == 0) doubt = false;
            }
            unsigned both[2] = {__float_as_uint(ss), __float_as_uint(m)};
            sum_and_max<TPR>(both, lds);
            const float rate = rsqrtf(__uint_as_float(both[0]) * inv_d + eps), top = __uint_as_float(both[1]);
            const Row8 row(top, rate);
            bool sure = row.plain;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float r[V];
                values(k, r);
                if (R && live && dup[k] < V)
                    store16<LINES>(R + (size_t)(r0 + u) * D + col[k], narrow<TIO>(r));
#pragma unroll
                for (int i = 0; i < V; ++i) r[i] *= w[k][i];
                unsigned q[V / 4];
#pragma unroll
                for (int i = 0; i < V / 4; ++i) q[i] = row.four(r + 4 * i, sure);
                if (live && dup[k] < V) __builtin_memcpy(Y + (size_t)(r0 + u) * D + col[k], q, V);
            }
            float of_row = Row8::scale_of(top, rate);
            bool again;
            if constexpr (TPR > 64) {
                if (!sure) doubt = true;
                __syncthreads();
                again = doubt;
            } else {
                again = __any(!sure);
            }
            if (again) {
                word64 mine = 0;
                if (row.may_have(m, top)) mine = exact_most();
                const double most = __longlong_as_double((long long)row_max<TPR>(mine, lds64));
                if (!row.plain) of_row = Row8::scale_of(most, rate);
                const Row64 row64(most, of_row);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    if (sure) break;
                    double t[V];
                    exact(k, t);
                    unsigned q[V / 4];
#pragma unroll
                    for (int i = 0; i < V / 4; ++i)
                        q[i] = pack_e4m3(row64(t[4 * i]), row64(t[4 * i + 1]), row64(t[4 * i + 2]),
                                         row64(t[4 * i + 3]));
                    if (live && dup[k] < V) __builtin_memcpy(Y + (size_t)(r0 + u) * D + col[k], q, V);
                }
            }
            if (live && lane == 0) scale[r0 + u] = of_row;
        }
    }
}

// Rows too long (or too short) for the registers' layout: a workgroup per row, the row read again
// for every pass, 8 elements of a thread at a time.  A thread adds 8 terms in fp32 and those sums in
// fp64: one fp32 sum of all its D / 256 terms would be off by as many roundings (mean(r^2) of equal
// values by 4e-4 at 2^23 features).
template <typename TIO, bool Q8>
__global__ __launch_bounds__(256) void rms_fwd_loop_kernel(const TIO* X, const TIO* residual,
                                                           const float* __restrict__ weight,
                                                           float eps, void* Y, float* scale, TIO* R,
                                                           long long rows, int D)
{
    constexpr int N = 8;
    __shared__ word64 lds[4];
    for (long long row = blockIdx.x; row < rows; row += gridDim.x) {
        const size_t base = (size_t)row * D;
        // f(first element, x, residual, weight) for this thread's elements: first, first + 256, ...;
        // zeros past the row's end.  (Loads without a condition: each one with one would be waited for
        // by itself.)
        const TIO* z = residual ? residual : X;
        auto eights = [&](auto&& f) {
            for (int i = threadIdx.x; i < D; i += 256 * N) {
                float x[N], a[N], w[N];
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const int at = min(i + 256 * n, D - 1);
                    x[n] = io<TIO>::load(X, base + at);
                    a[n] = io<TIO>::load(z, base + at);
                    w[n] = weight ? weight[at] : 1.f;
                }
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    if (i + 256 * n >= D) {
                        x[n] = a[n] = 0.f;
                        w[n] = 1.f;
                    }
                    if (!residual) a[n] = -0.f;
                }
                f(i, x, a, w);
            }
        };
        double ss = 0.0;
        word64 largest = 0;
        eights([&](int, const float (&x)[N], const float (&a)[N], const float (&w)[N]) {
            float s = 0.f;
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const float r = x[n] + a[n];
                s = fmaf(r, r, s);
                if constexpr (Q8) largest = larger(largest, ((double)x[n] + a[n]) * w[n]);
            }
            ss += s;
        });
        const float rate = rsqrtf(row_sum<256>((float)ss, lds) / D + eps);
        double most = 0.0;
        if constexpr (Q8) most = __longlong_as_double((long long)row_max<256>(largest, lds));
        const float of_row = Row8::scale_of(most, rate);
        const Row64 row64(most, of_row);
        if (Q8 && threadIdx.x == 0) scale[row] = of_row;
        eights([&](int i, const float (&x)[N], const float (&a)[N], const float (&w)[N]) {
#pragma unroll
            for (int n = 0; n < N; ++n) {
                if (i + 256 * n >= D) break;
                const size_t at = base + i + 256 * n;
                const float r = x[n] + a[n];
                if constexpr (Q8)
                    ((uint8_t*)Y)[at] = (uint8_t)pack_e4m3(row64(((double)x[n] + a[n]) * w[n]), 0.f, 0.f, 0.f);
                else
                    io<TIO>::store((TIO*)Y, at, r * (rate * w[n]));
                if (R) io<TIO>::store(R, at, r);
            }
        });
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
        over_row<TPR>(both, lds, add_bits);
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

// the same, a workgroup per row at a time, for the rows of rms_fwd_loop_kernel; where rows are short
// each thread keeps its columns' sums in the plane
template <typename TIO>
__global__ __launch_bounds__(256) void rms_bwd_loop_kernel(
    const TIO* __restrict__ R, const float* __restrict__ weight, const TIO* dY, const TIO* dR,
    float eps, TIO* dX, float* __restrict__ plane, long long rows, int D)
{
    constexpr int N = 8;
    __shared__ unsigned lds[4];
    if (plane)
        for (int i = threadIdx.x; i < D; i += 256) plane[(size_t)blockIdx.x * D + i] = 0.f;
    for (long long row = blockIdx.x; row < rows; row += gridDim.x) {
        const size_t base = (size_t)row * D;
        // f(first element, r, dy, weight) for this thread's elements: first, first + 256, ...; zeros past
        // the row's end
        auto eights = [&](auto&& f) {
            for (int i = threadIdx.x; i < D; i += 256 * N) {
                float r[N], dy[N], w[N];
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const int at = min(i + 256 * n, D - 1);
                    r[n] = io<TIO>::load(R, base + at);
                    dy[n] = io<TIO>::load(dY, base + at);
                    w[n] = weight ? weight[at] : 1.f;
                }
#pragma unroll
                for (int n = 0; n < N; ++n)
                    if (i + 256 * n >= D) {
                        r[n] = dy[n] = 0.f;
                        w[n] = 1.f;
                    }
                f(i, r, dy, w);
            }
        };
        const TIO* e = dR ? dR : R;
        double ss = 0.0, su = 0.0;
        eights([&](int, const float (&r)[N], const float (&dy)[N], const float (&w)[N]) {
            float a = 0.f, b = 0.f;
#pragma unroll
            for (int n = 0; n < N; ++n) {
                a = fmaf(r[n], r[n], a);
                b = fmaf(dy[n] * w[n], r[n], b);
            }
            ss += a;
            su += b;
        });
        const float rate = rsqrtf(row_sum<256>((float)ss, lds) / D + eps);
        const float m = row_sum<256>((float)su, lds) * rate / D;
        eights([&](int i, const float (&r)[N], const float (&dy)[N], const float (&w)[N]) {
            float dr[N];
#pragma unroll
            for (int n = 0; n < N; ++n) dr[n] = io<TIO>::load(e, base + min(i + 256 * n, D - 1));
#pragma unroll
            for (int n = 0; n < N; ++n) {
                if (i + 256 * n >= D) break;
                const float k = r[n] * rate;
                if (plane) plane[(size_t)blockIdx.x * D + i + 256 * n] += dy[n] * k;
                io<TIO>::store(dX, base + i + 256 * n, fmaf(rate, dy[n] * w[n] - k * m, dR ? dr[n] : 0.f));
            }
        });
    }
}

// dweight of long rows: the rows' rates first, then every column's sum by a thread, the rows dealt out to
// gridDim.y workgroups, 8 rows at a time: 8 terms in fp32, those sums in fp64.  (A plane of dweight for
// every workgroup of the kernel above would take 1024 times 4 D bytes, read and written for every row.)
// Both run before that kernel, as it may write dX at dY's place.
template <typename TIO>
__global__ __launch_bounds__(256) void rms_rate_kernel(const TIO* __restrict__ R, float eps,
                                                       float* __restrict__ rate, long long rows, int D)
{
    constexpr int N = 8;
    __shared__ unsigned lds[4];
    for (long long row = blockIdx.x; row < rows; row += gridDim.x) {
        const TIO* p = R + (size_t)row * D;
        double ss = 0.0;
        for (int i = threadIdx.x; i < D; i += 256 * N) {
            float s = 0.f;
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const float r = io<TIO>::load(p, min(i + 256 * n, D - 1));
                s = i + 256 * n < D ? fmaf(r, r, s) : s;
            }
            ss += s;
        }
        const float k = rsqrtf(row_sum<256>((float)ss, lds) / D + eps);
        if (threadIdx.x == 0) rate[row] = k;
    }
}

template <typename TIO>
__global__ __launch_bounds__(256) void rms_columns_kernel(const TIO* __restrict__ R,
                                                          const TIO* __restrict__ dY,
                                                          const float* __restrict__ rate,
                                                          float* __restrict__ plane, long long rows, int D)
{
    constexpr int N = 8;
    const int c = blockIdx.x * 256 + threadIdx.x, P = gridDim.y;
    if (c >= D) return;
    double sum = 0.0;
    for (long long row = blockIdx.y; row < rows; row += (long long)N * P) {
        float s = 0.f;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const long long at = row + (long long)n * P;
            const size_t from = at < rows ? at : rows - 1;
            const float r = io<TIO>::load(R, from * D + c), dy = io<TIO>::load(dY, from * D + c);
            s = at < rows ? fmaf(dy, r * rate[from], s) : s;
        }
        sum += s;
    }
    plane[(size_t)blockIdx.y * D + c] = (float)sum;
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
// (16384 x 2048 bf16 to e4m3: 47.4 us with twice as many, 46.2 with these).
template <int TPR> constexpr long long kMostBlocks = 256 * (1024 / kBlock<TPR>);

// The backward pass holds weight and dweight in fp32 next to three inputs: past 2048 vectors a row
// takes 1024 threads, which have 128 registers each, and four bf16 vectors take 161.  (fp32 vectors
// take 116; their rows go the same way.)
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
    // long rows: workgroups for 1024 threads a compute unit
    if (!s.tpr && D >= vec) return (int)std::max(1ll, std::min<long long>(rows, (1ll << 18) / D));
    const int block = std::max(256, s.tpr), groups = s.tpr ? block / s.tpr : 1;
    const long long most = 256 * (1024 / block) / (s.k > 1 ? 2 : 1);
    return (int)std::max(1ll, std::min<long long>((rows + groups - 1) / groups, most));
}

// bytes of the workspace before the planes: the rates of long rows
size_t rates_bytes(long long rows, int D, int vec)
{
    return bwd_shape_of(D, vec).tpr || D < vec ? 0 : ((size_t)rows * 4 + 255) / 256 * 256;
}

template <typename TIO, int TPR, int K, bool LINES>
void fwd_launch(const RmsArgs& a, hipStream_t s)
{
    constexpr int PER = kBlock<TPR> / TPR * kRows<TPR, K>;
    const dim3 grid((unsigned)std::min(kMostBlocks<TPR>, (a.rows + PER - 1) / PER)), block(kBlock<TPR>);
    hipLaunchKernelGGL((rms_fwd_kernel<TIO, TPR, K, LINES>), grid, block, 0, s, (const TIO*)a.X,
                       (const TIO*)a.residual, a.weight, a.eps, (TIO*)a.Y, (TIO*)a.R, a.rows, a.D);
}

template <typename TIO, int TPR, int K, bool LINES>
void q8_launch(const RmsArgs& a, hipStream_t s)
{
    constexpr int PER = kBlock<TPR> / TPR * kRows<TPR, K>;
    const dim3 grid((unsigned)std::min(kMostBlocks<TPR>, (a.rows + PER - 1) / PER)), block(kBlock<TPR>);
    hipLaunchKernelGGL((rms_q8_kernel<TIO, TPR, K, LINES>), grid, block, 0, s, (const TIO*)a.X,
                       (const TIO*)a.residual, a.weight, a.eps, (uint8_t*)a.Y, a.scale, (TIO*)a.R, a.rows,
                       a.D);
}

template <typename TIO, int TPR, int K, bool LINES>
void bwd_launch(const RmsBwdArgs& a, int planes, hipStream_t s)
{
    hipLaunchKernelGGL((rms_bwd_kernel<TIO, TPR, K, LINES>), dim3(planes), dim3(kBlock<TPR>), 0, s,
                       (const TIO*)a.R, a.weight, (const TIO*)a.dY, (const TIO*)a.dR, a.eps,
                       (TIO*)a.dX, a.dweight ? (float*)a.workspace : nullptr, a.rows, a.D);
}

// A case of the switches over shapes.  Rows of less than a line are never whole lines.
#define RMS_SHAPE(f, TPR, K, ...)                                                       \
    case TPR * 8 + K:                                                                   \
        if (a.D * sizeof(TIO) % 128) f<TIO, TPR, K, false>(__VA_ARGS__);                \
        else f<TIO, TPR, K, (TPR) * (K) * 16 >= 128>(__VA_ARGS__);                      \
        break;

template <typename TIO>
hipError_t fwd_typed(const RmsArgs& a, hipStream_t s)
{
    Shape shape = shape_of(a.D, kVec<TIO>);
    // To e4m3, four bf16 vectors and what fp64 may need of them fill the registers: two, and twice as
    // many threads (4096 x 8192 bf16 49 us, against 53; fp32 vectors have half as many values, and
    // take 81 us that way, against 75).
    constexpr int W = sizeof(TIO) == 4 ? 4 : 2;
    if (a.scale && shape.k == 4 && shape.tpr < 1024) shape = {shape.tpr * 4 / W, W};
    if (shape.tpr && a.scale) {
        switch (shape.tpr * 8 + shape.k) {
            RMS_SHAPE(q8_launch, 2, 1, a, s)
            RMS_SHAPE(q8_launch, 4, 1, a, s)
            RMS_SHAPE(q8_launch, 8, 1, a, s)
            RMS_SHAPE(q8_launch, 16, 1, a, s)
            RMS_SHAPE(q8_launch, 32, 1, a, s)
            RMS_SHAPE(q8_launch, 64, 1, a, s)
            RMS_SHAPE(q8_launch, 64, 2, a, s)
            RMS_SHAPE(q8_launch, 256, 1, a, s)
            RMS_SHAPE(q8_launch, 256, 2, a, s)
            RMS_SHAPE(q8_launch, 1024 / W, W, a, s)
            RMS_SHAPE(q8_launch, 2048 / W, W, a, s)
            RMS_SHAPE(q8_launch, 1024, 4, a, s)
        default: return hipErrorInvalidValue;
        }
        return hipGetLastError();
    }
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
    const size_t rates = rates_bytes(a.rows, a.D, kVec<TIO>);
    float* plane = (float*)((char*)a.workspace + rates);
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
        const dim3 grid((unsigned)std::max(1ll, std::min(kMostBlocks<256>, a.rows)));
        if (a.dweight && rates) {
            hipLaunchKernelGGL(rms_rate_kernel<TIO>, grid, dim3(256), 0, s, (const TIO*)a.R, a.eps,
                               (float*)a.workspace, a.rows, a.D);
            hipLaunchKernelGGL(rms_columns_kernel<TIO>, dim3((a.D + 255) / 256, planes), dim3(256), 0, s,
                               (const TIO*)a.R, (const TIO*)a.dY, (const float*)a.workspace, plane, a.rows,
                               a.D);
        }
        hipLaunchKernelGGL(rms_bwd_loop_kernel<TIO>, grid, dim3(256), 0, s, (const TIO*)a.R, a.weight,
                           (const TIO*)a.dY, (const TIO*)a.dR, a.eps, (TIO*)a.dX,
                           a.dweight && !rates ? plane : nullptr, a.rows, a.D);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.dweight) return e;
    hipLaunchKernelGGL(rms_planes_kernel, dim3((a.D + 31) / 32), dim3(1024), 0, s, (const float*)plane,
                       a.dweight, planes, a.D);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm_fwd(const RmsArgs& a, hipStream_t s)
{
    return a.bf16 ? fwd_typed<uint16_t>(a, s) : fwd_typed<float>(a, s);
}

size_t rmsnorm_bwd_workspace(long long rows, int D, bool bf16)
{
    const int vec = bf16 ? 8 : 4;
    return rates_bytes(rows, D, vec) + (size_t)planes_of(rows, D, vec) * D * 4;
}

hipError_t launch_rmsnorm_bwd(const RmsBwdArgs& a, hipStream_t s)
{
    return a.bf16 ? bwd_typed<uint16_t>(a, s) : bwd_typed<float>(a, s);
}

}  // namespace ttt
