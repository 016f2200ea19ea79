// Group norm with an activation over channels-last tensors [N, S, C]:
//   n = (x - mean) rstd over the S places and the C / G channels of a group,
//   y = act(n weight + bias),
// and its gradients:  dv = dy act'(v),  u = dv weight,
//   dx = rstd (u - mean(u) - n mean(u n)),  dweight = sum of dv n,  dbias = sum of dv.
//
// Three forms, by the size of a group.
//   rows    one place (S = 1: the norm of every head's output of every token) and at most 64 vectors
//           a group: it stays in registers, every input is read once, and a thread keeps the same
//           channels for all its rows, so weight and bias (and the backward pass's sums) stay in
//           registers too.  HBM bounds it: 16384 x 2048 bf16 in 32 groups with SiLU 33 us forward
//           (134 MB), 49 us backward (201 MB) and 5 us for the sums.
//   blocks  up to 4096 vectors a group: 16 to 512 threads hold it in registers, read once as well
//           (16384 x 4096 bf16 in one group 52 us forward; as a slab 769 us); the sums for weight
//           and bias take a second read, channel by channel.
//   slabs   larger ones: the places are shared out over the workgroups, each thread with channels
//           of its own: sums per channel first, then a workgroup per group joins them, then a
//           second read writes the result (8 x 4096 x 640 bf16 17, 4 and 20 us).
//
// Sums run in a fixed order: the same bits on every call.
#include <algorithm>

#include "block_launch.h"
#include "device_common.h"
#include "mfma_common.h"
#include "ttt.h"

namespace ttt {
namespace {

// A launch has fewer than 2^32 threads along an axis of its grid: workgroups past 2^22 go on along y.
__device__ __forceinline__ long long workgroup() { return (long long)blockIdx.y * gridDim.x + blockIdx.x; }
constexpr long long kMostX = 1 << 22;
dim3 workgroups(long long n)
{
    const long long x = std::min(n, kMostX);
    return dim3((unsigned)x, (unsigned)((n + x - 1) / x));
}

// V elements of the I/O type as fp32
template <typename TIO, int V> struct Vec {
    RawRow<TIO, V> raw;
    __device__ __forceinline__ void load(const TIO* p) { raw.load(p); }
    __device__ __forceinline__ float at(int i) const { return raw.at(i); }
};

template <typename TIO, int V>
__device__ __forceinline__ void store_vec(TIO* p, const float (&y)[V])
{
    if constexpr (sizeof(TIO) == 4) {
        if constexpr (V == 4) *reinterpret_cast<f32x4*>(p) = f32x4{y[0], y[1], y[2], y[3]};
        else if constexpr (V == 2) *reinterpret_cast<f32x2*>(p) = f32x2{y[0], y[1]};
        else *p = y[0];
    } else {
        if constexpr (V == 8)
            *reinterpret_cast<u32x4*>(p) = pack_bf16x8(f32x4{y[0], y[1], y[2], y[3]}, f32x4{y[4], y[5], y[6], y[7]});
        else if constexpr (V == 4) *reinterpret_cast<u32x2*>(p) = pack_bf16x4(f32x4{y[0], y[1], y[2], y[3]});
        else if constexpr (V == 2) *reinterpret_cast<unsigned*>(p) = pack_bf16x2(y[0], y[1]);
        else *p = (uint16_t)(pack_bf16x2(y[0], 0.f) & 0xffffu);
    }
}

// V neighbouring floats (aligned as one is), or a value for all where there are none
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef f32x2 f32x2_any __attribute__((aligned(4)));
template <int V>
__device__ __forceinline__ void floats(const float* p, long long at, float none, float (&x)[V])
{
    if (!p) {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = none;
        return;
    }
    p += at;
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const f32x4 v = *reinterpret_cast<const f32x4_any*>(p + i);
            x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
        }
    } else if constexpr (V == 2) {
        const f32x2 v = *reinterpret_cast<const f32x2_any*>(p);
        x[0] = v.x; x[1] = v.y;
    } else {
        x[0] = *p;
    }
}

// 1 / (1 + exp(-v)) by the hardware's exponential and reciprocal (a last place each, and |v| 2^-24
// of the exponential for its argument's rounding)
__device__ __forceinline__ float sigmoid(float v)
{
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504f * v));
}

template <int ACT>
__device__ __forceinline__ float act(float v)
{
    if constexpr (ACT == TTT_ACT_SILU) return v * sigmoid(v);
    if constexpr (ACT == TTT_ACT_GELU) return v * fmaf(0.5f, erff(0.70710678f * v), 0.5f);
    return v;
}

// the derivative
template <int ACT>
__device__ __forceinline__ float dact(float v)
{
    if constexpr (ACT == TTT_ACT_SILU) {
        const float y = sigmoid(v);
        return fmaf(v * y, 1.f - y, y);
    }
    if constexpr (ACT == TTT_ACT_GELU)
        return fmaf(v * 0.39894228f, __builtin_amdgcn_exp2f(-0.72134752f * v * v),
                    fmaf(0.5f, erff(0.70710678f * v), 0.5f));
    return 1.f;
}

// sum over L neighbouring lanes (a power of two), the same bits in each
template <int L>
__device__ __forceinline__ float lane_sum(float x)
{
    auto add = [&](int y) { x += __int_as_float(y); };
    if constexpr (L >= 2) add(__builtin_amdgcn_mov_dpp(__float_as_int(x), kDppQuadXor1, 0xF, 0xF, false));
    if constexpr (L >= 4) add(__builtin_amdgcn_mov_dpp(__float_as_int(x), kDppQuadXor2, 0xF, 0xF, false));
    if constexpr (L >= 8) add(__builtin_amdgcn_mov_dpp(__float_as_int(x), kDppRowHalfMirror, 0xF, 0xF, false));
    if constexpr (L >= 16) add(__builtin_amdgcn_mov_dpp(__float_as_int(x), kDppRowMirror, 0xF, 0xF, false));
    if constexpr (L >= 32) x += __shfl_xor(x, 16, 64);
    if constexpr (L >= 64) x += __shfl_xor(x, 32, 64);
    return x;
}

// ---- one place: a group in L lanes, one vector each ------------------------------------
// slots: rows that a workgroup works on at once (where its 256 threads hold several).
// block x: 256 threads' worth of channels, y: rows.
template <int L>
struct Place {
    int group, lane, slot;
    bool in;
    __device__ __forceinline__ Place(int G, int vectors)
    {
        const int per = G * L;     // threads of a row
        int t = blockIdx.x * 256 + threadIdx.x;
        slot = 0;
        if (per < 256) { slot = t / per; t -= slot * per; }
        group = t / L;
        lane = t % L;
        in = group < G && lane < vectors && slot < (per < 256 ? 256 / per : 1);
    }
};

template <typename TIO, int V, int L, int ACT>
__global__ void __launch_bounds__(256) group_row_fwd_kernel(GroupArgs a, int slots)
{
    const int per = a.C / a.G, vectors = per / V;
    const Place<L> p(a.G, vectors);
    const int ch = p.group * per + p.lane * V;
    float w[V], b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        w[i] = p.in && a.weight ? a.weight[ch + i] : 1.f;
        b[i] = p.in && a.bias ? a.bias[ch + i] : 0.f;
    }
    const TIO* X = (const TIO*)a.X;
    TIO* Y = (TIO*)a.Y;
    const float inv = 1.f / (float)per;
    const long long step = (long long)gridDim.y * slots;
    // (every lane goes through the same rows: the sums are over all lanes)
    for (long long r0 = (long long)blockIdx.y * slots; r0 < a.N; r0 += step) {
        const long long row = r0 + p.slot;
        const bool in = p.in && row < a.N;
        Vec<TIO, V> x;
        float v[V], s = 0.f;
        if (in) x.load(X + row * a.C + ch);
#pragma unroll
        for (int i = 0; i < V; ++i) s += v[i] = in ? x.at(i) : 0.f;
        const float mean = lane_sum<L>(s) * inv;
        s = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            v[i] -= mean;
            s = in ? fmaf(v[i], v[i], s) : 0.f;
        }
        const float rstd = __builtin_amdgcn_rsqf(fmaf(lane_sum<L>(s), inv, a.eps));
        if (in) {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = act<ACT>(fmaf(v[i] * rstd, w[i], b[i]));
            store_vec<TIO, V>(Y + row * a.C + ch, v);
            if (p.lane == 0) {
                a.mean[row * a.G + p.group] = mean;
                a.rstd[row * a.G + p.group] = rstd;
            }
        }
    }
}

// the sums for dweight and dbias go to planes [2][C], one for each (block y, slot)
template <typename TIO, int V, int L, int ACT>
__global__ void __launch_bounds__(256) group_row_bwd_kernel(GroupBwdArgs a, int slots, float* planes)
{
    const int per = a.C / a.G, vectors = per / V;
    const Place<L> p(a.G, vectors);
    const int ch = p.group * per + p.lane * V;
    float w[V], b[V], sw[V], sb[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        w[i] = p.in && a.weight ? a.weight[ch + i] : 1.f;
        b[i] = p.in && a.bias ? a.bias[ch + i] : 0.f;
        sw[i] = sb[i] = 0.f;
    }
    const TIO* X = (const TIO*)a.X;
    const TIO* dY = (const TIO*)a.dY;
    TIO* dX = (TIO*)a.dX;
    const float inv = 1.f / (float)per;
    const long long step = (long long)gridDim.y * slots;
    for (long long r0 = (long long)blockIdx.y * slots; r0 < a.N; r0 += step) {
        const long long row = r0 + p.slot;
        const bool in = p.in && row < a.N;
        Vec<TIO, V> x, dy;
        float n[V], u[V], s1 = 0.f, s2 = 0.f, mean = 0.f, rstd = 0.f;
        if (in) {
            x.load(X + row * a.C + ch);
            dy.load(dY + row * a.C + ch);
            mean = a.mean[row * a.G + p.group];
            rstd = a.rstd[row * a.G + p.group];
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            n[i] = u[i] = 0.f;
            if (in) {
                n[i] = (x.at(i) - mean) * rstd;
                const float dv = dy.at(i) * dact<ACT>(fmaf(n[i], w[i], b[i]));
                sw[i] = fmaf(dv, n[i], sw[i]);
                sb[i] += dv;
                u[i] = dv * w[i];
            }
            s1 += u[i];
            s2 = fmaf(u[i], n[i], s2);
        }
        s1 = lane_sum<L>(s1) * inv;
        s2 = lane_sum<L>(s2) * inv;
        if (in) {
#pragma unroll
            for (int i = 0; i < V; ++i) u[i] = rstd * (u[i] - fmaf(n[i], s2, s1));
            store_vec<TIO, V>(dX + row * a.C + ch, u);
        }
    }
    if (planes && p.in) {
        float* to = planes + ((size_t)blockIdx.y * slots + p.slot) * 2 * a.C + ch;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            to[i] = sw[i];
            to[a.C + i] = sb[i];
        }
    }
}

// dweight and dbias: columns of all planes [2][C] in fp64, 32 runs of planes a column
__global__ void __launch_bounds__(1024) group_planes_kernel(const float* planes, long long count, int C,
                                                            float* dweight, float* dbias)
{
    __shared__ double part[32][33];
    const int c = threadIdx.x & 31, k = threadIdx.x >> 5, at = blockIdx.x * 32 + c;
    double s = 0.0;
    if (at < 2 * C) {
#pragma unroll 8
        for (long long i = k; i < count; i += 32) s += planes[i * 2 * C + at];
    }
    part[k][c] = s;
    __syncthreads();
    // the columns' 32 sums lie across a half wave now
    double t = part[c][k];
    for (int o = 1; o < 32; o <<= 1) t += __shfl_xor(t, o, 64);
    const int to = blockIdx.x * 32 + k;
    if (c == 0 && to < 2 * C) {
        if (to < C) { if (dweight) dweight[to] = (float)t; }
        else if (dbias) dbias[to - C] = (float)t;
    }
}

// ---- many places: channels in the threads, places over the workgroups --------------------
// Workgroup (x and z: row by row 256 threads' worth of vectors of channels, y: places first .. last).
struct Slab {
    long long row;
    int ch, slot, slots;      // channel, place within a step, places a step
    bool in;
    long long first, last;
    __device__ __forceinline__ Slab(int vectors, int V, long long N, long long S, int parts)
    {
        const int wide = (vectors + 255) / 256;
        row = (long long)blockIdx.z * (gridDim.x / wide) + blockIdx.x / wide;
        int t = threadIdx.x, x = (int)(blockIdx.x % wide) * 256;
        slots = vectors < 256 ? 256 / vectors : 1;
        slot = 0;
        if (vectors < 256) { slot = t / vectors; t -= slot * vectors; }
        ch = (x + t) * V;
        in = x + t < vectors && slot < slots && row < N;
        const long long each = (S + parts - 1) / parts;
        first = each * blockIdx.y;
        last = first + each < S ? first + each : S;
    }
};

// (a, b) of each thread's channels joined over the slots, in LDS, slot after slot
template <int V, typename JOIN>
__device__ __forceinline__ void over_slots(const Slab& p, int vectors, float (&s)[V], float (&q)[V],
                                           JOIN join)
{
    __shared__ float ls[256][V + 1], lq[256][V + 1];
#pragma unroll
    for (int i = 0; i < V; ++i) { ls[threadIdx.x][i] = s[i]; lq[threadIdx.x][i] = q[i]; }
    __syncthreads();
    if (p.slot == 0 && p.in)
        for (int k = 1; k < p.slots; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i)
                join(i, k, ls[threadIdx.x + k * vectors][i], lq[threadIdx.x + k * vectors][i]);
}

// how many of the places first .. last slot k takes
__device__ __forceinline__ float taken(const Slab& p, int k)
{
    const long long n = p.last - p.first - k;
    return n > 0 ? (float)((n + p.slots - 1) / p.slots) : 0.f;
}

// (mean, sum of squares about it) of na and nb values joined
__device__ __forceinline__ void join_moments(float& na, float& mean, float& m2, float nb, float mb, float qb)
{
    if (nb == 0.f) return;
    const float n = na + nb, d = mb - mean, f = nb / n;
    mean = fmaf(d, f, mean);
    m2 += fmaf(d * d, na * f, qb);
    na = n;
}

// mean and squares about it of every channel over this workgroup's places.  A thread takes its
// places in runs of 16, sums of the distance to the mean of those before: with n the places so far,
//   mean += s / n,   squares about it += q - s^2 / n.
// That keeps the digits of a far mean, and of values behind a first one that is far from all others
// (sums about that one over the whole run would not: n^2 / 2 roundings of its square).
template <typename TIO, int V>
__global__ void __launch_bounds__(256) group_moments_kernel(GroupArgs a, int parts, float* planes)
{
    constexpr int RUN = 16;
    const int vectors = a.C / V;
    const Slab p(vectors, V, a.N, a.S, parts);
    const TIO* X = (const TIO*)a.X + p.row * a.S * a.C;
    float s[V], q[V];
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = q[i] = 0.f;
    const float mine = taken(p, p.slot);
    if (p.in && p.first + p.slot < p.last) {
        const TIO* at = X + (p.first + p.slot) * a.C + p.ch;
        const long long step = (long long)p.slots * a.C;
        Vec<TIO, V> x;
        x.load(at);
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = x.at(i);
        const long long all = (p.last - p.first - p.slot + p.slots - 1) / p.slots;
        for (long long done = 1; done < all;) {
            const int run = (int)min((long long)RUN, all - done);
            float d1[V], d2[V];
#pragma unroll
            for (int i = 0; i < V; ++i) d1[i] = d2[i] = 0.f;
            auto take = [&](const Vec<TIO, V>& y) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float d = y.at(i) - s[i];
                    d1[i] += d;
                    d2[i] = fmaf(d, d, d2[i]);
                }
            };
            if (run == RUN) {
#pragma unroll
                for (int k = 0; k < RUN; k += 4) {
                    Vec<TIO, V> y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e].load(at += step);
#pragma unroll
                    for (int e = 0; e < 4; ++e) take(y[e]);
                }
            } else {
                for (int k = 0; k < run; ++k) {
                    Vec<TIO, V> y;
                    y.load(at += step);
                    take(y);
                }
            }
            done += run;
            const float inv = 1.f / (float)done;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = d1[i] * inv;
                q[i] += fmaxf(d2[i] - d1[i] * d, d2[i] * 0.f);   // (not below 0; NaN stays)
                s[i] += d;
            }
        }
    }
    float n[V];
#pragma unroll
    for (int i = 0; i < V; ++i) n[i] = mine;
    over_slots<V>(p, vectors, s, q, [&](int i, int k, float mb, float qb) {
        join_moments(n[i], s[i], q[i], taken(p, k), mb, qb);
    });
    if (p.slot == 0 && p.in) {
        float* to = planes + ((size_t)p.row * parts + blockIdx.y) * 2 * a.C + p.ch;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            to[i] = s[i];
            to[a.C + i] = q[i];
        }
    }
}

// sum of 256 threads' values, in each
__device__ __forceinline__ double block_sum(double x, double* room)
{
    for (int o = 1; o < 64; o <<= 1) x += __shfl_xor(x, o, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) room[threadIdx.x >> 6] = x;
    __syncthreads();
    return (room[0] + room[1]) + (room[2] + room[3]);
}

// one workgroup per (row, group): mean and rstd from its channels' and parts' moments, each
// read twice: the mean first, then the squares about it
__global__ void __launch_bounds__(256) group_statistics_kernel(GroupArgs a, int parts, const float* planes)
{
    __shared__ double room[4];
    const long long id = workgroup(), row = id / a.G;
    const int group = (int)(id % a.G), per = a.C / a.G;
    if (row >= a.N) return;
    const long long each = (a.S + parts - 1) / parts;
    const float* from = planes + (size_t)row * parts * 2 * a.C + group * per;
    const int entries = parts * per;
    const double n = (double)a.S * per;
    auto have = [&](int part) { return (float)max(0ll, min(each, a.S - each * part)); };
    // (the first entries of a thread stay in registers)
    constexpr int KEPT = 12;
    float m[KEPT], q[KEPT], h[KEPT];
#pragma unroll
    for (int k = 0; k < KEPT; ++k) {
        const int e = threadIdx.x + 256 * k;
        m[k] = q[k] = h[k] = 0.f;
        if (e < entries) {
            const float* p = from + (size_t)(e / per) * 2 * a.C + e % per;
            m[k] = p[0];
            q[k] = p[a.C];
            h[k] = have(e / per);
        }
    }
    double s = 0.0;
#pragma unroll
    for (int k = 0; k < KEPT; ++k)
        if (h[k] > 0.f) s += (double)h[k] * m[k];
    for (int e = threadIdx.x + 256 * KEPT; e < entries; e += 256)
        s += (double)have(e / per) * from[(size_t)(e / per) * 2 * a.C + e % per];
    const double mean = block_sum(s, room) / n;
    s = 0.0;
#pragma unroll
    for (int k = 0; k < KEPT; ++k)
        if (h[k] > 0.f) s += q[k] + h[k] * (m[k] - mean) * (m[k] - mean);
    for (int e = threadIdx.x + 256 * KEPT; e < entries; e += 256) {
        const double g = have(e / per);
        const float* p = from + (size_t)(e / per) * 2 * a.C + e % per;
        const double d = p[0] - mean;
        if (g > 0.0) s += p[a.C] + g * d * d;
    }
    s = block_sum(s, room) / n;
    if (threadIdx.x == 0) {
        a.mean[id] = (float)mean;
        a.rstd[id] = (float)(1.0 / sqrt(s + (double)a.eps));
    }
}

template <typename TIO, int V, int ACT>
__global__ void __launch_bounds__(256) group_apply_kernel(GroupArgs a, int parts)
{
    const Slab p(a.C / V, V, a.N, a.S, parts);
    if (!p.in) return;
    const long long row = p.row;
    const TIO* X = (const TIO*)a.X + row * a.S * a.C + p.ch;
    TIO* Y = (TIO*)a.Y + row * a.S * a.C + p.ch;
    float mean[V], rstd[V], w[V], b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int ch = p.ch + i;
        const long long g = row * a.G + ch / (a.C / a.G);
        mean[i] = a.mean[g];
        rstd[i] = a.rstd[g];
        w[i] = a.weight ? a.weight[ch] : 1.f;
        b[i] = a.bias ? a.bias[ch] : 0.f;
    }
#pragma unroll 2
    for (long long t = p.first + p.slot; t < p.last; t += p.slots) {
        Vec<TIO, V> x;
        x.load(X + t * a.C);
        float y[V];
#pragma unroll
        for (int i = 0; i < V; ++i) y[i] = act<ACT>(fmaf((x.at(i) - mean[i]) * rstd[i], w[i], b[i]));
        store_vec<TIO, V>(Y + t * a.C, y);
    }
}

// sums of dv n and dv of every channel over this workgroup's places, to planes [2][C]
template <typename TIO, int V, int ACT>
__global__ void __launch_bounds__(256) group_sums_kernel(GroupBwdArgs a, int parts, float* planes)
{
    const int vectors = a.C / V;
    const Slab p(vectors, V, a.N, a.S, parts);
    const long long row = p.row;
    const TIO* X = (const TIO*)a.X + row * a.S * a.C + p.ch;
    const TIO* dY = (const TIO*)a.dY + row * a.S * a.C + p.ch;
    float s[V], q[V];
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = q[i] = 0.f;
    if (p.in) {
        float mean[V], rstd[V], w[V], b[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int ch = p.ch + i;
            const long long g = row * a.G + ch / (a.C / a.G);
            mean[i] = a.mean[g];
            rstd[i] = a.rstd[g];
            w[i] = a.weight ? a.weight[ch] : 1.f;
            b[i] = a.bias ? a.bias[ch] : 0.f;
        }
#pragma unroll 2
        for (long long t = p.first + p.slot; t < p.last; t += p.slots) {
            Vec<TIO, V> x, dy;
            x.load(X + t * a.C);
            dy.load(dY + t * a.C);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float n = (x.at(i) - mean[i]) * rstd[i];
                const float dv = dy.at(i) * dact<ACT>(fmaf(n, w[i], b[i]));
                s[i] = fmaf(dv, n, s[i]);
                q[i] += dv;
            }
        }
    }
    over_slots<V>(p, vectors, s, q, [&](int i, int, float sb, float qb) {
        s[i] += sb;
        q[i] += qb;
    });
    if (p.slot == 0 && p.in) {
        float* to = planes + ((size_t)row * parts + blockIdx.y) * 2 * a.C + p.ch;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            to[i] = s[i];
            to[a.C + i] = q[i];
        }
    }
}

// one workgroup per (row, group): means of u and u n
__global__ void __launch_bounds__(256) group_means_kernel(GroupBwdArgs a, int parts, const float* planes,
                                                          float* means)
{
    __shared__ double room[4];
    const long long id = workgroup(), row = id / a.G;
    const int group = (int)(id % a.G), per = a.C / a.G;
    if (row >= a.N) return;
    const float* from = planes + (size_t)row * parts * 2 * a.C + group * per;
    double m1 = 0.0, m2 = 0.0;
    for (int e = threadIdx.x; e < parts * per; e += 256) {
        const float* p = from + (size_t)(e / per) * 2 * a.C + e % per;
        const double w = a.weight ? a.weight[group * per + e % per] : 1.f;
        m2 += w * p[0];
        m1 += w * p[a.C];
    }
    m1 = block_sum(m1, room);
    m2 = block_sum(m2, room);
    if (threadIdx.x == 0) {
        const double n = (double)a.S * per;
        means[2 * id] = (float)(m1 / n);
        means[2 * id + 1] = (float)(m2 / n);
    }
}

template <typename TIO, int V, int ACT>
__global__ void __launch_bounds__(256) group_dx_kernel(GroupBwdArgs a, int parts, const float* means)
{
    const Slab p(a.C / V, V, a.N, a.S, parts);
    if (!p.in) return;
    const long long row = p.row, at = row * a.S * a.C + p.ch;
    const TIO* X = (const TIO*)a.X + at;
    const TIO* dY = (const TIO*)a.dY + at;
    TIO* dX = (TIO*)a.dX + at;
    float mean[V], rstd[V], w[V], b[V], m1[V], m2[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int ch = p.ch + i;
        const long long g = row * a.G + ch / (a.C / a.G);
        mean[i] = a.mean[g];
        rstd[i] = a.rstd[g];
        m1[i] = means[2 * g];
        m2[i] = means[2 * g + 1];
        w[i] = a.weight ? a.weight[ch] : 1.f;
        b[i] = a.bias ? a.bias[ch] : 0.f;
    }
#pragma unroll 2
    for (long long t = p.first + p.slot; t < p.last; t += p.slots) {
        Vec<TIO, V> x, dy;
        x.load(X + t * a.C);
        dy.load(dY + t * a.C);
        float y[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float n = (x.at(i) - mean[i]) * rstd[i];
            const float u = dy.at(i) * dact<ACT>(fmaf(n, w[i], b[i])) * w[i];
            y[i] = rstd[i] * (u - fmaf(n, m2[i], m1[i]));
        }
        store_vec<TIO, V>(dX + t * a.C, y);
    }
}

// ---- a group in the registers of TS threads ------------------------------------------------
constexpr int kHeld = 8;       // vectors of a thread

// sum over the TS threads of a slab, in each
template <int TS>
__device__ __forceinline__ float held_sum(float x, float* room)
{
    x = lane_sum<(TS < 64 ? TS : 64)>(x);
    if constexpr (TS > 64) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0) room[threadIdx.x >> 6] = x;
        __syncthreads();
        x = 0.f;
#pragma unroll
        for (int i = 0; i < TS / 64; ++i) x += room[i];
    }
    return x;
}

// this thread's place: slab, and the offsets of its vectors in it (a workgroup has 256 / TS slabs)
template <int V, int TS>
struct Held {
    long long slab, base, at[kHeld];
    int lane, ch[kHeld], first;      // channels, and the group's first
    bool in[kHeld], live;
    __device__ __forceinline__ Held(long long N, long long S, int C, int G)
    {
        const int per = C / G, pv = per / V, count = (int)(S * pv);
        lane = threadIdx.x % TS;
        slab = workgroup() * (blockDim.x / TS) + threadIdx.x / TS;
        live = slab < N * G;
        first = (int)(slab % G) * per;
        base = slab / G * S * C + first;
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
            const int e = lane + TS * k;
            in[k] = live && e < count;
            ch[k] = e % pv * V;
            at[k] = base + (long long)(e / pv) * C + ch[k];
        }
    }
};

template <typename TIO, int V, int ACT, int TS>
__global__ void __launch_bounds__(TS > 256 ? TS : 256) group_block_fwd_kernel(GroupArgs a)
{
    __shared__ float room[16];
    const Held<V, TS> p(a.N, a.S, a.C, a.G);
    const TIO* X = (const TIO*)a.X;
    float v[kHeld][V], s = 0.f;
    const float inv = 1.f / (float)(a.S * (a.C / a.G));
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
        Vec<TIO, V> x;
        if (p.in[k]) x.load(X + p.at[k]);
#pragma unroll
        for (int i = 0; i < V; ++i) s += v[k][i] = p.in[k] ? x.at(i) : 0.f;
    }
    const float mean = held_sum<TS>(s, room) * inv;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
        if (p.in[k])
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[k][i] -= mean;
                s = fmaf(v[k][i], v[k][i], s);
            }
    const float rstd = __builtin_amdgcn_rsqf(fmaf(held_sum<TS>(s, room), inv, a.eps));
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
        if (!p.in[k]) continue;
        float w[V], b[V];
        floats<V>(a.weight, p.first + p.ch[k], 1.f, w);
        floats<V>(a.bias, p.first + p.ch[k], 0.f, b);
#pragma unroll
        for (int i = 0; i < V; ++i) v[k][i] = act<ACT>(fmaf(v[k][i] * rstd, w[i], b[i]));
        store_vec<TIO, V>((TIO*)a.Y + p.at[k], v[k]);
    }
    if (p.live && p.lane == 0) {
        a.mean[p.slab] = mean;
        a.rstd[p.slab] = rstd;
    }
}

template <typename TIO, int V, int ACT, int TS>
__global__ void __launch_bounds__(TS > 256 ? TS : 256) group_block_bwd_kernel(GroupBwdArgs a)
{
    __shared__ float room[16];
    const Held<V, TS> p(a.N, a.S, a.C, a.G);
    float n[kHeld][V], u[kHeld][V], s1 = 0.f, s2 = 0.f;
    const float inv = 1.f / (float)(a.S * (a.C / a.G));
    const float mean = p.live ? a.mean[p.slab] : 0.f, rstd = p.live ? a.rstd[p.slab] : 0.f;
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
        if (!p.in[k]) continue;
        Vec<TIO, V> x, dy;
        x.load((const TIO*)a.X + p.at[k]);
        dy.load((const TIO*)a.dY + p.at[k]);
        float w[V], b[V];
        floats<V>(a.weight, p.first + p.ch[k], 1.f, w);
        floats<V>(a.bias, p.first + p.ch[k], 0.f, b);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            n[k][i] = (x.at(i) - mean) * rstd;
            u[k][i] = dy.at(i) * dact<ACT>(fmaf(n[k][i], w[i], b[i])) * w[i];
            s1 += u[k][i];
            s2 = fmaf(u[k][i], n[k][i], s2);
        }
    }
    s1 = held_sum<TS>(s1, room) * inv;
    s2 = held_sum<TS>(s2, room) * inv;
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
        if (!p.in[k]) continue;
#pragma unroll
        for (int i = 0; i < V; ++i) u[k][i] = rstd * (u[k][i] - fmaf(n[k][i], s2, s1));
        store_vec<TIO, V>((TIO*)a.dX + p.at[k], u[k]);
    }
}

// sums of dv n and dv over the N S rows of C channels, to planes [2][C] of each block y: run before
// the gradient is written, which may stand at X's or dY's place
template <typename TIO, int V, int ACT>
__global__ void __launch_bounds__(256) group_columns_kernel(GroupBwdArgs a, float* planes)
{
    const int vectors = a.C / V, per = a.C / a.G;
    const Slab p(vectors, V, 1, a.N * a.S, (int)gridDim.y);
    const bool one = per % V == 0;      // (a vector's channels are of one group)
    const int group = p.ch / per;
    float s[V], q[V];
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = q[i] = 0.f;
    if (p.in) {
        float w[V], b[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            w[i] = a.weight ? a.weight[p.ch + i] : 1.f;
            b[i] = a.bias ? a.bias[p.ch + i] : 0.f;
        }
#pragma unroll 2
        for (long long t = p.first + p.slot; t < p.last; t += p.slots) {
            Vec<TIO, V> x, dy;
            x.load((const TIO*)a.X + t * a.C + p.ch);
            dy.load((const TIO*)a.dY + t * a.C + p.ch);
            const long long row = a.S == 1 ? t : t / a.S;
            float mean[V], rstd[V];
            if (one) {
                const float m = a.mean[row * a.G + group], r = a.rstd[row * a.G + group];
#pragma unroll
                for (int i = 0; i < V; ++i) { mean[i] = m; rstd[i] = r; }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const long long g = row * a.G + (p.ch + i) / per;
                    mean[i] = a.mean[g];
                    rstd[i] = a.rstd[g];
                }
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float n = (x.at(i) - mean[i]) * rstd[i];
                const float dv = dy.at(i) * dact<ACT>(fmaf(n, w[i], b[i]));
                s[i] = fmaf(dv, n, s[i]);
                q[i] += dv;
            }
        }
    }
    over_slots<V>(p, vectors, s, q, [&](int i, int, float sb, float qb) {
        s[i] += sb;
        q[i] += qb;
    });
    if (p.slot == 0 && p.in) {
        float* to = planes + (size_t)blockIdx.y * 2 * a.C + p.ch;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            to[i] = s[i];
            to[a.C + i] = q[i];
        }
    }
}

// ---- launch shapes -----------------------------------------------------------------------
constexpr size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

// the largest power of two up to 16 bytes that divides n elements
int vector_of(int n, bool bf16)
{
    int v = bf16 ? 8 : 4;
    while (n % v) v /= 2;
    return v;
}

struct Shape {
    bool rows;               // the form for one place
    int held;                // threads that hold a group (0: they do not)
    int wide;                // vector of a row of all channels
    int V, L, x, y, slots;   // vector, lanes of a group, grid, rows a workgroup holds at once
    int parts;               // workgroups along the places
    size_t planes;           // of 2 C floats
};

Shape shape_of(long long N, long long S, int C, int G, bool bf16)
{
    Shape h = {};
    const int per = C / G;
    const int v = vector_of(per, bf16);
    if (S == 1 && per / v <= 64) {
        h.rows = true;
        h.V = v;
        h.L = 1;
        while (h.L < per / v) h.L *= 2;
        const long long threads = (long long)G * h.L;
        h.slots = threads < 256 ? (int)(256 / threads) : 1;
        h.x = (int)((threads + 255) / 256);
        // workgroups enough to fill the card several times over, and no more planes than that
        const long long steps = (N + h.slots - 1) / h.slots;
        h.y = (int)std::min<long long>(steps, std::max(1, 1024 / h.x));
        h.planes = (size_t)h.y * h.slots;
        return h;
    }
    h.wide = vector_of(C, bf16);
    const int vectors = C / h.wide;
    const long long count = per / v <= 4096 / S ? S * (per / v) : 4097;
    if (count <= 512 * kHeld) {
        h.V = v;
        h.held = count <= 64 ? 16 : count <= 64 * kHeld ? 64 : count <= 256 * kHeld ? 256 : 512;
        h.slots = vectors < 256 ? 256 / vectors : 1;
        h.x = (vectors + 255) / 256;
        h.y = (int)std::min<long long>((N * S + h.slots - 1) / h.slots, std::max(1, 1024 / h.x));
        h.planes = (size_t)h.y;
        return h;
    }
    h.V = h.wide;
    h.slots = vectors < 256 ? 256 / vectors : 1;
    h.x = (vectors + 255) / 256;
    const long long most = std::max<long long>(1, S / (16ll * h.slots));
    h.parts = (int)std::min<long long>(most, std::max<long long>(1, 1024 / (N * h.x)));
    h.planes = (size_t)N * h.parts;
    return h;
}

template <typename TIO, int V, int L>
void row_fwd(const GroupArgs& a, const Shape& h, hipStream_t s)
{
    const dim3 grid(h.x, h.y);
    if (a.act == TTT_ACT_SILU) group_row_fwd_kernel<TIO, V, L, TTT_ACT_SILU><<<grid, 256, 0, s>>>(a, h.slots);
    else if (a.act == TTT_ACT_GELU) group_row_fwd_kernel<TIO, V, L, TTT_ACT_GELU><<<grid, 256, 0, s>>>(a, h.slots);
    else group_row_fwd_kernel<TIO, V, L, TTT_ACT_NONE><<<grid, 256, 0, s>>>(a, h.slots);
}

template <typename TIO, int V, int L>
void row_bwd(const GroupBwdArgs& a, const Shape& h, float* planes, hipStream_t s)
{
    const dim3 grid(h.x, h.y);
    if (a.act == TTT_ACT_SILU)
        group_row_bwd_kernel<TIO, V, L, TTT_ACT_SILU><<<grid, 256, 0, s>>>(a, h.slots, planes);
    else if (a.act == TTT_ACT_GELU)
        group_row_bwd_kernel<TIO, V, L, TTT_ACT_GELU><<<grid, 256, 0, s>>>(a, h.slots, planes);
    else
        group_row_bwd_kernel<TIO, V, L, TTT_ACT_NONE><<<grid, 256, 0, s>>>(a, h.slots, planes);
}

template <typename TIO, int V, typename DO>
void lanes_as(int L, DO d)
{
    switch (L) {
    case 1: d(std::integral_constant<int, 1>()); break;
    case 2: d(std::integral_constant<int, 2>()); break;
    case 4: d(std::integral_constant<int, 4>()); break;
    case 8: d(std::integral_constant<int, 8>()); break;
    case 16: d(std::integral_constant<int, 16>()); break;
    case 32: d(std::integral_constant<int, 32>()); break;
    default: d(std::integral_constant<int, 64>());
    }
}

template <typename TIO, int V, int ACT>
void block_fwd(const GroupArgs& a, const Shape& h, hipStream_t s)
{
    const long long slabs = a.N * a.G;
    const int each = h.held < 256 ? 256 / h.held : 1;
    const dim3 grid = workgroups((slabs + each - 1) / each);
    if (h.held == 16) group_block_fwd_kernel<TIO, V, ACT, 16><<<grid, 256, 0, s>>>(a);
    else if (h.held == 64) group_block_fwd_kernel<TIO, V, ACT, 64><<<grid, 256, 0, s>>>(a);
    else if (h.held == 256) group_block_fwd_kernel<TIO, V, ACT, 256><<<grid, 256, 0, s>>>(a);
    else group_block_fwd_kernel<TIO, V, ACT, 512><<<grid, 512, 0, s>>>(a);
}

template <typename TIO, int V, int ACT>
void block_bwd(const GroupBwdArgs& a, const Shape& h, hipStream_t s)
{
    const long long slabs = a.N * a.G;
    const int each = h.held < 256 ? 256 / h.held : 1;
    const dim3 grid = workgroups((slabs + each - 1) / each);
    if (h.held == 16) group_block_bwd_kernel<TIO, V, ACT, 16><<<grid, 256, 0, s>>>(a);
    else if (h.held == 64) group_block_bwd_kernel<TIO, V, ACT, 64><<<grid, 256, 0, s>>>(a);
    else if (h.held == 256) group_block_bwd_kernel<TIO, V, ACT, 256><<<grid, 256, 0, s>>>(a);
    else group_block_bwd_kernel<TIO, V, ACT, 512><<<grid, 512, 0, s>>>(a);
}

template <typename TIO, int V>
void columns(const GroupBwdArgs& a, const Shape& h, float* planes, hipStream_t s)
{
    const dim3 grid(h.x, h.y);
    if (a.act == TTT_ACT_SILU) group_columns_kernel<TIO, V, TTT_ACT_SILU><<<grid, 256, 0, s>>>(a, planes);
    else if (a.act == TTT_ACT_GELU) group_columns_kernel<TIO, V, TTT_ACT_GELU><<<grid, 256, 0, s>>>(a, planes);
    else group_columns_kernel<TIO, V, TTT_ACT_NONE><<<grid, 256, 0, s>>>(a, planes);
}

// the slabs' kernels: rows along x, past its threads along z
dim3 slab_grid(const Shape& h, long long N)
{
    const long long rows = std::min(N, kMostX / h.x);
    return dim3((unsigned)(h.x * rows), h.parts, (unsigned)((N + rows - 1) / rows));
}

template <typename TIO, int V>
hipError_t fwd_as(const GroupArgs& a, const Shape& h, hipStream_t s)
{
    if (h.rows) {
        lanes_as<TIO, V>(h.L, [&](auto L) { row_fwd<TIO, V, decltype(L)::value>(a, h, s); });
        return hipGetLastError();
    }
    if (h.held) {
        if (a.act == TTT_ACT_SILU) block_fwd<TIO, V, TTT_ACT_SILU>(a, h, s);
        else if (a.act == TTT_ACT_GELU) block_fwd<TIO, V, TTT_ACT_GELU>(a, h, s);
        else block_fwd<TIO, V, TTT_ACT_NONE>(a, h, s);
        return hipGetLastError();
    }
    float* planes = (float*)a.workspace;
    const dim3 grid = slab_grid(h, a.N);
    group_moments_kernel<TIO, V><<<grid, 256, 0, s>>>(a, h.parts, planes);
    group_statistics_kernel<<<workgroups(a.N * a.G), 256, 0, s>>>(a, h.parts, planes);
    if (a.act == TTT_ACT_SILU) group_apply_kernel<TIO, V, TTT_ACT_SILU><<<grid, 256, 0, s>>>(a, h.parts);
    else if (a.act == TTT_ACT_GELU) group_apply_kernel<TIO, V, TTT_ACT_GELU><<<grid, 256, 0, s>>>(a, h.parts);
    else group_apply_kernel<TIO, V, TTT_ACT_NONE><<<grid, 256, 0, s>>>(a, h.parts);
    return hipGetLastError();
}

template <typename TIO, int V, int ACT>
void slab_bwd(const GroupBwdArgs& a, const Shape& h, float* planes, float* means, hipStream_t s)
{
    const dim3 grid = slab_grid(h, a.N);
    group_sums_kernel<TIO, V, ACT><<<grid, 256, 0, s>>>(a, h.parts, planes);
    group_means_kernel<<<workgroups(a.N * a.G), 256, 0, s>>>(a, h.parts, planes, means);
    group_dx_kernel<TIO, V, ACT><<<grid, 256, 0, s>>>(a, h.parts, means);
}

template <typename TIO, int V>
hipError_t bwd_as(const GroupBwdArgs& a, const Shape& h, hipStream_t s)
{
    const bool sums = a.dweight || a.dbias;
    float* planes = (float*)a.workspace;
    if (h.rows) {
        float* to = sums ? planes : nullptr;
        lanes_as<TIO, V>(h.L, [&](auto L) { row_bwd<TIO, V, decltype(L)::value>(a, h, to, s); });
    } else if (h.held) {
        if (sums) {
            if (h.wide == 8) { if constexpr (sizeof(TIO) == 2) columns<TIO, 8>(a, h, planes, s); }
            else if (h.wide == 4) columns<TIO, 4>(a, h, planes, s);
            else if (h.wide == 2) columns<TIO, 2>(a, h, planes, s);
            else columns<TIO, 1>(a, h, planes, s);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        if (a.act == TTT_ACT_SILU) block_bwd<TIO, V, TTT_ACT_SILU>(a, h, s);
        else if (a.act == TTT_ACT_GELU) block_bwd<TIO, V, TTT_ACT_GELU>(a, h, s);
        else block_bwd<TIO, V, TTT_ACT_NONE>(a, h, s);
    } else {
        float* means = (float*)((char*)a.workspace + up256(h.planes * 8 * a.C));
        if (a.act == TTT_ACT_SILU) slab_bwd<TIO, V, TTT_ACT_SILU>(a, h, planes, means, s);
        else if (a.act == TTT_ACT_GELU) slab_bwd<TIO, V, TTT_ACT_GELU>(a, h, planes, means, s);
        else slab_bwd<TIO, V, TTT_ACT_NONE>(a, h, planes, means, s);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (sums)
        group_planes_kernel<<<(unsigned)((2ll * a.C + 31) / 32), 1024, 0, s>>>(planes, (long long)h.planes, a.C,
                                                                            a.dweight, a.dbias);
    return hipGetLastError();
}

}  // namespace

size_t groupnorm_fwd_workspace(long long N, long long S, int C, int G, bool bf16)
{
    const Shape h = shape_of(N, S, C, G, bf16);
    return h.rows || h.held ? 0 : up256(h.planes * 8 * C);
}

size_t groupnorm_bwd_workspace(long long N, long long S, int C, int G, bool bf16)
{
    const Shape h = shape_of(N, S, C, G, bf16);
    return up256(h.planes * 8 * C) + (h.rows || h.held ? 0 : up256((size_t)N * G * 8));
}

hipError_t launch_groupnorm_fwd(const GroupArgs& a, hipStream_t s)
{
    const Shape h = shape_of(a.N, a.S, a.C, a.G, a.bf16);
    if (a.bf16)
        return h.V == 8 ? fwd_as<uint16_t, 8>(a, h, s) : h.V == 4 ? fwd_as<uint16_t, 4>(a, h, s)
             : h.V == 2 ? fwd_as<uint16_t, 2>(a, h, s) : fwd_as<uint16_t, 1>(a, h, s);
    return h.V == 4 ? fwd_as<float, 4>(a, h, s) : h.V == 2 ? fwd_as<float, 2>(a, h, s) : fwd_as<float, 1>(a, h, s);
}

hipError_t launch_groupnorm_bwd(const GroupBwdArgs& a, hipStream_t s)
{
    if (a.N == 0 || a.S == 0) {
        if (a.dweight || a.dbias)
            group_planes_kernel<<<(unsigned)((2ll * a.C + 31) / 32), 1024, 0, s>>>(nullptr, 0, a.C, a.dweight,
                                                                                a.dbias);
        return hipGetLastError();
    }
    const Shape h = shape_of(a.N, a.S, a.C, a.G, a.bf16);
    if (a.bf16)
        return h.V == 8 ? bwd_as<uint16_t, 8>(a, h, s) : h.V == 4 ? bwd_as<uint16_t, 4>(a, h, s)
             : h.V == 2 ? bwd_as<uint16_t, 2>(a, h, s) : bwd_as<uint16_t, 1>(a, h, s);
    return h.V == 4 ? bwd_as<float, 4>(a, h, s) : h.V == 2 ? bwd_as<float, 2>(a, h, s) : bwd_as<float, 1>(a, h, s);
}

}  // namespace ttt
