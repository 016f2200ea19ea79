// Norm over many gradient tensors, and their scaling to a given largest norm.
//
// Two launches for every 64 tensors, whatever their sizes: the tensors' addresses travel
// as a kernel argument (so a captured call needs no table in memory), and the workgroups
// go over all their 32 KiB pieces in turn.  The first launch leaves one fp64 sum of
// squares per workgroup; in the second every workgroup adds those sums, in the same
// order, while its first piece is on its way, and scales.  Sums are in fp64 because
// squares of fp32 values leave fp32's range.
//
// HBM bounds it: one read for the norm and, since no element can be scaled before the
// last one is read, a second read and a write.  The second launch takes the pieces in the
// opposite order, so that what the first read last, up to the 256 MB of the last cache,
// need not come from HBM again.
#include <stdint.h>

#include <algorithm>

#include "block_launch.h"
#include "device_common.h"
#include "mfma_common.h"

namespace ttt {
namespace {

constexpr int kThreads = 256;
constexpr int kParts = 1024;       // workgroups of the first launch, and partial sums
constexpr int kTensors = 64;       // of one launch
constexpr int kQuads = 8;          // 16-byte accesses of a thread per piece
constexpr int kPiece = kThreads * kQuads * 16;

typedef uint32_t quad __attribute__((ext_vector_type(4)));
typedef quad quad_any __attribute__((aligned(2)));

struct Table {
    const void* grad[kTensors];
    void* out[kTensors];
    long long size[kTensors];      // elements
    long long first[kTensors];     // piece that the tensor starts with
    unsigned long long bf16;       // bit per tensor
    long long pieces;
    int n;
};

__device__ __forceinline__ double block_sum(double x, double* lds)
{
    for (int o = 32; o; o >>= 1) x += __shfl_xor(x, o);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    return lds[0] + lds[1] + lds[2] + lds[3];
}

// the tensor that a piece lies in
__device__ __forceinline__ int tensor_of(const Table& t, long long piece)
{
    int lo = 0, hi = t.n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (t.first[mid] <= piece) lo = mid;
        else hi = mid;
    }
    return lo;
}

// A piece's elements as this thread holds them: quads of whole ones, and at the tensor's end one
// element more.
template <typename TIO>
struct Held {
    static constexpr int V = 16 / (int)sizeof(TIO);
    quad q[kQuads];
    TIO last;
    long long at, n;               // element of the first quad (later ones kThreads quads on); size

    __device__ __forceinline__ long long place(int k) const { return at + (long long)k * kThreads * V; }
    __device__ __forceinline__ bool whole(int k) const { return place(k) + V <= n; }
    // the tensor's last n % V elements belong to the first threads of its last piece
    __device__ __forceinline__ long long extra(long long piece) const
    {
        const long long i = n / V * V + threadIdx.x;
        const bool ends = (piece + 1) * kPiece / (int)sizeof(TIO) >= n;
        return ends && threadIdx.x < V && i < n ? i : -1;
    }
    __device__ __forceinline__ void load(const TIO* p, long long size, long long piece)
    {
        n = size;
        at = piece * (kPiece / (int)sizeof(TIO)) + (long long)threadIdx.x * V;
#pragma unroll
        for (int k = 0; k < kQuads; ++k) {
            q[k] = quad{0, 0, 0, 0};
            if (whole(k)) q[k] = *reinterpret_cast<const quad_any*>(p + place(k));
        }
        const long long e = extra(piece);
        last = e >= 0 ? p[e] : TIO(0);
    }
};

__device__ __forceinline__ float wide(float v) { return v; }
__device__ __forceinline__ float wide(uint16_t v) { return bf16_bits_to_f32(v); }

__device__ __forceinline__ void squares(float v, double& s) { s = fma((double)v, (double)v, s); }

template <typename TIO>
__device__ __forceinline__ double square_piece(const void* p, long long size, long long piece)
{
    Held<TIO> h;
    h.load((const TIO*)p, size, piece);
    double s[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
    for (int k = 0; k < kQuads; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(TIO) == 4) {
                squares(__uint_as_float(h.q[k][i]), s[i]);
            } else {
                squares(__uint_as_float(h.q[k][i] << 16), s[i]);
                squares(__uint_as_float(h.q[k][i] & 0xffff0000u), s[i]);
            }
        }
    squares(wide(h.last), s[0]);
    return (s[0] + s[1]) + (s[2] + s[3]);
}

// more: sums of earlier tensors are there already
__global__ __launch_bounds__(kThreads) void clip_square_kernel(const Table t, double* part, bool more)
{
    __shared__ double lds[4];
    double s = 0.0;
    for (long long i = blockIdx.x; i < t.pieces; i += gridDim.x) {
        const int k = tensor_of(t, i);
        const long long piece = i - t.first[k];
        s += t.bf16 >> k & 1 ? square_piece<uint16_t>(t.grad[k], t.size[k], piece)
                             : square_piece<float>(t.grad[k], t.size[k], piece);
    }
    s = block_sum(s, lds);
    if (threadIdx.x == 0) part[blockIdx.x] = more ? part[blockIdx.x] + s : s;
}

__device__ __forceinline__ double norm_of(const double* part, int parts, double* lds)
{
    double s = 0.0;
    for (int i = threadIdx.x; i < parts; i += kThreads) s += part[i];
    return sqrt(block_sum(s, lds));
}

template <typename TIO>
__device__ __forceinline__ void scale_piece(const Held<TIO>& h, void* out, long long piece, float f)
{
    TIO* o = (TIO*)out;
#pragma unroll
    for (int k = 0; k < kQuads; ++k) {
        if (!h.whole(k)) continue;
        quad r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = h.q[k][i];
            if constexpr (sizeof(TIO) == 4) r[i] = __float_as_uint(__uint_as_float(w) * f);
            else r[i] = pack_bf16x2(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xffff0000u) * f);
        }
        __builtin_nontemporal_store(r, reinterpret_cast<quad_any*>(o + h.place(k)));
    }
    const long long e = h.extra(piece);
    if (e >= 0) io<TIO>::store(o, e, wide(h.last) * f);
}

// norm: written by the first workgroup, where it is not nullptr
__global__ __launch_bounds__(kThreads) void clip_scale_kernel(const Table t,
                                                              const double* __restrict__ part,
                                                              int parts, float max_norm, float eps,
                                                              float* norm)
{
    __shared__ double lds[4];
    float f = 0.f;
    bool first = true;
    for (long long i = t.pieces - 1 - blockIdx.x; i >= 0 || first; i -= gridDim.x) {
        const int k = i >= 0 ? tensor_of(t, i) : 0;
        const long long piece = i - t.first[k];
        const bool bf16 = t.bf16 >> k & 1;
        Held<uint16_t> hb;
        Held<float> hf;
        if (i >= 0 && bf16) hb.load((const uint16_t*)t.grad[k], t.size[k], piece);
        if (i >= 0 && !bf16) hf.load((const float*)t.grad[k], t.size[k], piece);
        if (first) {
            const double n = norm_of(part, parts, lds), q = (double)max_norm / (n + (double)eps);
            f = q > 1.0 ? 1.f : (float)q;      // NaN stays one
            if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
            first = false;
        }
        if (i < 0 || (f == 1.f && t.out[k] == t.grad[k])) continue;
        if (bf16) scale_piece(hb, t.out[k], piece, f);
        else scale_piece(hf, t.out[k], piece, f);
    }
}

}  // namespace

size_t clip_workspace() { return kParts * sizeof(double); }

hipError_t launch_clip(const ClipArgs& a, hipStream_t s)
{
    double* part = (double*)a.workspace;
    const dim3 block(kThreads);
    // `use` gets every table of up to kTensors tensors in turn
    auto tables = [&](auto&& use) {
        for (int i = 0;;) {
            Table t;
            t.n = 0;
            t.pieces = 0;
            t.bf16 = 0;
            for (; i < a.n && t.n < kTensors; ++i) {
                if (!a.sizes[i]) continue;
                const long long per = kPiece / (a.dtypes[i] ? 2 : 4);
                t.grad[t.n] = a.grads[i];
                t.out[t.n] = a.outs ? a.outs[i] : nullptr;
                t.size[t.n] = a.sizes[i];
                t.first[t.n] = t.pieces;
                t.bf16 |= (unsigned long long)(a.dtypes[i] != 0) << t.n;
                t.pieces += (a.sizes[i] + per - 1) / per;
                ++t.n;
            }
            use(t);
            if (i >= a.n) return;
        }
    };
    // as many partial sums as the table with the most pieces has work for
    int parts = 1;
    tables([&](const Table& t) { parts = (int)std::max<long long>(parts, std::min<long long>(kParts, t.pieces)); });
    bool more = false;
    tables([&](const Table& t) {
        hipLaunchKernelGGL(clip_square_kernel, dim3(parts), block, 0, s, t, part, more);
        more = true;
    });
    float* norm = a.norm;
    tables([&](Table& t) {
        if (!a.outs) t.pieces = 0;
        if (!norm && !t.pieces) return;
        const unsigned grid = (unsigned)std::max<long long>(1, std::min<long long>(2 * kParts, t.pieces));
        hipLaunchKernelGGL(clip_scale_kernel, dim3(grid), block, 0, s, t, part, parts, a.max_norm,
                           a.eps, norm);
        norm = nullptr;
    });
    return hipGetLastError();
}

}  // namespace ttt
