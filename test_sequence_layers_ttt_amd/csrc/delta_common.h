// Shared pieces of the gated delta rule's kernels: chunk geometry, products of values
// split into bf16 parts, the LDS tiles of keys and queries, and the workspace's records.
//
// A chunk is 64 tokens.  With G_t the sum of the log decays from the chunk's start
// through t, E_ts = exp(G_t - G_s), W the state at the chunk's start and
//   L_ts = E_ts k_t.k_s (s < t),   P_ts = E_ts q_t.k_s (s <= t),
//   S = (I + L diag(eta))^-1 L     (strictly lower, so (I + L diag(eta))^-1 = I - S diag(eta)
//                                   and (I + diag(eta) L)^-1 = I - diag(eta) S),
// the forward pass of a chunk is
//   R = V - exp(G) K W^T,   U = R - S (eta R),   u = eta U,
//   Z = exp(G) Q W^T + P u,   W' = exp(G_C) W + (exp(G_C - G) u)^T K
// and its adjoint, with D the gradient that reaches W',
//   dU = P^T dZ + exp(G_C - G) K D^T,   F = dU - S^T (eta dU),   dV = eta F,
//   D' = exp(G_C) D + (exp(G) dZ)^T Q - (exp(G) dV)^T K.
// Nothing is divided by eta, so eta = 0 needs no case of its own.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "delta_launch.h"
#include "device_common.h"
#include "mfma_common.h"

namespace ttt {

constexpr int kChunk = 64;
constexpr float kForget = -1e30f;     // log decays from here down forget everything

// ---- values as sums of bf16 parts ----------------------------------------
// An fp32 operand of a product is the exact sum of three bf16 parts (8 + 8 + 8 bits);
// a bf16 input is one part.  Products of parts are exact in the matrix cores' fp32 sums,
// and those below 2^-24 of the whole are left out: one part by three takes 3
// instructions, three by three 6, against 16 times the time of one for the fp32 form.
template <int N> struct Parts { u32x4 p[N]; };

__device__ __forceinline__ f32x4 widen4(u32x2 v)
{
    return f32x4{__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                 __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u)};
}

// slots 0..3 from a, 4..7 from b
template <int N>
__device__ __forceinline__ Parts<N> split(f32x4 a, f32x4 b)
{
    Parts<N> r;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        r.p[k] = pack_bf16x8(a, b);
        if (k + 1 < N) {
            a -= widen4(lo_half(r.p[k]));
            b -= widen4(hi_half(r.p[k]));
        }
    }
    return r;
}

// c + a b over 32 contraction slots, part products of order up to 2, the smallest first
template <int NA, int NB>
__device__ __forceinline__ f32x4 mma(const Parts<NA>& a, const Parts<NB>& b, f32x4 c)
{
#pragma unroll
    for (int s = 2; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int j = s - i;
            if (j >= 0 && j < NB) c = mfma32(a.p[i], b.p[j], c);
        }
    return c;
}

template <typename TIO> constexpr int kParts = sizeof(TIO) == 2 ? 1 : 3;

// ---- token tensors ---------------------------------------------------------
// rows of one (batch, head) of [B, H, T, d] or [B, T, H, d]
template <typename TIO>
struct Rows {
    TIO* p;
    size_t stride;     // elements from token to token
    __device__ __forceinline__ Rows(TIO* base, int b, int h, int H, int T, int d, bool tokens_first)
        : p(base + (tokens_first ? ((size_t)b * T * H + h) * d : ((size_t)b * H + h) * T * d)),
          stride(tokens_first ? (size_t)H * d : (size_t)d)
    {
    }
    __device__ __forceinline__ TIO* at(int t) const { return p + (size_t)t * stride; }
};

template <typename TIO> constexpr int kGran = 16 / (int)sizeof(TIO);   // elements of 16 bytes

// 16 bytes of row `row` from column `col` (columns past d are 0); `whole`: rows are
// multiples of 16 bytes
template <typename TIO>
__device__ __forceinline__ quad load_granule(const TIO* row, int col, int d, bool whole)
{
    quad q = {0u, 0u, 0u, 0u};
    if (whole) {
        if (col < d) q = *reinterpret_cast<const quad*>(row + col);
        return q;
    }
#pragma unroll
    for (int i = 0; i < kGran<TIO>; ++i)
        if (col + i < d) {
            if constexpr (sizeof(TIO) == 4) q[i] = reinterpret_cast<const uint32_t*>(row)[col + i];
            else q[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(row)[col + i] << (16 * (i & 1));
        }
    return q;
}

// ---- LDS tile of 64 tokens by DK features, rows padded by 16 bytes ----------
template <typename TIO, int DK>
struct Tile {
    static constexpr int LD = DK + kGran<TIO>;
    static constexpr int GRANULES = kChunk * DK / kGran<TIO>;
    TIO x[kChunk * LD];
};

// a tile on its way from memory: each of N threads holds its granules
template <typename TIO, int DK, int THREADS = 256>
struct TileLoad {
    static constexpr int N = Tile<TIO, DK>::GRANULES / THREADS;
    static constexpr int ROW = DK / kGran<TIO>;
    quad q[N];
    // a tile that lies within the rows and columns
    __device__ __forceinline__ void load_inside(const Rows<const TIO>& src, int t0, int tid, int first = 0)
    {
        const TIO* p = src.at(t0) + ((size_t)(tid / ROW) * src.stride + first + (tid % ROW) * kGran<TIO>);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            q[i] = *reinterpret_cast<const quad*>(p);
            p += THREADS / ROW * src.stride;
        }
    }
    // (columns from `first` of rows of d)
    __device__ __forceinline__ void load(const Rows<const TIO>& src, int t0, int T, int d, bool whole,
                                         int tid, int first = 0)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = tid + THREADS * i, r = e / ROW, col = first + (e % ROW) * kGran<TIO>;
            q[i] = t0 + r < T ? load_granule(src.at(t0 + r), col, d, whole) : quad{0u, 0u, 0u, 0u};
        }
    }
    __device__ __forceinline__ void put(Tile<TIO, DK>& to, int tid) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = tid + THREADS * i, r = e / ROW, col = (e % ROW) * kGran<TIO>;
            *reinterpret_cast<quad*>(to.x + r * Tile<TIO, DK>::LD + col) = q[i];
        }
    }
};

// Operand with the tile's token 16 i + c in the lane and features in the slots: slots
// 0..3 are features 32 j + 4 g + v, 4..7 are 32 j + 16 + 4 g + v (the order in which two
// result tiles, one above the other, are an operand).
template <typename TIO, int DK>
__device__ __forceinline__ Parts<kParts<TIO>> by_token(const Tile<TIO, DK>& t, int i, int j, int lane)
{
    const TIO* row = t.x + (16 * i + (lane & 15)) * Tile<TIO, DK>::LD + 32 * j + 4 * (lane >> 4);
    if constexpr (sizeof(TIO) == 2) {
        const u32x2 a = *reinterpret_cast<const u32x2*>(row);
        const u32x2 b = *reinterpret_cast<const u32x2*>(row + 16);
        return Parts<1>{{u32x4{a.x, a.y, b.x, b.y}}};
    } else {
        return split<3>(*reinterpret_cast<const f32x4*>(row), *reinterpret_cast<const f32x4*>(row + 16));
    }
}

// Operand with feature 16 m + c in the lane and tokens in the slots: 32 j + 4 g + v and
// 32 j + 16 + 4 g + v.  (bf16: by the transposing LDS read, see lds_transpose16)
template <typename TIO, int DK>
__device__ __forceinline__ Parts<kParts<TIO>> by_feature(const Tile<TIO, DK>& t, int m, int j, int lane)
{
    constexpr int LD = Tile<TIO, DK>::LD;
    const int c = lane & 15, g = lane >> 4;
    if constexpr (sizeof(TIO) == 2) {
        auto at = [&](int token) {
            auto p = (__attribute__((address_space(3))) s16x4*)(t.x + (token + (c >> 2)) * LD + 16 * m +
                                                                4 * (c & 3));
            return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(p));
        };
        const u32x2 a = at(32 * j + 4 * g), b = at(32 * j + 16 + 4 * g);
        return Parts<1>{{u32x4{a.x, a.y, b.x, b.y}}};
    } else {
        const TIO* p = t.x + (32 * j + 4 * g) * LD + 16 * m + c;
        const f32x4 a = {p[0], p[LD], p[2 * LD], p[3 * LD]};
        p += 16 * LD;
        return split<3>(a, f32x4{p[0], p[LD], p[2 * LD], p[3 * LD]});
    }
}

// four consecutive features of one token, widened
template <typename TIO, int DK>
__device__ __forceinline__ f32x4 token4(const Tile<TIO, DK>& t, int token, int feature)
{
    const TIO* p = t.x + token * Tile<TIO, DK>::LD + feature;
    if constexpr (sizeof(TIO) == 2) return widen4(*reinterpret_cast<const u32x2*>(p));
    else return *reinterpret_cast<const f32x4*>(p);
}

// ---- what the preparing kernel leaves for a (head, chunk) -------------------
// A lower triangular 64 x 64 matrix as the row operands of products: 6 operands that are not
// zero, row tile i against the token pair of tiles (2 j, 2 j + 1), j <= i / 2; of its transpose
// j >= i / 2.
constexpr int kFrags = 6;
__host__ __device__ constexpr int frag_lower(int i, int j) { return i < 2 ? i : 2 * (i - 1) + j; }
__host__ __device__ constexpr int frag_upper(int i, int j) { return i < 2 ? 2 * i + j : i + 2; }

// In memory it is the 10 tiles that are not zero, fp32, 16 bytes for each lane as the operand
// takes them (row c, columns 4 g ..); on the way into LDS each is split into parts and becomes
// half of an operand.  The two halves beyond the diagonal are zero from the start.  Where the
// waves that load also compute, it is the operands' three parts instead.
constexpr int kHalves = 10, kHalfQuads = kHalves * 64;
__host__ __device__ constexpr int half_lower(int i, int j) { return i * (i + 1) / 2 + j; }
__host__ __device__ constexpr int half_upper(int i, int j) { return 4 * i - i * (i - 1) / 2 + j - i; }

// An operand is its parts, one after the other, 16 bytes for each lane (1 KB a part).
constexpr int kFragQuads = kFrags * 64;       // of one part of a matrix's operands
struct Record {                               // decays of a chunk's tokens
    float hi[kChunk], lo[kChunk];             // sums of their binary logarithms, in two parts
    float eta[kChunk];
    float start[kChunk];                      // decay from the chunk's start through the token
    float end[kChunk];                        // decay from after the token to the chunk's end
    int forgets[kChunk];                      // whether the token's decay leaves nothing
};

// A decay's binary logarithm is taken no lower than this: its power is 0 by far, and sums over a
// chunk still leave the other tokens' digits alone (64 times this and 2^-27 in 53 bits).
constexpr double kLeast = -1048576.0;

// product of the decays after s up to t, s <= t: the difference of two sums that may both be far
// from 0 (two floats each), then the hardware's power of two (a last place, and the argument's
// rounding: at most 0.4 2^-24 of 1)
__device__ __forceinline__ float pair_decay(float ht, float lt, float hs, float ls)
{
    return __builtin_amdgcn_exp2f((ht - hs) + (lt - ls));
}

// operand f of N parts each, from result tiles a over b
template <int N>
__device__ __forceinline__ void store_frag(quad* to, int f, int lane, f32x4 a, f32x4 b)
{
    const Parts<N> s = split<N>(a, b);
#pragma unroll
    for (int k = 0; k < N; ++k) to[(f * N + k) * 64 + lane] = __builtin_bit_cast(quad, s.p[k]);
}

template <int N>
__device__ __forceinline__ Parts<N> load_frag(const quad* from, int f, int lane)
{
    Parts<N> r;
#pragma unroll
    for (int k = 0; k < N; ++k) r.p[k] = __builtin_bit_cast(u32x4, from[(f * N + k) * 64 + lane]);
    return r;
}

// N quads on their way from memory to LDS
template <int N, int THREADS>
struct LinearLoad {
    static constexpr int PER = (N + THREADS - 1) / THREADS;
    quad q[PER];
    __device__ __forceinline__ void load(const quad* from, int tid)
    {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (N % THREADS == 0 || tid + THREADS * i < N) q[i] = from[tid + THREADS * i];
    }
    __device__ __forceinline__ void put(quad* to, int tid) const
    {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (N % THREADS == 0 || tid + THREADS * i < N) to[tid + THREADS * i] = q[i];
    }
};

// a triangular matrix on its way from memory into N parts in LDS
template <int THREADS>
struct HalvesLoad {
    static constexpr int PER = (kHalfQuads + THREADS - 1) / THREADS;
    f32x4 q[PER];
    __device__ __forceinline__ void load(const f32x4* from, int tid)
    {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (kHalfQuads % THREADS == 0 || tid + THREADS * i < kHalfQuads) q[i] = from[tid + THREADS * i];
    }
    template <int N, bool UPPER>
    __device__ __forceinline__ void put(quad* to, int tid) const
    {
        const int w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int h = w + THREADS / 64 * i;
            if (kHalfQuads % THREADS != 0 && h >= kHalves) continue;
            // the half's place among 12, of which two are zero
            const int p = UPPER ? h + (h >= 4) + (h >= 9) : h + (h >= 1) + (h >= 6);
            u32x2* at = reinterpret_cast<u32x2*>(to) + p / 2 * (N * 128) + (p & 1) + 2 * lane;
            f32x4 x = q[i];
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const u32x2 b = pack_bf16x4(x);
                at[k * 128] = b;
                if (k + 1 < N) x -= widen4(b);
            }
        }
    }
};

// the two halves that no load writes
template <int N, bool UPPER>
__device__ __forceinline__ void zero_halves(quad* to, int tid, int threads)
{
    for (int e = tid; e < 2 * N * 64; e += threads) {
        const int p = e < N * 64 ? (UPPER ? 4 : 1) : (UPPER ? 10 : 7), k = e % (N * 64);
        reinterpret_cast<u32x2*>(to)[(size_t)(p / 2 * N * 64 + k) * 2 + (p & 1)] = u32x2{0u, 0u};
    }
}

// A scan's workgroup: CW waves that compute, 16 columns of values each, and as many that load;
// four waves that do both where registers do not allow eight, and in the backward pass (BACK), whose
// triangular operands then come in parts from memory (both scans at 8 x 12 x 2048 tokens of 64
// features 133 us so, 188 us with waves apart; the whole forward call at 1 x 32 x 32768 694 us with
// waves apart, 838 us with four that do both).
template <typename TIO, int DK, int CW, bool BACK>
constexpr bool kApart = CW == 2 || (!BACK && sizeof(TIO) == 2 && DK <= 64);
template <typename TIO, int DK, int CW, bool BACK>
constexpr int kScanThreads = 64 * CW * (kApart<TIO, DK, CW, BACK> ? 2 : 1);

// What it needs of a chunk: keys, queries, its columns of V or dZ, operands of S (3 parts) and
// P (NP of them), eta, start and end of the tokens.
template <typename TIO, int DK, int NP, bool Q, int CW>
struct ChunkTiles {
    Tile<TIO, DK> k;
    Tile<TIO, Q ? DK : kGran<TIO>> q;
    Tile<TIO, 16 * CW> v;
    quad s[3 * kFragQuads], p[NP ? NP * kFragQuads : 1];
    float eta[kChunk], start[kChunk], end[kChunk];
};

// the same on its way, in the loading waves' registers
template <typename TIO, int DK, int NP, bool Q, bool UPPER, int CW, bool PARTS>
struct ChunkLoad {
    TileLoad<TIO, DK, 64 * CW> k, q;
    TileLoad<TIO, 16 * CW, 64 * CW> v;
    typename std::conditional<PARTS, LinearLoad<3 * kFragQuads, 64 * CW>, HalvesLoad<64 * CW>>::type s, p;
    LinearLoad<3 * kChunk / 4, 64 * CW> rec;
    __device__ __forceinline__ void load(const Rows<const TIO>& K, const Rows<const TIO>& Qr,
                                         const Rows<const TIO>& V, const f32x4* S, const f32x4* P,
                                         const Record* r, int t0, int T, int dk, int dv, int first,
                                         bool whole_k, bool whole_v, int tid)
    {
        if (whole_k && whole_v && dk == DK && first + 16 * CW <= dv && t0 + kChunk <= T) {
            k.load_inside(K, t0, tid);
            if constexpr (Q) q.load_inside(Qr, t0, tid);
            v.load_inside(V, t0, tid, first);
        } else {
            k.load(K, t0, T, dk, whole_k, tid);
            if constexpr (Q) q.load(Qr, t0, T, dk, whole_k, tid);
            v.load(V, t0, T, dv, whole_v, tid, first);
        }
        if constexpr (PARTS) {
            s.load(reinterpret_cast<const quad*>(S), tid);
            if constexpr (NP > 0) p.load(reinterpret_cast<const quad*>(P), tid);
        } else {
            s.load(S, tid);
            if constexpr (NP > 0) p.load(P, tid);
        }
        rec.load(reinterpret_cast<const quad*>(r->eta), tid);   // (eta, start and end: one after the other)
    }
    __device__ __forceinline__ void put(ChunkTiles<TIO, DK, NP, Q, CW>& to, int tid) const
    {
        k.put(to.k, tid);
        if constexpr (Q) q.put(to.q, tid);
        v.put(to.v, tid);
        if constexpr (PARTS) {
            s.put(to.s, tid);
            if constexpr (NP > 0) p.put(to.p, tid);
        } else {
            s.template put<3, UPPER>(to.s, tid);
            if constexpr (NP > 0) p.template put<NP, UPPER>(to.p, tid);
        }
        rec.put(reinterpret_cast<quad*>(to.eta), tid);
    }
};

// LDS reads stay before it: operands are read a product ahead of the one that takes them (a wave
// has its SIMD to itself, so nothing else covers a read's latency)
__device__ __forceinline__ void reads_before() { asm volatile("" ::: "memory"); }

// as many buffers of a chunk as LDS holds, up to two
template <typename TILES> constexpr int kBuffers = 2 * sizeof(TILES) <= 160 * 1024 ? 2 : 1;

template <int N>
__device__ __forceinline__ f32x4 widen_parts(const Parts<N>& x, bool upper)
{
    f32x4 r = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = N - 1; k >= 0; --k) r += widen4(upper ? hi_half(x.p[k]) : lo_half(x.p[k]));
    return r;
}

// ---- one element of the I/O type at CL positions ----------------------------
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_bits_to_f32(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v)
{
    *p = (uint16_t)(pack_bf16x2(v, 0.f) & 0xffffu);
}

// columns f .. f + 3 of a row of d (`fours`: d is a multiple of 4)
template <typename TIO>
__device__ __forceinline__ void store4(TIO* row, int f, int d, bool fours, f32x4 x)
{
    if (fours) {
        if (f < d) {
            if constexpr (sizeof(TIO) == 2) *reinterpret_cast<u32x2*>(row + f) = pack_bf16x4(x);
            else *reinterpret_cast<f32x4*>(row + f) = x;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (f + e < d) store1(row + f + e, x[e]);
    }
}

template <typename TIO>
__device__ __forceinline__ f32x4 load4(const TIO* row, int f, int d, bool fours)
{
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
    if (fours) {
        if (f < d) {
            if constexpr (sizeof(TIO) == 2) x = widen4(*reinterpret_cast<const u32x2*>(row + f));
            else x = *reinterpret_cast<const f32x4*>(row + f);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (f + e < d) x[e] = load1(row + f + e);
    }
    return x;
}

// state [dv, dk] fp32, row `col`, features 16 m + 4 g + v
__device__ __forceinline__ f32x4 load_state(const float* W, int col, int f, int dv, int dk)
{
    f32x4 r = {0.f, 0.f, 0.f, 0.f};
    if (!W || col >= dv) return r;
#pragma unroll
    for (int v = 0; v < 4; ++v)
        if (f + v < dk) r[v] = W[(size_t)col * dk + f + v];
    return r;
}

__device__ __forceinline__ void store_state(float* W, int col, int f, int dv, int dk, f32x4 r)
{
    if (!W || col >= dv) return;
#pragma unroll
    for (int v = 0; v < 4; ++v)
        if (f + v < dk) W[(size_t)col * dk + f + v] = r[v];
}

}  // namespace ttt
