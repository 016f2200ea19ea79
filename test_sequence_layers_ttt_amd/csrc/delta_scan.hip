// The gated delta rule's scans over the chunks: forward, and from the last chunk to the first.
// (delta_common.h has the formulas.)
//
// A wave keeps W^T (or D^T) for 16 columns of values in fp32 registers, since columns never meet:
// the result tiles of one product are, as they lie in registers, operands of the next, and only
// what all waves need goes through LDS.  A workgroup has 32 or 64 columns of a head.  A chunk's data
// is loaded to registers one or two chunks ahead and goes to the other LDS buffer while this one is
// worked on: one barrier a chunk.  What bounds a chunk (64 features: 2.7 us with 32 columns and the
// card half empty, 4.1 us with 64 and the card full) is that each computing wave reads every operand
// from LDS for its own 16 columns (62 KB), and its 500 vector instructions, most of which split
// operands into parts, next to 144 matrix products of 16 cycles.
//
// The reverse scan needs nothing of the forward one, so in a backward pass both run at once.
// Where there are too few heads for the card, each sequence is cut into segments.  First the
// segments' ends are found from a start of zero, together with what becomes of a unit matrix
// (the segment's transition: V = 0, the features' unit vectors as rows of the state); a chain of
// small products then gives every segment its start; and all segments run again from there.
#include <algorithm>

#include "delta_common.h"

namespace ttt {
namespace {

// what a scan leaves: Z, or states and U (or D and F) for the gradients, or its last state alone
enum { kRead, kSave, kEnd };

template <int N>
__device__ __forceinline__ void store_plane(float* X, int ld, int col, int g, const f32x4 (&x)[N])
{
#pragma unroll
    for (int m = 0; m < N; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) X[(size_t)(16 * m + 4 * g + e) * ld + col] = x[m][e];
}

template <int N>
__device__ __forceinline__ void load_plane(const float* X, int ld, int col, int g, f32x4 (&x)[N])
{
#pragma unroll
    for (int m = 0; m < N; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[m][e] = X[(size_t)(16 * m + 4 * g + e) * ld + col];
}

// a workgroup's share: 16 CW columns from `first` of one head's segment
struct Share {
    int local, segment, first;
};

// where a segment's first state lies: the end of the one before it; W0's copy in the last place
__device__ __forceinline__ float* start_of(const DeltaPass& a, int local, int segment, int DK)
{
    return a.ends + ((size_t)local * a.cut.segments + (segment ? segment - 1 : a.cut.segments - 1)) * DK * a.dvp;
}

// Z comes out with its columns down the lanes (operands the other way round): 8-byte stores.
template <typename TIO, int DK, int KEEP, int CW, bool BACK>
struct Forward {
    // parts of P: fp32 products behind a bf16 Z too (two parts: 111 us for 119 at 8 x 12 x 2048)
    static constexpr int NZ = KEEP == kRead ? 3 : 0;
    typedef ChunkTiles<TIO, DK, NZ, KEEP == kRead, CW> Tiles;
    static constexpr int NB = kBuffers<Tiles>;
    static constexpr bool APART = kApart<TIO, DK, CW, BACK>, PARTS = BACK && CW == 4;
    static constexpr size_t LOWER = PARTS ? 3 * kFragQuads : kHalfQuads;   // of 16 bytes, a chunk's S

    // `unit`: V = 0 and a unit matrix for the start, columns are features
    static __device__ __forceinline__ void run(const DeltaPass& a, Tiles* tiles, Share s, bool unit)
    {
        constexpr int M = DK / 16, J = DK / 32;
        const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, g = lane >> 4;
        const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int local = s.local, head = a.head0 + local, first = s.first;
        const int b = head / a.f.H, h = head % a.f.H, hk = h / (a.f.H / a.f.Hk);
        const int T = a.f.T, dk = a.f.dk, dv = a.f.dv;
        const int col = first + 16 * w + c;
        const bool works = first + 16 * w < (unit ? DK : a.dvp);
        const bool whole_k = dk % kGran<TIO> == 0, whole_v = dv % kGran<TIO> == 0, fours = dv % 4 == 0;
        const Rows<const TIO> K((const TIO*)a.f.K, b, hk, a.f.Hk, T, dk, a.f.tokens_first);
        const Rows<const TIO> Q((const TIO*)a.f.Q, b, hk, a.f.Hk, T, dk, a.f.tokens_first);
        const Rows<const TIO> V((const TIO*)a.f.V, b, h, a.f.H, T, dv, a.f.tokens_first);
        const Rows<TIO> Z((TIO*)a.f.Z, b, h, a.f.H, T, dv, a.f.tokens_first);
        const size_t state = (size_t)head * dv * dk, unit0 = (size_t)local * a.chunks;
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        const int begin = s.segment * a.cut.chunks;
        const int stop = begin + a.cut.chunks < a.chunks ? begin + a.cut.chunks : a.chunks;

        for (int e = 0; !PARTS && e < NB; ++e) {
            zero_halves<3, false>(tiles[e].s, tid, kScanThreads<TIO, DK, CW, BACK>);
            if constexpr (NZ > 0) zero_halves<NZ, false>(tiles[e].p, tid, kScanThreads<TIO, DK, CW, BACK>);
        }
        const int id = APART ? tid - 64 * CW : tid;
        typedef ChunkLoad<TIO, DK, NZ, KEEP == kRead, false, CW, PARTS> Load;
        auto fetch = [&](Load& l, int n) {
            const size_t at = unit0 + n;
            l.load(K, Q, V, a.S + at * LOWER, a.P + at * kHalfQuads, a.records + at,
                   n * kChunk, T, dk, dv, first, whole_k, whole_v, id);
        };
        auto put = [&](const Load& l, int n) { l.put(tiles[NB == 2 ? (n - begin) & 1 : 0], id); };
        Load next;
        if (APART && w >= CW) {
            fetch(next, begin);
            put(next, begin);
            if (begin + 1 < stop) fetch(next, begin + 1);
            __syncthreads();
            for (int n = begin; n < stop; ++n) {
                if constexpr (NB == 1) __syncthreads();
                if (n + 1 < stop) put(next, n + 1);
                if (n + 2 < stop) fetch(next, n + 2);
                __syncthreads();
            }
            return;
        }
        if constexpr (!APART) fetch(next, begin);
        f32x4 W[M];
#pragma unroll
        for (int m = 0; m < M; ++m) W[m] = zero;
        if (unit) {
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) W[m][e] = 16 * m + 4 * g + e == col ? 1.f : 0.f;
        } else if (s.segment == 0 && (KEEP == kEnd || a.cut.segments == 1)) {
            if (a.f.W0)
#pragma unroll
                for (int m = 0; m < M; ++m) W[m] = load_state(a.f.W0 + state, col, 16 * m + 4 * g, dv, dk);
            // the second run takes the first state from here: the last segment may write W_out at its place
            if (KEEP == kEnd && works) store_plane(start_of(a, local, 0, DK), a.dvp, col, g, W);
        } else if (KEEP != kEnd && works) {
            load_plane(start_of(a, local, s.segment, DK), a.dvp, col, g, W);
        }
        if constexpr (!APART) put(next, begin);
        __syncthreads();

        for (int n = begin; n < stop; ++n) {
            const Tiles& t = tiles[NB == 2 ? (n - begin) & 1 : 0];
            if (!APART && n + 1 < stop) fetch(next, n + 1);
            if (works) {
                typedef Parts<kParts<TIO>> In;
                In kt[J][4], vp[2];
                Parts<3> S[kFrags], x[2];
                f32x4 r[4], z[4], eta[4], start[4], ends[4];
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) kt[j][i] = by_token(t.k, i, j, lane);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    start[i] = *reinterpret_cast<const f32x4*>(t.start + 16 * i + 4 * g);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    vp[j] = by_feature(t.v, w, j, lane);
                }
#pragma unroll
                for (int f = 0; f < kFrags; ++f) S[f] = load_frag<3>(t.s, f, lane);
                const float all = t.start[kChunk - 1];
                reads_before();

#pragma unroll
                for (int i = 0; i < 4; ++i) r[i] = z[i] = zero;
                Parts<3> wp[J];
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    wp[j] = split<3>(W[2 * j], W[2 * j + 1]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) r[i] = mma(kt[j][i], wp[j], r[i]);
                }
                if constexpr (KEEP == kSave) store_plane(a.states + (unit0 + n) * DK * a.dvp, a.dvp, col, g, W);
#pragma unroll
                for (int i = 0; i < 4; ++i) eta[i] = *reinterpret_cast<const f32x4*>(t.eta + 16 * i + 4 * g);
                In kf[M][2];
#pragma unroll
                for (int m = 0; m < M; ++m)
#pragma unroll
                    for (int j = 0; j < 2; ++j) kf[m][j] = by_feature(t.k, m, j, lane);
                reads_before();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    r[i] *= -start[i];
                    if (!unit) r[i] += widen_parts(vp[i / 2], i & 1);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    x[j] = split<3>(-(eta[2 * j] * r[2 * j]), -(eta[2 * j + 1] * r[2 * j + 1]));
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 2 * j; i < 4; ++i) r[i] = mma(S[frag_lower(i, j)], x[j], r[i]);
#pragma unroll
                for (int i = 0; i < 4; ++i) ends[i] = *reinterpret_cast<const f32x4*>(t.end + 16 * i + 4 * g);
                In qt[J][4];
                Parts<NZ ? NZ : 1> P[kFrags], u[2];
                if constexpr (KEEP == kRead) {
#pragma unroll
                    for (int j = 0; j < J; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) qt[j][i] = by_token(t.q, i, j, lane);
#pragma unroll
                    for (int f = 0; f < kFrags; ++f) P[f] = load_frag<NZ>(t.p, f, lane);
                    reads_before();
                }
                if constexpr (KEEP == kSave) store_plane(a.U + (unit0 + n) * kChunk * a.dvp, a.dvp, col, g, r);
#pragma unroll
                for (int i = 0; i < 4; ++i) r[i] *= eta[i];
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    x[j] = split<3>(ends[2 * j] * r[2 * j], ends[2 * j + 1] * r[2 * j + 1]);
#pragma unroll
                for (int m = 0; m < M; ++m) W[m] *= all;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int m = 0; m < M; ++m) W[m] = mma(kf[m][j], x[j], W[m]);
                if constexpr (KEEP == kRead) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) u[j] = split<NZ>(r[2 * j], r[2 * j + 1]);
#pragma unroll
                    for (int j = 0; j < J; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) z[i] = mma(wp[j], qt[j][i], z[i]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) z[i] *= t.start[16 * i + c];
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int i = 2 * j; i < 4; ++i) z[i] = mma(u[j], P[frag_lower(i, j)], z[i]);
                    const int token = n * kChunk + c;
                    if (fours && first + 16 * CW <= dv && (n + 1) * kChunk <= T) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            store4(Z.at(token + 16 * i), first + 16 * w + 4 * g, dv, true, z[i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (token + 16 * i < T)
                                store4(Z.at(token + 16 * i), first + 16 * w + 4 * g, dv, fours, z[i]);
                    }
                }
            }
            if constexpr (NB == 1) __syncthreads();
            if (!APART && n + 1 < stop) put(next, n + 1);
            __syncthreads();
        }
        if constexpr (KEEP == kEnd) {
            if (!works) return;
            const size_t at = (size_t)local * a.cut.segments + s.segment;
            if (unit) store_plane(a.transitions + at * DK * DK, DK, col, g, W);
            else store_plane(a.ends + at * DK * a.dvp, a.dvp, col, g, W);
        }
        if constexpr (KEEP == kRead) {
            if (stop == a.chunks && a.f.W_out)
#pragma unroll
                for (int m = 0; m < M; ++m) store_state(a.f.W_out + state, col, 16 * m + 4 * g, dv, dk, W[m]);
        }
    }
};

template <typename TIO, int DK, int KEEP, int CW>
struct Reverse {
    typedef ChunkTiles<TIO, DK, 3, true, CW> Tiles;
    static constexpr int NB = kBuffers<Tiles>;
    static constexpr bool APART = kApart<TIO, DK, CW, true>, PARTS = CW == 4;
    static constexpr size_t UPPER = PARTS ? 3 * kFragQuads : kHalfQuads;

    static __device__ __forceinline__ void run(const DeltaPass& a, const DeltaBwdArgs& o, Tiles* tiles, Share s)
    {
        constexpr int NP = kParts<TIO>, M = DK / 16, J = DK / 32;
        const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, g = lane >> 4;
        const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int local = s.local, head = a.head0 + local, first = s.first;
        const int b = head / a.f.H, h = head % a.f.H, hk = h / (a.f.H / a.f.Hk);
        const int T = a.f.T, dk = a.f.dk, dv = a.f.dv;
        const int col = first + 16 * w + c;
        const bool works = first + 16 * w < a.dvp;
        const bool whole_k = dk % kGran<TIO> == 0, whole_v = dv % kGran<TIO> == 0;
        const Rows<const TIO> K((const TIO*)a.f.K, b, hk, a.f.Hk, T, dk, a.f.tokens_first);
        const Rows<const TIO> Q((const TIO*)a.f.Q, b, hk, a.f.Hk, T, dk, a.f.tokens_first);
        const Rows<const TIO> dZ((const TIO*)o.dZ, b, h, a.f.H, T, dv, a.f.tokens_first);
        const size_t state = (size_t)head * dv * dk, unit0 = (size_t)local * a.chunks;
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        const int begin = s.segment * a.cut.chunks;
        const int last = (begin + a.cut.chunks < a.chunks ? begin + a.cut.chunks : a.chunks) - 1;

        for (int e = 0; !PARTS && e < NB; ++e) {
            zero_halves<3, true>(tiles[e].s, tid, kScanThreads<TIO, DK, CW, true>);
            zero_halves<3, true>(tiles[e].p, tid, kScanThreads<TIO, DK, CW, true>);
        }
        const int id = APART ? tid - 64 * CW : tid;
        typedef ChunkLoad<TIO, DK, 3, true, true, CW, PARTS> Load;
        auto fetch = [&](Load& l, int n) {
            const size_t at = unit0 + n;
            l.load(K, Q, dZ, a.St + at * UPPER, a.P + at * UPPER, a.records + at,
                   n * kChunk, T, dk, dv, first, whole_k, whole_v, id);
        };
        auto put = [&](const Load& l, int n) { l.put(tiles[NB == 2 ? n & 1 : 0], id); };
        Load next;
        if (APART && w >= CW) {
            fetch(next, last);
            put(next, last);
            if (last > begin) fetch(next, last - 1);
            __syncthreads();
            for (int n = last; n >= begin; --n) {
                if constexpr (NB == 1) __syncthreads();
                if (n > begin) put(next, n - 1);
                if (n > begin + 1) fetch(next, n - 2);
                __syncthreads();
            }
            return;
        }
        if constexpr (!APART) fetch(next, last);
        f32x4 D[M];
#pragma unroll
        for (int m = 0; m < M; ++m) D[m] = zero;
        if (last == a.chunks - 1) {
            if (o.dW_T)
#pragma unroll
                for (int m = 0; m < M; ++m) D[m] = load_state(o.dW_T + state, col, 16 * m + 4 * g, dv, dk);
        } else if (KEEP != kEnd && works) {
            load_plane(a.ends_back + ((size_t)local * a.cut.segments + s.segment + 1) * DK * a.dvp, a.dvp, col, g, D);
        }
        if constexpr (!APART) put(next, last);
        __syncthreads();

        for (int n = last; n >= begin; --n) {
            const Tiles& t = tiles[NB == 2 ? n & 1 : 0];
            if (!APART && n > begin) fetch(next, n - 1);
            if (works) {
                const size_t unit = unit0 + n;
                typedef Parts<NP> In;
                In kt[J][4], zp[2];
                Parts<3> P[kFrags], S[kFrags], x[2];
                f32x4 f[4], kd[4], z[4], eta[4], start[4], ends[4];
#pragma unroll
                for (int j = 0; j < 2; ++j) zp[j] = by_feature(t.v, w, j, lane);
#pragma unroll
                for (int e = 0; e < kFrags; ++e) P[e] = load_frag<3>(t.p, e, lane);
                const float all = t.start[kChunk - 1];
                reads_before();
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) kt[j][i] = by_token(t.k, i, j, lane);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    ends[i] = *reinterpret_cast<const f32x4*>(t.end + 16 * i + 4 * g);
                    eta[i] = *reinterpret_cast<const f32x4*>(t.eta + 16 * i + 4 * g);
                }
                reads_before();

                if constexpr (KEEP == kSave) store_plane(a.cotangents + unit * DK * a.dvp, a.dvp, col, g, D);
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] = kd[i] = zero;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < 2 * j + 2; ++i) f[i] = mma(P[frag_upper(i, j)], zp[j], f[i]);
#pragma unroll
                for (int e = 0; e < kFrags; ++e) S[e] = load_frag<3>(t.s, e, lane);
                reads_before();
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const Parts<3> dp = split<3>(D[2 * j], D[2 * j + 1]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) kd[i] = mma(kt[j][i], dp, kd[i]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] += ends[i] * kd[i];
                In kf[M][2];
#pragma unroll
                for (int m = 0; m < M; ++m)
#pragma unroll
                    for (int j = 0; j < 2; ++j) kf[m][j] = by_feature(t.k, m, j, lane);
                reads_before();
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    x[j] = split<3>(-(eta[2 * j] * f[2 * j]), -(eta[2 * j + 1] * f[2 * j + 1]));
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < 2 * j + 2; ++i) f[i] = mma(S[frag_upper(i, j)], x[j], f[i]);
#pragma unroll
                for (int i = 0; i < 4; ++i) start[i] = *reinterpret_cast<const f32x4*>(t.start + 16 * i + 4 * g);
                In qf[M][2];
#pragma unroll
                for (int m = 0; m < M; ++m)
#pragma unroll
                    for (int j = 0; j < 2; ++j) qf[m][j] = by_feature(t.q, m, j, lane);
                reads_before();

                if constexpr (KEEP == kSave) store_plane(a.F + unit * kChunk * a.dvp, a.dvp, col, g, f);
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] *= -(start[i] * eta[i]);
#pragma unroll
                for (int j = 0; j < 2; ++j) x[j] = split<3>(f[2 * j], f[2 * j + 1]);
#pragma unroll
                for (int m = 0; m < M; ++m) D[m] *= all;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int m = 0; m < M; ++m) D[m] = mma(kf[m][j], x[j], D[m]);
#pragma unroll
                for (int i = 0; i < 4; ++i) z[i] = start[i] * widen_parts(zp[i / 2], i & 1);
#pragma unroll
                for (int j = 0; j < 2; ++j) x[j] = split<3>(z[2 * j], z[2 * j + 1]);
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int m = 0; m < M; ++m) D[m] = mma(qf[m][j], x[j], D[m]);
            }
            if constexpr (NB == 1) __syncthreads();
            if (!APART && n > begin) put(next, n - 1);
            __syncthreads();
        }
        if constexpr (KEEP == kEnd) {
            if (works) store_plane(a.ends_back + ((size_t)local * a.cut.segments + s.segment) * DK * a.dvp, a.dvp, col, g, D);
        } else if (begin == 0 && o.dW0) {
#pragma unroll
            for (int m = 0; m < M; ++m) store_state(o.dW0 + state, col, 16 * m + 4 * g, dv, dk, D[m]);
        }
    }
};

// column parts of a head's segment, the transition's among them
template <int CW>
__host__ __device__ __forceinline__ int widest(const DeltaPass& a, int DK)
{
    return ((a.cut.segments > 1 && DK > a.dvp ? DK : a.dvp) + 16 * CW - 1) / (16 * CW);
}

// One launch of all shares of a kind, the column parts of a segment on one XCD (they share its
// keys and operands in L2).  Forward alone: kRead over all segments, or the ends of
// all but the last and the transitions of all but the first and last.  With the backward pass:
// kSave of both scans, or all three kinds of ends.
template <typename TIO, int DK, int KEEP, int CW>
__global__ void __launch_bounds__((kScanThreads<TIO, DK, CW, false>), KEEP == kEnd && CW == 2 && DK <= 64 && sizeof(TIO) == 2 ? 2 : 1)
delta_scan_kernel(DeltaPass a)
{
    typedef typename Forward<TIO, DK, KEEP, CW, false>::Tiles Tiles;
    __shared__ __align__(16) Tiles tiles[kBuffers<Tiles>];
    const int ends = KEEP == kEnd ? a.cut.segments - 1 : a.cut.segments;
    const int each = ends + (KEEP == kEnd ? a.cut.segments - 2 : 0);
    int id, part;
    xcd_unit_part(blockIdx.x, widest<CW>(a, DK), id, part);
    const int local = id / each, k = id % each;
    const bool unit = k >= ends;
    const Share s = {local, unit ? 1 + k - ends : k, 16 * CW * part};
    if (local >= a.heads || s.first >= (unit ? DK : a.dvp)) return;
    Forward<TIO, DK, KEEP, CW, false>::run(a, tiles, s, unit);
}

template <typename TIO, int DK, int KEEP, int CW>
__global__ void __launch_bounds__((kScanThreads<TIO, DK, CW, true>), 1) delta_scans_kernel(DeltaPass a, DeltaBwdArgs o)
{
    typedef typename Forward<TIO, DK, KEEP, CW, true>::Tiles There;
    typedef typename Reverse<TIO, DK, KEEP, CW>::Tiles Back;
    constexpr size_t room = kBuffers<There> * sizeof(There) > kBuffers<Back> * sizeof(Back)
                                ? kBuffers<There> * sizeof(There) : kBuffers<Back> * sizeof(Back);
    __shared__ __align__(16) char tiles[room];
    const int ends = KEEP == kEnd ? a.cut.segments - 1 : a.cut.segments;
    const int each = 2 * ends + (KEEP == kEnd ? a.cut.segments - 2 : 0);
    int id, part;
    xcd_unit_part(blockIdx.x, widest<CW>(a, DK), id, part);
    const int local = id / each, k = id % each;
    const bool back = k < ends, unit = k >= 2 * ends;
    const Share s = {local, back ? k + (KEEP == kEnd ? 1 : 0) : unit ? 1 + k - 2 * ends : k - ends,
                     16 * CW * part};
    if (local >= a.heads || s.first >= (unit ? DK : a.dvp)) return;
    if (back) {
        Reverse<TIO, DK, KEEP, CW>::run(a, o, (Back*)tiles, s);
        return;
    }
    Forward<TIO, DK, KEEP, CW, true>::run(a, (There*)tiles, s, unit);
}

// The segments' ends, one after the other: with X^T_s the state that segment s - 1 leaves (its end
// from the true start) and A the transition as it was stored, X^T_(s+1) = A X^T_s + end_s; backward
// by A^T.  One workgroup for 16 columns of a head: a wave has every fourth tile of features, the
// columns go round by LDS, and the next transition is on its way while this one is multiplied.
template <int DK>
__global__ void __launch_bounds__(256) delta_join_kernel(DeltaPass a)
{
    constexpr int M = DK / 16, J = DK / 32, MW = (M + 3) / 4, LD = 17;
    __shared__ float X[DK * LD];
    const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, g = lane >> 4, parts = a.dvp / 16;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6), segments = a.cut.segments;
    const bool back = blockIdx.x >= (unsigned)(a.heads * parts);
    const int id = blockIdx.x % (a.heads * parts), local = id / parts, col = 16 * (id % parts) + c;
    const size_t plane = (size_t)DK * a.dvp;
    float* ends = (back ? a.ends_back : a.ends) + (size_t)local * segments * plane;
    f32x4 A[MW][J][2], E[MW];
    auto at = [&](int k) { return back ? segments - 1 - k : k; };
    auto fetch = [&](int s) {
        const float* T = a.transitions + ((size_t)local * segments + s) * DK * DK;
#pragma unroll
        for (int i = 0; i < MW; ++i) {
            const int m = w + 4 * i;
            if (m >= M) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) E[i][e] = ends[s * plane + (size_t)(16 * m + 4 * g + e) * a.dvp + col];
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int f = 32 * j + 16 * h + 4 * g;
                    if (back) {
                        const float* p = T + (size_t)f * DK + 16 * m + c;
                        A[i][j][h] = f32x4{p[0], p[DK], p[2 * DK], p[3 * DK]};
                    } else {
                        A[i][j][h] = *reinterpret_cast<const f32x4*>(T + (size_t)(16 * m + c) * DK + f);
                    }
                }
        }
    };
    for (int e = tid; e < DK * 16; e += 256)
        X[e / 16 * LD + e % 16] = ends[at(0) * plane + (size_t)(e / 16) * a.dvp + 16 * (id % parts) + e % 16];
    fetch(at(1));
    for (int k = 1; k < segments - 1; ++k) {
        __syncthreads();
        Parts<3> x[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const float* p = X + (32 * j + 4 * g) * LD + c;
            const f32x4 lo = {p[0], p[LD], p[2 * LD], p[3 * LD]};
            p += 16 * LD;
            x[j] = split<3>(lo, f32x4{p[0], p[LD], p[2 * LD], p[3 * LD]});
        }
        f32x4 y[MW];
#pragma unroll
        for (int i = 0; i < MW; ++i) {
            y[i] = E[i];
            if (w + 4 * i >= M) continue;
#pragma unroll
            for (int j = 0; j < J; ++j) y[i] = mma(split<3>(A[i][j][0], A[i][j][1]), x[j], y[i]);
        }
        if (k + 1 < segments - 1) fetch(at(k + 1));
        __syncthreads();
#pragma unroll
        for (int i = 0; i < MW; ++i) {
            const int m = w + 4 * i;
            if (m >= M) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                X[(16 * m + 4 * g + e) * LD + c] = y[i][e];
                ends[at(k) * plane + (size_t)(16 * m + 4 * g + e) * a.dvp + col] = y[i][e];
            }
        }
    }
}

template <typename TIO, int DK, int KEEP, int CW>
hipError_t launch(const DeltaPass& p, const DeltaBwdArgs* o, hipStream_t s)
{
    const size_t ends = KEEP == kEnd ? p.cut.segments - 1 : p.cut.segments;
    const size_t each = (o ? 2 : 1) * ends + (KEEP == kEnd ? p.cut.segments - 2 : 0);
    const unsigned grid = (unsigned)((p.heads * each + 7) / 8 * 8 * widest<CW>(p, DK));
    if constexpr (KEEP != kSave) {
        if (!o) {
            delta_scan_kernel<TIO, DK, KEEP, CW><<<grid, kScanThreads<TIO, DK, CW, false>, 0, s>>>(p);
            return hipGetLastError();
        }
    }
    if constexpr (KEEP != kRead)
        delta_scans_kernel<TIO, DK, KEEP, CW><<<grid, kScanThreads<TIO, DK, CW, true>, 0, s>>>(p, *o);
    return hipGetLastError();
}

template <typename TIO, int DK, int CW>
hipError_t scans_as(const DeltaPass& p, const DeltaBwdArgs* o, hipStream_t s)
{
    if (p.cut.segments > 1) {
        hipError_t e = launch<TIO, DK, kEnd, CW>(p, o, s);
        if (e != hipSuccess) return e;
        const unsigned grid = (unsigned)(p.heads * (p.dvp / 16)) * (o ? 2 : 1);
        delta_join_kernel<DK><<<grid, 256, 0, s>>>(p);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return o ? launch<TIO, DK, kSave, CW>(p, o, s) : launch<TIO, DK, kRead, CW>(p, o, s);
}

template <typename TIO, int DK>
hipError_t scans(const DeltaPass& p, const DeltaBwdArgs* o, hipStream_t s)
{
    return p.cut.narrow ? scans_as<TIO, DK, 2>(p, o, s) : scans_as<TIO, DK, 4>(p, o, s);
}

}  // namespace

hipError_t launch_delta_scans(const DeltaPass& p, const DeltaBwdArgs* o, hipStream_t s)
{
    const int DK = delta_padded_dk(p.f.dk);
    if (p.f.bf16)
        return DK == 32 ? scans<uint16_t, 32>(p, o, s)
             : DK == 64 ? scans<uint16_t, 64>(p, o, s) : scans<uint16_t, 128>(p, o, s);
    return DK == 32 ? scans<float, 32>(p, o, s)
         : DK == 64 ? scans<float, 64>(p, o, s) : scans<float, 128>(p, o, s);
}

// How a sequence is cut: into how many segments, and whether a workgroup takes 32 columns or 64.
// One filling of the 256 compute units takes its chunks times (8 x 12 heads of 64
// features, us a chunk) 4.0 with 64 columns and 2.6 with 32, where the workgroup's waves meet less
// in LDS; where only ends are found 2.3 and 1.8.  The ends and the second run cost 2 / segments of
// the sequence where they fit at once, so segments pay from few heads on (1 x 32 heads of 64
// features, 32768 tokens: the whole call 2.05 ms, in 8 segments 0.70 ms).
DeltaCut delta_cut(int heads, int chunks, int dv, int dk, bool backward)
{
    const long long sides = backward ? 2 : 1, cus = 256;
    auto fillings = [&](long long shares) { return (heads * shares + cus - 1) / cus; };
    DeltaCut best = {1, chunks, false};
    long long least = -1;
    for (int narrow = 0; narrow < 2; ++narrow) {
        const int columns = narrow ? 32 : 64;
        const long long parts = (dv + columns - 1) / columns;
        const long long wide = (delta_padded_dk(dk) + columns - 1) / columns;
        for (int n = 1; n <= 32 && (n == 1 || chunks / n >= 4); ++n) {
            if (n == 2) continue;                      // (the ends alone are half of it then)
            const int each = (chunks + n - 1) / n;
            if ((chunks + each - 1) / each != n) continue;   // (no empty segments)
            long long cost = fillings(sides * n * parts) * (narrow ? 26 : 40) * each;
            // the ends, and joins of about a chunk's time
            if (n > 1)
                cost += fillings(sides * (n - 1) * parts + (n - 2) * wide) * (narrow ? 18 : 23) * each + 40 * n;
            if (least < 0 || cost < least) {
                least = cost;
                best = {n, each, narrow != 0};
            }
        }
    }
    return best;
}

}  // namespace ttt
