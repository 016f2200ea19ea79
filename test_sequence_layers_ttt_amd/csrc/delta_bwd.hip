// Gated delta rule: backward pass by chunks of 64 tokens (delta_common.h has the formulas).
//
// The forward scan is run again and keeps every chunk's first state and U, while a second scan
// carries the state's gradient D from the last chunk to the first; the gradients of keys, queries,
// step sizes and decays then follow chunk by chunk, all chunks at once.  Every sum has a fixed order:
// the same bits on every call.
//
// The decay's gradient is the product of D and the state across the token, that is of all
// that is read from token t on with all that was written before it.  Within a chunk, with the
// gradients dP and dL that are left of the pairs (s reads what r wrote) after their decays,
//   dg_t = sum over s >= t > r of (dP_sr q_s.k_r + dL_sr k_s.k_r)        (pairs across t)
//        + sum over s >= t of what s reads of the chunk's first state
//        + sum over r < t of what is left of r's write at the chunk's end
//        + start_C <D, W>.
// Every term has the decay of t in it, so a strong one makes all of them small: the sum has its
// own digits.  (A difference of sums over whole rows and columns of the pairs keeps only the
// digits of what does not cross t: all that dg_t is after a decay of exp(-16).)
#include <algorithm>

#include "delta_common.h"

namespace ttt {
namespace {

struct BwdPass {
    DeltaPass p;
    DeltaBwdArgs a;
    float *dK, *dQ;          // [heads][chunks][64][DK] where heads share keys, else nullptr
};

// ---- gradients of a chunk ------------------------------------------------------------
// One workgroup of four waves per chunk and head of values (where heads share keys, dQ and dK
// go to fp32 planes that another kernel adds up).  Wave w has the gradients of tokens
// 16 w .. 16 w + 15, transposed: tokens in the lanes, features down the result tiles.  The 64 x 64
// products over the columns (dZ u^T and dV u^T, both ways up) come out as operands of what
// follows, as they lie.
// The planes that the scans left (U, F, and the states and their gradients) are taken 32
// columns at a time: each is loaded once, split into parts by the wave that loads it and
// handed to the others as operands in LDS, while the next 32 columns are on their way (8 x 12 x
// 2048 tokens of 64 features 124 us, 398 us when every wave read and split the planes by itself;
// 134 us with the decays' gradients from the pairs across each token).
template <typename TIO, int DK>
__global__ void __launch_bounds__(256) delta_grads_kernel(BwdPass q_)
{
    constexpr int NP = kParts<TIO>, M = DK / 16, MW = (M + 3) / 4;
    const DeltaPass& a = q_.p;
    __shared__ __align__(16) Tile<TIO, DK> tk;
    __shared__ __align__(16) Tile<TIO, DK> tq;
    __shared__ __align__(16) quad fu[4 * 3 * 64], fv[4 * 3 * 64], fz[4 * NP * 64], fw[M * 3 * 64], fd[M * 3 * 64];
    __shared__ double across[4];
    __shared__ __align__(16) float hi[kChunk], lo[kChunk];
    // of dg: what a token reads of the first state, leaves at the end, reads of tiles before its
    // own; pairs across it in its own tile; what the tiles after it read of it, a row for each
    __shared__ float reads[kChunk], leaves[kChunk], rows[kChunk], inner[kChunk];
    __shared__ __align__(16) float later[4][kChunk];

    const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, g = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int chunk = blockIdx.x % a.chunks, local = blockIdx.x / a.chunks, head = a.head0 + local;
    const int b = head / a.f.H, h = head % a.f.H, hk = h / (a.f.H / a.f.Hk);
    const size_t unit = (size_t)local * a.chunks + chunk;
    const int T = a.f.T, dk = a.f.dk, dv = a.f.dv, dvp = a.dvp, t0 = chunk * kChunk;
    const int own = 16 * w + c, steps = dvp / 32;
    const bool whole = dk % kGran<TIO> == 0, fours = dv % 4 == 0, inside = t0 + own < T;
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};

    // 32 columns on their way: this wave's rows of U, F and dZ, and of the states' tiles w, w + 4
    f32x4 lu[2], lf[2], lz[2], lw[MW][2], ld[MW][2];
    const Rows<const TIO> dZ((const TIO*)q_.a.dZ, b, h, a.f.H, T, dv, a.f.tokens_first);
    auto fetch = [&](int j) {
        const size_t at = 32 * j + 4 * g;
        const float* u = a.U + (unit * kChunk + own) * dvp + at;
        const float* f = a.F + (unit * kChunk + own) * dvp + at;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            lu[e] = *reinterpret_cast<const f32x4*>(u + 16 * e);
            lf[e] = *reinterpret_cast<const f32x4*>(f + 16 * e);
            lz[e] = inside ? load4(dZ.at(t0 + own), 32 * j + 16 * e + 4 * g, dv, fours) : zero;
#pragma unroll
            for (int m = 0; m < MW; ++m)
                if (w + 4 * m < M) {
                    const size_t row = (unit * DK + 16 * (w + 4 * m) + c) * dvp + at + 16 * e;
                    lw[m][e] = *reinterpret_cast<const f32x4*>(a.states + row);
                    ld[m][e] = *reinterpret_cast<const f32x4*>(a.cotangents + row);
                }
        }
    };
    fetch(0);
    {
        TileLoad<TIO, DK> lk, lq;
        const Rows<const TIO> K((const TIO*)a.f.K, b, hk, a.f.Hk, T, dk, a.f.tokens_first);
        const Rows<const TIO> Q((const TIO*)a.f.Q, b, hk, a.f.Hk, T, dk, a.f.tokens_first);
        if (whole && dk == DK && t0 + kChunk <= T) {
            lk.load_inside(K, t0, tid);
            lq.load_inside(Q, t0, tid);
        } else {
            lk.load(K, t0, T, dk, whole, tid);
            lq.load(Q, t0, T, dk, whole, tid);
        }
        lk.put(tk, tid);
        lq.put(tq, tid);
    }
    const Record& rec = a.records[unit];
    const Rows<TIO> dV((TIO*)q_.a.dV, b, h, a.f.H, T, dv, a.f.tokens_first);
    const float eo = rec.eta[own], so = rec.start[own], no = rec.end[own], all = rec.start[kChunk - 1];

    f32x4 p[4], pt[4], l[4], lt[4], aw[M], av[M], ad[M];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = pt[i] = l[i] = lt[i] = zero;
#pragma unroll
    for (int m = 0; m < M; ++m) aw[m] = av[m] = ad[m] = zero;
    float de = 0.f, kept = 0.f;
    for (int j = 0; j < steps; ++j) {
        f32x4 u[2], v[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            u[e] = eo * lu[e];
            v[e] = eo * lf[e];
#pragma unroll
            for (int k = 0; k < 4; ++k) de = fmaf(lu[e][k], lf[e][k], de);
            if (inside) store4(dV.at(t0 + own), 32 * j + 16 * e + 4 * g, dv, fours, v[e]);
        }
        const Parts<3> uo = split<3>(u[0], u[1]), vo = split<3>(v[0], v[1]);
        const Parts<NP> zo = split<NP>(lz[0], lz[1]);
        __syncthreads();               // (the columns before have been read)
        if (j == 0 && tid < kChunk) {
            hi[tid] = rec.hi[tid];
            lo[tid] = rec.lo[tid];
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            fu[(3 * w + k) * 64 + lane] = __builtin_bit_cast(quad, uo.p[k]);
            fv[(3 * w + k) * 64 + lane] = __builtin_bit_cast(quad, vo.p[k]);
        }
#pragma unroll
        for (int k = 0; k < NP; ++k) fz[(NP * w + k) * 64 + lane] = __builtin_bit_cast(quad, zo.p[k]);
#pragma unroll
        for (int m = 0; m < MW; ++m)
            if (w + 4 * m < M) {
                store_frag<3>(fw, w + 4 * m, lane, lw[m][0], lw[m][1]);
                store_frag<3>(fd, w + 4 * m, lane, ld[m][0], ld[m][1]);
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int k = 0; k < 4; ++k) kept = fmaf(lw[m][e][k], ld[m][e][k], kept);
            }
        __syncthreads();
        if (j + 1 < steps) fetch(j + 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i <= w) {
                const Parts<3> x = load_frag<3>(fu, i, lane);
                pt[i] = mma(x, zo, pt[i]);
                lt[i] = mma(x, vo, lt[i]);
            }
            if (i >= w) {
                p[i] = mma(load_frag<NP>(fz, i, lane), uo, p[i]);
                l[i] = mma(load_frag<3>(fv, i, lane), uo, l[i]);
            }
        }
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const Parts<3> s = load_frag<3>(fw, m, lane);
            aw[m] = mma(s, zo, aw[m]);
            av[m] = mma(s, vo, av[m]);
            ad[m] = mma(load_frag<3>(fd, m, lane), uo, ad[m]);
        }
    }
    // pt, lt: rows s, column t = own; p, l: rows t, column s = own
    const float ho = hi[own], loo = lo[own];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f32x4 hr = *reinterpret_cast<const f32x4*>(hi + 16 * i + 4 * g);
        const f32x4 lr = *reinterpret_cast<const f32x4*>(lo + 16 * i + 4 * g);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int row = 16 * i + 4 * g + e;
            if (i <= w) {
                const float d = pair_decay(ho, loo, hr[e], lr[e]);
                pt[i][e] = row <= own ? pt[i][e] * d : 0.f;
                lt[i][e] = row < own ? -lt[i][e] * d : 0.f;
            }
            if (i >= w) {
                const float d = pair_decay(hr[e], lr[e], ho, loo);
                p[i][e] = row >= own ? p[i][e] * d : 0.f;
                l[i][e] = row > own ? -l[i][e] * d : 0.f;
            }
        }
    }
    // pairs (rows r, column s = own) across a token: those that end at s in the tiles of r before
    // its own (row sum), what each r has in this tile of s (column sums), and in the tile on the
    // diagonal, for t = 4 g + e + 1, all r < t <= s
    {
        float row = 0.f;
        if (lane < 16) inner[own] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i > w) continue;
            f32x4 qk = zero, kk = zero;
#pragma unroll
            for (int j = 0; j < DK / 32; ++j) {
                const Parts<NP> r = by_token(tk, i, j, lane);
                qk = mma(r, by_token(tq, w, j, lane), qk);
                kk = mma(r, by_token(tk, w, j, lane), kk);
            }
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[e] = 16 * i + 4 * g + e < own ? fmaf(pt[i][e], qk[e], lt[i][e] * kk[e]) : 0.f;
            if (i < w) {
                row += (x[0] + x[1]) + (x[2] + x[3]);
                row_sum16_n(x);
                if (c == 0) *reinterpret_cast<f32x4*>(later[w] + 16 * i + 4 * g) = f32x4{x[0], x[1], x[2], x[3]};
            } else {
#pragma unroll
                for (int e = 1; e < 4; ++e) x[e] += x[e - 1];
                float all4 = x[3];
#pragma unroll
                for (int o = 16; o < 64; o <<= 1) {
                    const float y = __shfl_up(all4, o, 64);
                    if (lane >= o) all4 += y;
                }
                const float before = __shfl_up(all4, 16, 64);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = 4 * g + e < c ? x[e] + (g ? before : 0.f) : 0.f;
                row_sum16_n(x);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c == 0 && 4 * g + e < 15) inner[16 * w + 4 * g + e + 1] = x[e];
            }
        }
        row += __shfl_xor(row, 16, 64);
        row += __shfl_xor(row, 32, 64);
        if (g == 0) rows[own] = row;
    }
    float wrote = 0.f, read = 0.f;
#pragma unroll
    for (int m = 0; m < M; ++m) {
        aw[m] *= so;
        av[m] *= -so;
        ad[m] *= no;
        const f32x4 k4 = token4(tk, own, 16 * m + 4 * g), q4 = token4(tq, own, 16 * m + 4 * g);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            wrote = fmaf(k4[e], ad[m][e], wrote);
            read = fmaf(q4[e], aw[m][e], fmaf(k4[e], av[m][e], read));
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (2 * j <= w) {
            const Parts<3> x = split<3>(pt[2 * j], pt[2 * j + 1]), y = split<3>(lt[2 * j], lt[2 * j + 1]);
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const Parts<NP> kf = by_feature(tk, m, j, lane);
                aw[m] = mma(kf, x, aw[m]);
                av[m] = mma(kf, y, av[m]);
            }
        }
        if (2 * j + 1 >= w) {
            const Parts<3> x = split<3>(p[2 * j], p[2 * j + 1]), y = split<3>(l[2 * j], l[2 * j + 1]);
#pragma unroll
            for (int m = 0; m < M; ++m) {
                ad[m] = mma(by_feature(tq, m, j, lane), x, ad[m]);
                ad[m] = mma(by_feature(tk, m, j, lane), y, ad[m]);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < M; ++m) av[m] += ad[m];
    double cross = (double)kept * all;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) cross += __shfl_xor(cross, o, 64);
    auto over_groups = [](float x) {
        x += __shfl_xor(x, 16, 64);
        return x + __shfl_xor(x, 32, 64);
    };
    wrote = over_groups(wrote);
    read = over_groups(read);
    de = over_groups(de);
    if (g == 0) {
        reads[own] = read;
        leaves[own] = wrote;
        const Rows<float> o(q_.a.deta, b, h, a.f.H, T, 1, a.f.tokens_first);
        if (q_.a.deta && inside) *o.at(t0 + own) = de;
    }
    if (lane == 0) across[w] = cross;
    __syncthreads();
    if (w == 0 && q_.a.dg) {
        const int t = lane, tile = lane >> 4;
        double r = reads[t], l = leaves[t];
        float y = rows[t], x[4];
#pragma unroll
        for (int i = 1; i < 4; ++i) x[i] = t < 16 * i ? later[i][t] : 0.f;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const double r1 = __shfl_down(r, o, 64), l1 = __shfl_up(l, o, 64);
            if (t + o < 64) r += r1;
            if (t >= o) l += l1;
            const float y1 = __shfl_down(y, o, 64);
            if (o < 16 && c + o < 16) y += y1;
#pragma unroll
            for (int i = 1; i < 4; ++i) {
                const float x1 = __shfl_up(x[i], o, 64);
                if (t >= o) x[i] += x1;
            }
        }
        // (sums over r < t: those through t - 1)
        l = __shfl_up(l, 1, 64);
        double pairs = (double)y + inner[t];
#pragma unroll
        for (int i = 1; i < 4; ++i) {
            const float x1 = __shfl_up(x[i], 1, 64);
            if (t && i > tile) pairs += x1;
        }
        const double all_ = (across[0] + across[1]) + (across[2] + across[3]);
        const Rows<float> o(q_.a.dg, b, h, a.f.H, T, 1, a.f.tokens_first);
        if (t0 + t < T) *o.at(t0 + t) = rec.forgets[t] ? 0.f : (float)(pairs + r + (t ? l : 0.0) + all_);
    }
    if (q_.dK) {
        float* to = q_.dK + (unit * kChunk + own) * DK + 4 * g;
        float* tq_ = q_.dQ + (unit * kChunk + own) * DK + 4 * g;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            *reinterpret_cast<f32x4*>(to + 16 * m) = av[m];
            *reinterpret_cast<f32x4*>(tq_ + 16 * m) = aw[m];
        }
    } else if (inside) {
        const Rows<TIO> dQ((TIO*)q_.a.dQ, b, hk, a.f.Hk, T, dk, a.f.tokens_first);
        const Rows<TIO> dK((TIO*)q_.a.dK, b, hk, a.f.Hk, T, dk, a.f.tokens_first);
#pragma unroll
        for (int m = 0; m < M; ++m) {
            store4(dQ.at(t0 + own), 16 * m + 4 * g, dk, dk % 4 == 0, aw[m]);
            store4(dK.at(t0 + own), 16 * m + 4 * g, dk, dk % 4 == 0, av[m]);
        }
    }
}

// dK and dQ of a chunk of a head of keys: the sum over the heads of values that share it, in
// their order
template <typename TIO>
__global__ void __launch_bounds__(256) delta_shared_kernel(BwdPass q_, int DK)
{
    const DeltaPass& a = q_.p;
    const int share = a.f.H / a.f.Hk, chunk = blockIdx.x % a.chunks, group = blockIdx.x / a.chunks;
    const int key = a.head0 / share + group, b = key / a.f.Hk, hk = key % a.f.Hk, dk = a.f.dk, T = a.f.T;
    const Rows<TIO> dK((TIO*)q_.a.dK, b, hk, a.f.Hk, T, dk, a.f.tokens_first);
    const Rows<TIO> dQ((TIO*)q_.a.dQ, b, hk, a.f.Hk, T, dk, a.f.tokens_first);
    for (int e = threadIdx.x; e < kChunk * DK / 4; e += 256) {
        const int row = e / (DK / 4), f = 4 * (e % (DK / 4)), t = chunk * kChunk + row;
        if (t >= T || f >= dk) continue;
        f32x4 k = {0.f, 0.f, 0.f, 0.f}, q = k;
        for (int r = 0; r < share; ++r) {
            const size_t at = (((size_t)(group * share + r) * a.chunks + chunk) * kChunk + row) * DK + f;
            k += *reinterpret_cast<const f32x4*>(q_.dK + at);
            q += *reinterpret_cast<const f32x4*>(q_.dQ + at);
        }
        store4(dK.at(t), f, dk, dk % 4 == 0, k);
        store4(dQ.at(t), f, dk, dk % 4 == 0, q);
    }
}

template <typename TIO, int DK>
hipError_t gradients(const BwdPass& q, hipStream_t s)
{
    const DeltaPass& p = q.p;
    delta_grads_kernel<TIO, DK><<<(unsigned)((size_t)p.heads * p.chunks), 256, 0, s>>>(q);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !q.dK) return e;
    const size_t groups = p.heads / (p.f.H / p.f.Hk);
    delta_shared_kernel<TIO><<<(unsigned)(groups * p.chunks), 256, 0, s>>>(q, DK);
    return hipGetLastError();
}

constexpr size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
constexpr size_t kPassBytes = (size_t)4 << 30;   // of workspace a pass, as in the forward pass

struct Plan {
    DeltaCut cut;
    int chunks, groups, dvp;
    size_t S, St, P, states, cotangents, U, F, dK, dQ, ends, ends_back, transitions, bytes;
};

Plan bwd_plan(int B, int H, int Hk, int T, int dk, int dv)
{
    Plan p;
    p.chunks = (T + kChunk - 1) / kChunk;
    p.dvp = (dv + 31) / 32 * 32;
    const size_t unit = (size_t)p.chunks * (H / Hk), DK = delta_padded_dk(dk);
    const size_t state = 4 * DK * p.dvp, rows = 4 * (size_t)kChunk * p.dvp, frags = 3 * kFragQuads * sizeof(quad);
    const size_t sums = H > Hk ? 4 * (size_t)kChunk * DK : 0;   // a plane of dK or dQ
    const size_t one = unit * (sizeof(Record) + 3 * frags + 2 * state + 2 * rows + 2 * sums);
    p.groups = (int)std::min<size_t>((size_t)B * Hk, std::max<size_t>(1, kPassBytes / one));
    const size_t units = unit * p.groups;
    p.S = up256(units * sizeof(Record));
    p.St = p.S + up256(units * frags);
    p.P = p.St + up256(units * frags);
    p.states = p.P + up256(units * frags);
    p.cotangents = p.states + up256(units * state);
    p.U = p.cotangents + up256(units * state);
    p.F = p.U + up256(units * rows);
    p.dK = p.F + up256(units * rows);
    p.dQ = p.dK + up256(units * sums);
    const size_t heads = (size_t)p.groups * (H / Hk);
    p.cut = delta_cut((int)heads, p.chunks, dv, dk, true);
    const size_t cut = p.cut.segments > 1 ? heads * p.cut.segments * DK * 4 : 0;
    p.ends = p.dQ + up256(units * sums);
    p.ends_back = p.ends + up256(cut * p.dvp);
    p.transitions = p.ends_back + up256(cut * p.dvp);
    p.bytes = p.transitions + up256(cut * DK);
    return p;
}

}  // namespace

size_t delta_bwd_workspace(int B, int H, int Hk, int T, int dk, int dv, bool)
{
    return bwd_plan(B, H, Hk, T, dk, dv).bytes;
}

hipError_t launch_delta_bwd(const DeltaBwdArgs& a, hipStream_t s)
{
    const DeltaArgs& f = a.f;
    const Plan plan = bwd_plan(f.B, f.H, f.Hk, f.T, f.dk, f.dv);
    char* ws = (char*)f.workspace;
    BwdPass q = {};
    q.a = a;
    DeltaPass& p = q.p;
    p.f = f;
    p.chunks = plan.chunks;
    p.dvp = plan.dvp;
    p.cut = plan.cut;
    p.ends = (float*)(ws + plan.ends);
    p.ends_back = (float*)(ws + plan.ends_back);
    p.transitions = (float*)(ws + plan.transitions);
    p.records = (Record*)ws;
    p.S = (f32x4*)(ws + plan.S);
    p.St = (f32x4*)(ws + plan.St);
    p.P = (f32x4*)(ws + plan.P);
    p.states = (float*)(ws + plan.states);
    p.cotangents = (float*)(ws + plan.cotangents);
    p.U = (float*)(ws + plan.U);
    p.F = (float*)(ws + plan.F);
    if (f.H > f.Hk) {
        q.dK = (float*)(ws + plan.dK);
        q.dQ = (float*)(ws + plan.dQ);
    }
    const int share = f.H / f.Hk, all = f.B * f.Hk, DK = delta_padded_dk(f.dk);
    for (int first = 0; first < all; first += plan.groups) {
        p.head0 = first * share;
        p.heads = std::min(plan.groups, all - first) * share;
        hipError_t e = launch_delta_prepare(p, true, s);
        if (e == hipSuccess) e = launch_delta_scans(p, &a, s);
        if (e != hipSuccess) return e;
        if (f.bf16)
            e = DK == 32 ? gradients<uint16_t, 32>(q, s)
              : DK == 64 ? gradients<uint16_t, 64>(q, s)
                         : gradients<uint16_t, 128>(q, s);
        else
            e = DK == 32 ? gradients<float, 32>(q, s)
              : DK == 64 ? gradients<float, 64>(q, s)
                         : gradients<float, 128>(q, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace ttt
