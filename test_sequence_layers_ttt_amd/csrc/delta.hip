// Gated delta rule: forward pass by chunks of 64 tokens, and the token-by-token form.
// (delta_common.h has the formulas.)
//
// The first kernel prepares every chunk of every head by itself: decays, K K^T, Q K^T and the
// triangular solve S.  The scans over the chunks (delta_scan.hip) take it from there.
#include <algorithm>

#include "delta_common.h"
#include "mfma_f32.h"

namespace ttt {
namespace {

__device__ __forceinline__ double shift_up(double x, int by) { return __shfl_up(x, by, 64); }

// ---- per chunk: decays, L, S, P -------------------------------------------------
// One workgroup of four waves per (chunk, head).  P's operands (or its transpose's) come out
// of the products of keys and queries as they lie, with the operands' order chosen for it.
// S = (I + L eta)^-1 L column tile by column tile: the four 16 x 16 diagonal blocks are
// inverted by substitution, the tiles below follow from them in order, in fp32 throughout.
// HBM and latency bound it: 16384 chunks of 64 features 140 us for 640 MB.
// LDS decides how many workgroups a compute unit holds: S takes the place of the tiles, and
// the inverted blocks stand in the tiles of L above its diagonal.
template <typename TIO, int DK, bool BACKWARD>
__global__ void __launch_bounds__(256) delta_prepare_kernel(DeltaPass a)
{
    constexpr int LD = kChunk + 4;
    struct Inputs { Tile<TIO, DK> k, q; };
    union Room {
        Inputs in;
        float S[kChunk * LD];
    };
    __shared__ __align__(16) Room room;
    __shared__ __align__(16) float Lm[kChunk * LD];
    __shared__ __align__(16) float hi[kChunk], lo[kChunk], eta[kChunk];
    const Tile<TIO, DK>&tk = room.in.k, &tq = room.in.q;
    float* Sm = room.S;

    const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, g = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int chunk = blockIdx.x % a.chunks, local = blockIdx.x / a.chunks;
    const int head = a.head0 + local, b = head / a.f.H, h = head % a.f.H;
    const int hk = h / (a.f.H / a.f.Hk), t0 = chunk * kChunk, T = a.f.T, dk = a.f.dk;
    const bool whole = dk % kGran<TIO> == 0;
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};

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
    const size_t unit = (size_t)local * a.chunks + chunk;
    Record& rec = a.records[unit];
    if (w == 0) {
        const int t = t0 + lane;
        const Rows<const float> rg(a.f.g, b, h, a.f.H, T, 1, a.f.tokens_first);
        const Rows<const float> re(a.f.eta, b, h, a.f.H, T, 1, a.f.tokens_first);
        const float gt = a.f.g && t < T ? *rg.at(t) : 0.f;   // (tokens past the end change nothing)
        const float et = t < T ? (a.f.eta ? *re.at(t) : a.f.eta_scalar) : 0.f;
        // (sums in fp64: differences of far sums have to keep their own digits)
        double x = (double)gt * 1.4426950408889634;
        const bool none = x <= kLeast;
        if (none) x = kLeast;
        for (int o = 1; o < 64; o <<= 1) {
            const double y = shift_up(x, o);
            if (lane >= o) x += y;
        }
        const double all = __shfl(x, 63, 64);
        const float h = (float)x, l = (float)(x - (double)h);
        hi[lane] = h; lo[lane] = l; eta[lane] = et;
        rec.hi[lane] = h; rec.lo[lane] = l; rec.eta[lane] = et;
        rec.start[lane] = __builtin_amdgcn_exp2f(h);
        rec.end[lane] = __builtin_amdgcn_exp2f((float)(all - x));
        rec.forgets[lane] = gt * 1.4426950408889634f < -150.f;
    }
    lk.put(room.in.k, tid);
    lq.put(room.in.q, tid);
    __syncthreads();

    // row tile w of L, and of P: rows s by column t (P's operand as it lies) up to the diagonal,
    // or rows t by column s from the diagonal on (its transpose's)
    f32x4 p[4];
    const f32x4 hw = *reinterpret_cast<const f32x4*>(hi + 16 * w + 4 * g);
    const f32x4 lw = *reinterpret_cast<const f32x4*>(lo + 16 * w + 4 * g);
    const float hc = hi[16 * w + c], lc = lo[16 * w + c];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f32x4 kk = zero;
        p[i] = zero;
        const f32x4 hr = *reinterpret_cast<const f32x4*>(hi + 16 * i + 4 * g);
        const f32x4 lr = *reinterpret_cast<const f32x4*>(lo + 16 * i + 4 * g);
        if (i <= w) {
#pragma unroll
            for (int j = 0; j < DK / 32; ++j) {
                const auto s = by_token(tk, i, j, lane);
                kk = mma(by_token(tk, w, j, lane), s, kk);
                if constexpr (!BACKWARD) p[i] = mma(s, by_token(tq, w, j, lane), p[i]);
            }
            const float hs = hi[16 * i + c], ls = lo[16 * i + c];
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                kk[v] = 16 * i + c < 16 * w + 4 * g + v ? kk[v] * pair_decay(hw[v], lw[v], hs, ls) : 0.f;
                if constexpr (!BACKWARD)
                    p[i][v] = 16 * i + 4 * g + v <= 16 * w + c ? p[i][v] * pair_decay(hc, lc, hr[v], lr[v]) : 0.f;
            }
            put_cl<LD>(Lm + 16 * w * LD, 16 * i, lane, kk);
        }
        if constexpr (BACKWARD) {
            if (i >= w) {
#pragma unroll
                for (int j = 0; j < DK / 32; ++j)
                    p[i] = mma(by_token(tq, i, j, lane), by_token(tk, w, j, lane), p[i]);
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    p[i][v] = 16 * w + c <= 16 * i + 4 * g + v ? p[i][v] * pair_decay(hr[v], lr[v], hc, lc) : 0.f;
            }
        }
    }
    // (backward with wide workgroups: three parts of each operand)
    const bool parts = BACKWARD && !a.cut.narrow;
    const size_t each = parts ? 3 * kFragQuads : kHalfQuads;
    f32x4* fp = a.P + unit * each;
    if (parts) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (j >= w / 2) store_frag<3>((quad*)fp, frag_upper(w, j), lane, p[2 * j], p[2 * j + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!BACKWARD && i <= w) fp[64 * half_lower(w, i) + lane] = p[i];
            if (BACKWARD && i >= w) fp[64 * half_upper(w, i) + lane] = p[i];
        }
    }
    __syncthreads();

    // (I + L eta)^-1 of diagonal block w, column c (the four groups of lanes do the same), into
    // one of the tiles (0, 1), (0, 2), (0, 3), (1, 2)
    auto inverse_at = [&](int i) { return Lm + (i < 3 ? 16 * (i + 1) : 16 * LD + 32); };
    {
        float x[16];
        const float* L = Lm + 16 * w * LD + 16 * w;
        f32x4 e[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) e[s] = *reinterpret_cast<const f32x4*>(eta + 16 * w + 4 * s);
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            float y = t == c ? 1.f : 0.f;
#pragma unroll
            for (int s = 0; s < t; s += 4) {
                const f32x4 n = *reinterpret_cast<const f32x4*>(L + t * LD + s) * e[s / 4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (s + i < t) y = fmaf(-n[i], x[s + i], y);
            }
            x[t] = y;
        }
        float* to = inverse_at(w);
        if (g == 0)
#pragma unroll
            for (int t = 0; t < 16; ++t) to[t * LD + c] = x[t];
    }
    __syncthreads();

    // column tile w of S, from its diagonal block down
    {
        f32x4 S[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            S[i] = zero;
            if (i >= w) {
                f32x4 r = cl<LD>(Lm + 16 * i * LD, 16 * w, lane);
#pragma unroll
                for (int j = 0; j < i; ++j)
                    if (j >= w) {
                        const f32x4 n = rl<LD>(Lm + 16 * i * LD, 16 * j, lane);
                        const f32x4 e = *reinterpret_cast<const f32x4*>(eta + 16 * j + 4 * g);
                        r = mm16(-(n * e), S[j], r);
                    }
                S[i] = mm16(rl<LD>(inverse_at(i), 0, lane), r, zero);
            }
            put_cl<LD>(Sm + 16 * i * LD, 16 * w, lane, S[i]);
        }
        if constexpr (BACKWARD) {
            f32x4* ft = a.St + unit * each;
            if (parts) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (j >= w / 2) store_frag<3>((quad*)ft, frag_upper(w, j), lane, S[2 * j], S[2 * j + 1]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i >= w) ft[64 * half_upper(w, i) + lane] = S[i];
            }
        }
    }
    __syncthreads();
    f32x4* fs = a.S + unit * each;
    auto row = [&](int i) { return rl<LD>(Sm + 16 * w * LD, 16 * i, lane); };
    if (parts) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (j <= w / 2) store_frag<3>((quad*)fs, frag_lower(w, j), lane, row(2 * j), row(2 * j + 1));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i <= w) fs[64 * half_lower(w, i) + lane] = row(i);
    }
}

// ---- token after token ---------------------------------------------------------------
// 16 lanes hold R rows of the state, 4 X features of each; a workgroup of 256 threads 16 R rows.
// HBM bounds the decoded token of a large batch (the state in and out).  W k and W q are
// summed at once: z = exp(g) W q + eta u (k.q).
template <typename TIO, int X, int R>
__global__ void __launch_bounds__(256) delta_step_kernel(DeltaArgs a, int parts)
{
    const int tid = threadIdx.x, c = tid & 15;
    const int head = blockIdx.x / parts, row0 = (blockIdx.x % parts) * 16 * R + (tid >> 4);
    const int b = head / a.H, h = head % a.H, hk = h / (a.H / a.Hk), T = a.T, dk = a.dk, dv = a.dv;
    const Rows<const TIO> K((const TIO*)a.K, b, hk, a.Hk, T, dk, a.tokens_first);
    const Rows<const TIO> Q((const TIO*)a.Q, b, hk, a.Hk, T, dk, a.tokens_first);
    const Rows<const TIO> V((const TIO*)a.V, b, h, a.H, T, dv, a.tokens_first);
    const Rows<TIO> Z((TIO*)a.Z, b, h, a.H, T, dv, a.tokens_first);
    const Rows<const float> rg(a.g, b, h, a.H, T, 1, a.tokens_first);
    const Rows<const float> re(a.eta, b, h, a.H, T, 1, a.tokens_first);
    const bool fours = dk % 4 == 0;
    const size_t state = ((size_t)head * dv + row0) * dk;
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};

    f32x4 W[R][X];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int x = 0; x < X; ++x)
            W[r][x] = a.W0 && row0 + 16 * r < dv
                          ? load4(a.W0 + state + (size_t)(16 * r) * dk, 64 * x + 4 * c, dk, fours) : zero;
    for (int t = 0; t < T; ++t) {
        f32x4 k[X], q[X];
        float v[R];
#pragma unroll
        for (int x = 0; x < X; ++x) {
            k[x] = load4(K.at(t), 64 * x + 4 * c, dk, fours);
            q[x] = load4(Q.at(t), 64 * x + 4 * c, dk, fours);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) v[r] = row0 + 16 * r < dv ? load1(V.at(t) + row0 + 16 * r) : 0.f;
        const float gt = a.g ? *rg.at(t) : 0.f, eta = a.eta ? *re.at(t) : a.eta_scalar;
        const float decay = gt <= kForget ? 0.f : expf(gt);
        float sum[2 * R + 1] = {};
#pragma unroll
        for (int x = 0; x < X; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sum[2 * R] = fmaf(k[x][e], q[x][e], sum[2 * R]);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    W[r][x][e] *= decay;
                    sum[2 * r] = fmaf(W[r][x][e], k[x][e], sum[2 * r]);
                    sum[2 * r + 1] = fmaf(W[r][x][e], q[x][e], sum[2 * r + 1]);
                }
            }
        row_sum16_n(sum);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float u = eta * (v[r] - sum[2 * r]);
#pragma unroll
            for (int x = 0; x < X; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) W[r][x][e] = fmaf(u, k[x][e], W[r][x][e]);
            if (row0 + 16 * r < dv && c == 0) store1(Z.at(t) + row0 + 16 * r, fmaf(u, sum[2 * R], sum[2 * r + 1]));
        }
    }
    if (a.W_out)
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int x = 0; x < X; ++x)
                if (row0 + 16 * r < dv)
                    store4(a.W_out + state + (size_t)(16 * r) * dk, 64 * x + 4 * c, dk, fours, W[r][x]);
}

template <typename TIO, int DK>
hipError_t prepare_as(const DeltaPass& p, bool backward, hipStream_t s)
{
    const unsigned grid = (unsigned)((size_t)p.heads * p.chunks);
    if (backward) delta_prepare_kernel<TIO, DK, true><<<grid, 256, 0, s>>>(p);
    else delta_prepare_kernel<TIO, DK, false><<<grid, 256, 0, s>>>(p);
    return hipGetLastError();
}

constexpr size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
// Heads are taken in passes that need no more workspace than this each, a group of heads that share
// keys at least: every pass of a gigabyte still fills the card (21.5 KB a chunk).
constexpr size_t kPassBytes = (size_t)1 << 30;

struct Plan {
    DeltaCut cut;
    int chunks, groups, dvp;   // groups of heads that share keys, in one pass
    size_t S, P, ends, transitions, bytes;   // places in the workspace, which begins with the records
};

Plan fwd_plan(int B, int H, int Hk, int T, int dk, int dv)
{
    Plan p;
    p.chunks = (T + kChunk - 1) / kChunk;
    p.dvp = (dv + 31) / 32 * 32;
    const size_t share = H / Hk, unit = p.chunks * share, half = kHalfQuads * sizeof(f32x4);
    const size_t one = unit * (sizeof(Record) + 2 * half);
    p.groups = (int)std::min<size_t>((size_t)B * Hk, std::max<size_t>(1, kPassBytes / one));
    const size_t heads = p.groups * share, units = unit * p.groups, DK = delta_padded_dk(dk);
    p.cut = delta_cut((int)heads, p.chunks, dv, dk, false);
    const size_t cut = p.cut.segments > 1 ? heads * p.cut.segments * DK * 4 : 0;
    p.S = up256(units * sizeof(Record));
    p.P = p.S + up256(units * half);
    p.ends = p.P + up256(units * half);
    p.transitions = p.ends + up256(cut * p.dvp);
    p.bytes = p.transitions + up256(cut * DK);
    return p;
}

}  // namespace

hipError_t launch_delta_prepare(const DeltaPass& p, bool backward, hipStream_t s)
{
    const int DK = delta_padded_dk(p.f.dk);
    if (p.f.bf16)
        return DK == 32 ? prepare_as<uint16_t, 32>(p, backward, s)
             : DK == 64 ? prepare_as<uint16_t, 64>(p, backward, s)
                        : prepare_as<uint16_t, 128>(p, backward, s);
    return DK == 32 ? prepare_as<float, 32>(p, backward, s)
         : DK == 64 ? prepare_as<float, 64>(p, backward, s)
                    : prepare_as<float, 128>(p, backward, s);
}

size_t delta_fwd_workspace(int B, int H, int Hk, int T, int dk, int dv, bool)
{
    return fwd_plan(B, H, Hk, T, dk, dv).bytes;
}

hipError_t launch_delta_fwd(const DeltaArgs& a, hipStream_t s)
{
    const Plan plan = fwd_plan(a.B, a.H, a.Hk, a.T, a.dk, a.dv);
    char* ws = (char*)a.workspace;
    DeltaPass p = {};
    p.f = a;
    p.chunks = plan.chunks;
    p.dvp = plan.dvp;
    p.cut = plan.cut;
    p.records = (Record*)ws;
    p.S = (f32x4*)(ws + plan.S);
    p.P = (f32x4*)(ws + plan.P);
    p.ends = (float*)(ws + plan.ends);
    p.transitions = (float*)(ws + plan.transitions);
    const int share = a.H / a.Hk, all = a.B * a.Hk;
    for (int first = 0; first < all; first += plan.groups) {
        p.head0 = first * share;
        p.heads = std::min(plan.groups, all - first) * share;
        hipError_t e = launch_delta_prepare(p, false, s);
        if (e == hipSuccess) e = launch_delta_scans(p, nullptr, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <typename TIO>
static void step_as(const DeltaArgs& a, hipStream_t s)
{
    // four rows a lane where the card is full of workgroups all the same (256 x 12 heads of 64
    // features 21 us for 101 MB, with one row 29 us); one for few heads, whose latency counts
    // (8 x 12: 4.3 us)
    const bool four = (long long)a.B * a.H * a.dv >= 65536;
    const int parts = (a.dv + (four ? 63 : 15)) / (four ? 64 : 16);
    const unsigned grid = (unsigned)(a.B * a.H * parts);
    if (a.dk <= 64) {
        if (four) delta_step_kernel<TIO, 1, 4><<<grid, 256, 0, s>>>(a, parts);
        else delta_step_kernel<TIO, 1, 1><<<grid, 256, 0, s>>>(a, parts);
    } else {
        if (four) delta_step_kernel<TIO, 2, 4><<<grid, 256, 0, s>>>(a, parts);
        else delta_step_kernel<TIO, 2, 1><<<grid, 256, 0, s>>>(a, parts);
    }
}

hipError_t launch_delta_step(const DeltaArgs& a, hipStream_t s)
{
    if (a.bf16) step_as<uint16_t>(a, s);
    else step_as<float>(a, s);
    return hipGetLastError();
}

}  // namespace ttt
