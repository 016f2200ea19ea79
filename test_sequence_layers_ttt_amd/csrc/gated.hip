// Gated linear recurrence h_t = exp(g_t) h_{t-1} + x_t per channel, and its backward pass.
//
// The step h -> exp(g) h + x is affine, and affine maps compose: a run of tokens is the
// pair (sum of its g, B) with h_end = exp(sum g) h_start + B.  The gates' product is kept
// as the sum of the g, with -inf for a run with a reset in it: a product that underflowed
// would look the same.
//
// A tile is all that one workgroup holds in registers: `rows` runs of L tokens over the
// channels of one block, each thread a run of L tokens of V neighbouring channels (16
// bytes).  Every input is read once:
//   1. each thread reduces its run to its pair;
//   2. the pairs of the tile's runs are scanned in LDS (threads as channel x part);
//   3. the tile publishes its pair, takes the state before it from the tiles before, and
//      publishes the state after it;
//   4. each thread runs its tokens again from its own start state and writes them.
// Step 3 is a chain along the sequence, of groups of 8 tiles.  A tile composes the pairs of
// the tiles before it in its group, which wait for nothing; the group's last tile publishes
// the group's pair and then the state after the group; and a tile takes the state before
// its group from the nearest group that has one and the pairs of the groups since.  (With
// the states chained from tile to tile instead, 1 x 131072 x 64 took 75 us, against 28.)
// Tiles take their place by a ticket, so a tile only ever waits for tiles that run already.
// The words they pass on are 64 bits wide, written whole and read until they are there (an
// unwritten word is all ones, which no published one is): no fence, no flag.  What is
// composed with what does not depend on what was published when, so every output has the
// same bits on every call.
//
// The backward pass is the same chain from the other end: lambda_t = dz_t + exp(g_{t+1})
// lambda_{t+1}; then dx_t = lambda_t and dg_t = exp(g_t) lambda_t h_{t-1}.
#include <stdint.h>

#include <algorithm>

#include "block_launch.h"
#include "device_common.h"
#include "mfma_common.h"

namespace ttt {
namespace {

constexpr float kLog2e = 1.44269504088896f;
constexpr float kShut = -__builtin_inff();   // the summed g of a run with a reset in it
// A gate below this (times log2(e)) is a reset: -inf, a type's lowest value.  Sums of the others
// stay finite over any run.
constexpr float kLowest = -1e30f * kLog2e;
constexpr int kThreads = 256;
constexpr int kTicket = 32;                  // words from ticket to ticket
constexpr int kGroup = 8;                    // tiles of a group
constexpr int kWindow = 8;                   // groups looked back over at once
constexpr int kMostPolls = 1 << 22;          // seconds: only a workspace in use twice gets there

// V elements of the I/O type at any element-aligned address, as raw words.  Where rows are whole
// cache lines (LINES), every line is read or written once, at once, and 16-byte accesses take the
// non-temporal policy (8 x 12 x 2048 x 64 bf16, forward / backward: 23.0 / 35.0 us without, 21.1 /
// 27.0 with; 1 x 32 x 32768 x 64: 96 / 157 and 85 / 138).  Elsewhere a line takes several accesses,
// which meet in the caches only without it (64 x 32768 x 16 bf16: 106 / 260 us with, 60 / 109
// without; 64 x 8192 x 50: 64 / 142 and 50 / 85).
typedef uint32_t quad __attribute__((ext_vector_type(4)));
typedef quad quad_any __attribute__((aligned(2)));

template <typename TIO, int V, bool LINES>
struct Raw {
    static constexpr int BYTES = V * (int)sizeof(TIO);
    static constexpr int WORDS = (BYTES + 3) / 4;
    struct __attribute__((packed, aligned(sizeof(TIO)))) Mem { TIO e[V]; };
    uint32_t w[WORDS];
    __device__ __forceinline__ void load(const TIO* p)
    {
        if constexpr (BYTES == 16) {
            auto from = reinterpret_cast<const quad_any*>(p);
            const quad q = LINES ? __builtin_nontemporal_load(from) : *from;
            w[0] = q.x; w[1] = q.y; w[2] = q.z; w[3] = q.w;
            return;
        }
        const Mem m = *reinterpret_cast<const Mem*>(p);
        if constexpr (BYTES < 4) w[0] = m.e[0];
        else __builtin_memcpy(w, &m, BYTES);
    }
    __device__ __forceinline__ void store(TIO* p) const
    {
        if constexpr (BYTES == 16) {
            const quad q = {w[0], w[1], w[2], w[3]};
            auto to = reinterpret_cast<quad_any*>(p);
            if constexpr (LINES) __builtin_nontemporal_store(q, to);
            else *to = q;
            return;
        }
        Mem m;
        if constexpr (BYTES < 4) m.e[0] = (TIO)w[0];
        else __builtin_memcpy(&m, w, BYTES);
        *reinterpret_cast<Mem*>(p) = m;
    }
    // the elements from `skip` on
    __device__ __forceinline__ void store_from(TIO* p, int skip) const
    {
        if (skip == 0) return store(p);
        Mem m;
        if constexpr (BYTES < 4) m.e[0] = (TIO)w[0];
        else __builtin_memcpy(&m, w, BYTES);
#pragma unroll
        for (int i = 1; i < V; ++i)
            if (i >= skip) p[i] = m.e[i];
    }
    // hides that the words are the ones a first pass has used: the second computes its
    // gates again instead of keeping the first one's in registers
    __device__ __forceinline__ void again()
    {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) asm volatile("" : "+v"(w[i]));
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = 0;
    }
    __device__ __forceinline__ float at(int i) const
    {
        if constexpr (sizeof(TIO) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float((i & 1) ? (w[i >> 1] & 0xffff0000u) : (w[i >> 1] << 16));
    }
    __device__ __forceinline__ void put(const float (&v)[V])
    {
        if constexpr (sizeof(TIO) == 4) {
#pragma unroll
            for (int i = 0; i < V; ++i) w[i] = __float_as_uint(v[i]);
        } else if constexpr (V == 1) {
            w[0] = f32_to_bf16_bits(v[0]);
        } else {
#pragma unroll
            for (int i = 0; i < V; i += 2)
                w[i / 2] = pack_bf16x2(v[i], v[i + 1]);
        }
    }
};

// One token: g2 = g log2(e).  A reset takes x whatever h is, infinite and NaN included; under any other
// gate an infinite state stays infinite, also where the gate's exponential is 0 in fp32 (a run's is
// sooner than a token's, and what comes out is not to depend on where runs begin).  EXACT = false
// leaves that out and gives NaN there: right as long as no state before it was infinite, which costs
// less to look out for (8 x 12 x 2048 x 64 bf16, forward / backward: 22.5 / 28.0 us with EXACT
// throughout, 21.5 / 26.5 this way).
template <bool EXACT>
__device__ __forceinline__ float token(float g2, float x, float h)
{
    float e = __builtin_amdgcn_exp2f(g2);
    if constexpr (EXACT) e = isinf(h) && g2 == g2 ? 1.f : e;
    return fmaf(e, g2 <= kLowest ? 0.f : h, x);
}

// one run: (S, B) with S the summed g2 (where S is NaN so is B)
__device__ __forceinline__ float run(float S, float B, float h)
{
    return S == kShut ? B : fmaf(isinf(h) ? 1.f : __builtin_amdgcn_exp2f(S), h, B);
}

// the largest of m and the magnitudes of v that are numbers
template <int V>
__device__ __forceinline__ float largest(float m, const float (&v)[V])
{
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, fabsf(v[i]));
    return m;
}

// h <- the states after one token more
template <bool EXACT, int V, typename W>
__device__ __forceinline__ void next(const W& g, const W& x, float (&h)[V])
{
#pragma unroll
    for (int i = 0; i < V; ++i) h[i] = token<EXACT>(g.at(i) * kLog2e, x.at(i), h[i]);
}

// (S, B) <- the pairs of a run with one token more
template <bool EXACT, int V, typename W>
__device__ __forceinline__ void next(const W& g, const W& x, float (&S)[V], float (&B)[V])
{
    next<EXACT>(g, x, B);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float g2 = g.at(i) * kLog2e;
        S[i] = g2 <= kLowest ? kShut : S[i] + g2;
    }
}

// The pairs of L tokens of gates g and inputs x; where a B is NaN once more, exactly, over the n tokens
// that there are, as `reload` brings them (one after the other: the registers are full).
template <int L, int V, typename W, typename F>
__device__ __forceinline__ void reduce_run(W* g, W* x, int n, F&& reload, float (&S)[V], float (&B)[V])
{
    static_assert(L % 2 == 0, "");
#pragma unroll
    for (int i = 0; i < V; ++i) S[i] = B[i] = 0.f;
#pragma unroll
    for (int l = 0; l < L; ++l) {
        next<false>(g[l], x[l], S, B);
        if (l % 2 == 0) continue;
        // (two tokens at a time: with all of them widened at once registers run out)
#pragma unroll
        for (int i = 0; i < V; ++i) asm volatile("" : "+v"(B[i]), "+v"(S[i]));
#pragma unroll
        for (int k = l + 1; k < L && k < l + 3; ++k) {
            g[k].again();
            x[k].again();
        }
    }
    bool nan = false;
#pragma unroll
    for (int i = 0; i < V; ++i) nan = nan || B[i] != B[i];
    if (!nan) return;
#pragma unroll
    for (int i = 0; i < V; ++i) S[i] = B[i] = 0.f;
#pragma unroll 1
    for (int l = 0; l < n; ++l) {
        W a, b;
        reload(l, a, b);
        next<true>(a, b, S, B);
    }
}

// how the channels of a row lie over workgroups and threads (host and device)
struct Layout {
    int V;        // channels of a thread
    int lanes;    // threads over the channels of a block
    int rows;     // runs of a tile
    int blocks;   // channel blocks of a row
    int parts;    // parts that the scan over the runs is split into
    int per;      // runs of a part
    int width;    // lanes * V: channel slots of a block
    int threads;  // of a workgroup
    bool lines;   // a row is whole cache lines
};

Layout layout_of(int d, bool bf16, int threads)
{
    Layout y;
    y.threads = threads;
    y.V = bf16 ? 8 : 4;
    while (y.V > d) y.V >>= 1;
    // Where rows are whole cache lines, a block is one line wide, or two where that makes more
    // than four blocks: long tiles, so few of them wait for each other (15 x 4097 x 96 fp32,
    // forward: 19.1 us with lines, 20.0 with whole rows; x 64: 16 either way).  Elsewhere blocks
    // would share lines (x 80: 22.2 with lines, 19.3 with whole rows).
    const int groups = (d + y.V - 1) / y.V, bytes = d * (bf16 ? 2 : 4);
    y.lines = bytes % 128 == 0;
    const int most = !y.lines ? 256 / y.V : bytes <= 512 ? 8 : 16;
    y.blocks = (groups + most - 1) / most;
    y.lanes = (groups + y.blocks - 1) / y.blocks;
    y.rows = threads / y.lanes;
    y.width = y.lanes * y.V;
    y.parts = std::min({threads / y.width, y.rows, 16});
    y.per = (y.rows + y.parts - 1) / y.parts;
    return y;
}

constexpr int kRunFwd = 8, kRunBwd = 8;      // tokens of a thread's run

// Workspace of a chain: tickets [sequences], each in a cache line of its own (counts in one
// line wait for each other, about 14 ns each: with the 15 of 15 x 4097 x 83 side by side the
// last workgroup had its ticket after 9 us), then a 64-bit word for every channel slot of
// every (sequence, tile), its pair (B above, S below), and one for every slot of every
// (sequence, group), first the group's pair and then (state after the group, kShut): a
// pair that needs no state before it.  A sequence here is one channel block of one row.
struct Chain {
    unsigned* ticket;
    unsigned long long* tile;
    unsigned long long* group;
    int groups;               // of a sequence
};

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

size_t chain_bytes(long long seqs, long long tiles, int width, Chain* c, void* ws)
{
    const long long groups = (tiles + kGroup - 1) / kGroup;
    const size_t t = up256(4 * (size_t)kTicket * seqs);
    const size_t n = up256(8 * (size_t)seqs * tiles * width);
    if (c) {
        unsigned char* p = (unsigned char*)ws;
        c->ticket = (unsigned*)p;
        c->tile = (unsigned long long*)(p + t);
        c->group = (unsigned long long*)(p + t + n);
        c->groups = (int)groups;
    }
    return t + n + up256(8 * (size_t)seqs * groups * width);
}

// tickets to 0, everything else to all ones
__global__ __launch_bounds__(kThreads) void gated_clear_kernel(uint4* p, size_t zeros, size_t n)
{
    for (size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x; i < n;
         i += (size_t)gridDim.x * kThreads) {
        const unsigned v = i < zeros ? 0u : 0xffffffffu;
        p[i] = make_uint4(v, v, v, v);
    }
}

constexpr unsigned long long kNothing = ~0ull;

// never kNothing
__device__ __forceinline__ void publish(unsigned long long* p, float S, float B)
{
    const unsigned s = S != S ? 0x7fc00000u : __float_as_uint(S);
    __hip_atomic_store(p, (unsigned long long)__float_as_uint(B) << 32 | s, __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ float part_S(unsigned long long p) { return __uint_as_float((unsigned)p); }
__device__ __forceinline__ float part_B(unsigned long long p) { return __uint_as_float((unsigned)(p >> 32)); }

// (s, b) <- the pair of (s, b) followed by (S, B)
__device__ __forceinline__ void follow(float& s, float& b, float S, float B)
{
    b = run(S, B, b);
    s = S == kShut ? kShut : s + S;
}

// The pair of the n < kGroup tiles whose words start at `word`, `width` apart.
__device__ __forceinline__ void pairs_before(const unsigned long long* word, int n, int width,
                                             float& s, float& b)
{
    s = b = 0.f;
    for (int poll = 0; poll < kMostPolls; ++poll) {
        unsigned long long p[kGroup - 1];
        bool all = true;
#pragma unroll
        for (int k = 0; k < kGroup - 1; ++k)
            if (k < n)
                p[k] = __hip_atomic_load(word + (size_t)k * width, __ATOMIC_RELAXED,
                                         __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
        for (int k = 0; k < kGroup - 1; ++k)
            if (k < n) all = all && p[k] != kNothing;
        if (all) {
#pragma unroll
            for (int k = 0; k < kGroup - 1; ++k)
                if (k < n) follow(s, b, part_S(p[k]), part_B(p[k]));
            return;
        }
        __builtin_amdgcn_s_sleep(1);
    }
    b = __builtin_nanf("");
}

// The state that enters group g > 0: `word` is group 0's.
__device__ __forceinline__ float state_before(const unsigned long long* word, int g, int width)
{
    for (int poll = 0; poll < kMostPolls; ++poll) {
        unsigned long long p[kWindow];
#pragma unroll
        for (int k = 0; k < kWindow; ++k)
            p[k] = __hip_atomic_load(word + (size_t)max(g - 1 - k, 0) * width, __ATOMIC_RELAXED,
                                     __HIP_MEMORY_SCOPE_AGENT);
        // the nearest group whose state is known, with every pair from there on
        int from = -1;
        bool open = true;
#pragma unroll
        for (int k = 0; k < kWindow; ++k) {
            open = open && p[k] != kNothing;
            if (open && part_S(p[k]) == kShut) {
                from = k;
                open = false;
            }
        }
        if (from >= 0) {
            float h = 0.f;
#pragma unroll
            for (int k = kWindow - 1; k >= 0; --k)
                if (k <= from) h = run(part_S(p[k]), part_B(p[k]), h);
            return h;
        }
        __builtin_amdgcn_s_sleep(1);
    }
    return __builtin_nanf("");
}

// Waits until group 0 has its state, which it has once all of its tiles have published: whether it
// came to that.
__device__ __forceinline__ bool first_group_done(const unsigned long long* word)
{
    for (int poll = 0; poll < kMostPolls; ++poll) {
        if (__hip_atomic_load(word, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != kNothing) return true;
        __builtin_amdgcn_s_sleep(1);
    }
    return false;
}

struct Tile {
    int seq, j;        // sequence (row, channel block) and place of the tile in it
    int row;           // of the input
    int r, lane;       // this thread's run and channel group
    int c0;            // its first channel
    int skip;          // how many of them the group before has as well
    bool on;           // it has any

    // channel of a slot of the block, or -1
    __device__ __forceinline__ int channel(const Layout& y, int d, int slot) const
    {
        const int g = (seq - row * y.blocks) * y.lanes + slot / y.V;
        return g * y.V < d ? min(g * y.V, d - y.V) + slot % y.V : -1;
    }
};

// A workgroup's tile; j < 0: there is none left (a workspace in use twice).
__device__ __forceinline__ Tile take_tile(const Layout& y, int d, int tiles, int seqs,
                                          const Chain& chain, int* lds)
{
    Tile t;
    t.seq = blockIdx.x % seqs;
    t.j = 0;
    if (tiles > 1) {
        if (threadIdx.x == 0)
            *lds = (int)__hip_atomic_fetch_add(chain.ticket + (size_t)t.seq * kTicket, 1u,
                                               __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        t.j = *lds;
        if ((unsigned)t.j >= (unsigned)tiles) t.j = -1;
    }
    t.row = t.seq / y.blocks;
    t.r = threadIdx.x / y.lanes;
    t.lane = threadIdx.x - t.r * y.lanes;
    const int group = (t.seq - t.row * y.blocks) * y.lanes + t.lane;
    // The last group of a row whose width V does not divide starts early enough to be whole: the
    // channels it shares with the group before are computed by both, to the same bits.
    t.c0 = min(group * y.V, d - y.V);
    t.skip = group * y.V - t.c0;
    t.on = t.r < y.rows && group * y.V < d;
    return t;
}

// V floats of LDS, 4 V-byte aligned: in 16-byte accesses (single words of lanes V apart would meet
// in the same banks)
template <int V>
__device__ __forceinline__ void lds_put(float* p, const float (&v)[V])
{
    if constexpr (V >= 4) {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = v[i];
    }
}

template <int V>
__device__ __forceinline__ void lds_get(const float* p, float (&v)[V])
{
    if constexpr (V >= 4) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 q = *reinterpret_cast<const float4*>(p + i);
            v[i] = q.x; v[i + 1] = q.y; v[i + 2] = q.z; v[i + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = p[i];
    }
}

// The pairs of a tile's runs and of its parts; once scanned, those before each run in its part, and the
// states before the parts (pB).
template <int V, int NT>
struct Pairs {
    alignas(16) float sS[NT * V], sB[NT * V];
    float pS[NT];
    alignas(16) float pB[NT];
};

// the state before a thread's run, from the scanned pairs
template <int V, int NT>
__device__ __forceinline__ void run_start(const Layout& y, const Tile& t, const Pairs<V, NT>& lds,
                                          float (&start)[V])
{
    if (!t.on) return;
    const int w = y.width;
    float s[V], b[V];
    lds_get<V>(lds.sS + t.r * w + t.lane * V, s);
    lds_get<V>(lds.sB + t.r * w + t.lane * V, b);
    lds_get<V>(lds.pB + t.r / y.per * w + t.lane * V, start);
#pragma unroll
    for (int i = 0; i < V; ++i) start[i] = run(s[i], b[i], start[i]);
}

// The start state of each thread's run, from its pairs (S, B) and the states that enter the
// sequence (`first` of the row's channels, or nullptr for zero).  in_place: the row's last tile writes
// where `first` is read; on return every tile that reads it has done so.
template <int V, int NT>
__device__ __forceinline__ void start_states(const Layout& y, const Tile& t, int d, int tiles,
                                             const Chain& chain, const float* first, bool in_place,
                                             const float (&S)[V], const float (&B)[V],
                                             Pairs<V, NT>& lds, float (&start)[V])
{
    float *sS = lds.sS, *sB = lds.sB, *pS = lds.pS, *pB = lds.pB;
    const int w = y.width, tid = threadIdx.x;
    const int part = tid / w, c = tid - part * w;
    float h = 0.f;               // of the thread's channel slot, before the tile
    if (part == 0 && t.j < kGroup && first) {
        const int ch = t.channel(y, d, c);
        if (ch >= 0) h = first[ch];
    }
    if (t.r < y.rows) {
        float s[V], b[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            s[i] = t.on ? S[i] : 0.f;
            b[i] = t.on ? B[i] : 0.f;
        }
        lds_put<V>(sS + t.r * w + t.lane * V, s);
        lds_put<V>(sB + t.r * w + t.lane * V, b);
    }
    __syncthreads();
    // threads as (part, channel): each part's runs in turn, exclusive pairs left in place
    const bool scans = part < y.parts;
    if (scans) {
        float s = 0.f, b = 0.f;
        const int end = min((part + 1) * y.per, y.rows);
        for (int r = part * y.per; r < end; ++r) {
            const float ts = sS[r * w + c], tb = sB[r * w + c];
            sS[r * w + c] = s;
            sB[r * w + c] = b;
            follow(s, b, ts, tb);
        }
        pS[tid] = s;
        pB[tid] = b;
    }
    __syncthreads();
    if (part == 0) {
        // the tile's pair, then the state before it, then every part's start.  A tile has read `first`
        // before it publishes.
        asm volatile("s_waitcnt vmcnt(0)" : "+v"(h) : : "memory");
        if (tiles > 1) {
            float s = 0.f, b = 0.f;
            for (int p = 0; p < y.parts; ++p) follow(s, b, pS[p * w + c], pB[p * w + c]);
            const int g = t.j / kGroup, i = t.j % kGroup;
            const bool more = t.j + 1 < tiles, closes = i == kGroup - 1;
            unsigned long long* word = chain.tile + ((size_t)t.seq * tiles + (t.j - i)) * w + c;
            unsigned long long* group = chain.group + (size_t)t.seq * chain.groups * w + c;
            if (more && !closes) publish(word + (size_t)i * w, s, b);
            float before_s = 0.f, before_b = 0.f;
            if (i > 0) pairs_before(word, i, w, before_s, before_b);
            if (closes && more) {
                float gs = before_s, gb = before_b;
                follow(gs, gb, s, b);
                if (g > 0) {
                    publish(group + (size_t)g * w, gs, gb);
                    h = state_before(group, g, w);
                }
                publish(group + (size_t)g * w, kShut, run(gs, gb, h));
            } else if (g > 0) {
                h = state_before(group, g, w);
            }
            h = run(before_s, before_b, h);
            // The tiles of group 0 read `first`.  A last tile in group 0 has seen their pairs; one
            // further on may have taken its state from a group with a reset in it, which waits for no
            // tile of group 0.
            if (in_place && !more && g > 0 && !first_group_done(group)) h = __builtin_nanf("");
        }
        for (int p = 0; p < y.parts; ++p) {
            const float ts = pS[p * w + c], tb = pB[p * w + c];
            pB[p * w + c] = h;
            h = run(ts, tb, h);
        }
    }
    __syncthreads();
    run_start<V>(y, t, lds, start);
}

// in_place: h_out is h0.  Where a row has several blocks a channel is then written by one group of
// threads alone (the other group's copy may have started from what was written).
template <typename TIO, int V, int NT, bool LINES>
__global__ __launch_bounds__(NT) void gated_fwd_kernel(
    const TIO* __restrict__ X, const TIO* __restrict__ G, const float* h0, TIO* __restrict__ Z,
    float* h_out, int T, int d, int tiles, int seqs, Layout y, Chain chain, bool in_place)
{
    constexpr int L = kRunFwd;
    __shared__ int ticket;
    __shared__ Pairs<V, NT> lds;
    const Tile t = take_tile(y, d, tiles, seqs, chain, &ticket);
    if (t.j < 0) return;
    const long long t0 = ((long long)t.j * y.rows + t.r) * L;
    const int n = t.on ? (int)min(max(T - t0, 0ll), (long long)L) : 0;
    const size_t at = ((size_t)t.row * T + t0) * d + t.c0;

    Raw<TIO, V, LINES> x[L], g[L];
#pragma unroll
    for (int l = 0; l < L; ++l) {
        x[l].zero();
        g[l].zero();
        if (l < n) {
            g[l].load(G + at + (size_t)l * d);
            x[l].load(X + at + (size_t)l * d);
        }
    }
    float S[V], B[V], h[V];
    auto reload = [&](int l, Raw<TIO, V, LINES>& a, Raw<TIO, V, LINES>& b) {
        a.load(G + at + (size_t)l * d);
        b.load(X + at + (size_t)l * d);
    };
    reduce_run<L>(g, x, n, reload, S, B);
    start_states<V, NT>(y, t, d, tiles, chain, h0 ? h0 + (size_t)t.row * d : nullptr, in_place, S, B,
                        lds, h);
    const int skip = in_place && y.blocks > 1 ? t.skip : 0;
    float most = largest(0.f, h);
#pragma unroll
    for (int l = 0; l < L; ++l) {
        if (l >= n) break;
        g[l].again();
        x[l].again();
        next<false>(g[l], x[l], h);
        most = largest(most, h);
        asm volatile("" : "+v"(most));     // (now: the states are not kept for it)
        Raw<TIO, V, LINES> z;
        z.put(h);
        z.store_from(Z + at + (size_t)l * d, skip);
    }
    if (isinf(most)) {
        run_start<V>(y, t, lds, h);
#pragma unroll 1
        for (int l = 0; l < n; ++l) {
            Raw<TIO, V, LINES> a, b;
            reload(l, a, b);
            next<true>(a, b, h);
            b.put(h);
            b.store_from(Z + at + (size_t)l * d, skip);
        }
    }
    if (h_out && n > 0 && t0 + n == T) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i >= skip) h_out[(size_t)t.row * d + t.c0 + i] = h[i];
    }
}

template <typename TIO, int V, int NT, bool LINES>
__global__ __launch_bounds__(NT) void gated_bwd_kernel(
    const TIO* __restrict__ G, const TIO* __restrict__ Z, const float* __restrict__ h0,
    const TIO* __restrict__ dZ, const float* __restrict__ dh_T, TIO* __restrict__ dX,
    TIO* __restrict__ dG, float* __restrict__ dh0, int T, int d, int tiles, int seqs, Layout y,
    Chain chain)
{
    constexpr int L = kRunBwd;
    __shared__ int ticket;
    __shared__ Pairs<V, NT> lds;
    const Tile t = take_tile(y, d, tiles, seqs, chain, &ticket);
    if (t.j < 0) return;
    // this run's tokens, from the last one down: T - 1 - p0, ...
    const long long p0 = ((long long)t.j * y.rows + t.r) * L;
    const int n = t.on ? (int)min(max(T - p0, 0ll), (long long)L) : 0;
    const size_t at = ((size_t)t.row * T + (T - 1 - p0)) * d + t.c0;
    const bool first_token = n > 0 && p0 + n == T;   // the run ends with token 0

    Raw<TIO, V, LINES> dz[L], g[L + 1], z[L];               // g[l]: the gate after token l's
    g[0].zero();
    if (n > 0 && p0 > 0) g[0].load(G + at + d);
#pragma unroll
    for (int l = 0; l < L; ++l) {
        dz[l].zero();
        g[l + 1].zero();
        z[l].zero();
        if (l < n) {
            dz[l].load(dZ + at - (size_t)l * d);
            g[l + 1].load(G + at - (size_t)l * d);
            if (p0 + l + 1 < T) z[l].load(Z + at - (size_t)(l + 1) * d);
        }
    }
    float S[V], B[V], lam[V];
    auto reload = [&](int l, Raw<TIO, V, LINES>& a, Raw<TIO, V, LINES>& b) {
        a.zero();
        if (p0 + l > 0) a.load(G + at - (size_t)l * d + d);
        b.load(dZ + at - (size_t)l * d);
    };
    reduce_run<L>(g, dz, n, reload, S, B);
    start_states<V, NT>(y, t, d, tiles, chain, dh_T ? dh_T + (size_t)t.row * d : nullptr, false, S, B,
                        lds, lam);
    float most = largest(0.f, lam);
    g[0].again();
#pragma unroll
    for (int l = 0; l < L; ++l) {
        if (l >= n) break;
        g[l + 1].again();
        dz[l].again();
        next<false>(g[l], dz[l], lam);
        most = largest(most, lam);
        float dg[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float before = z[l].at(i);
            if (first_token && l == n - 1) before = h0 ? h0[(size_t)t.row * d + t.c0 + i] : 0.f;
            const float g2 = g[l + 1].at(i) * kLog2e;
            const float back = token<false>(g2, 0.f, lam[i]);
            dg[i] = g2 <= kLowest ? 0.f : back * before;
            if (dh0 && first_token && l == n - 1) dh0[(size_t)t.row * d + t.c0 + i] = back;
        }
        asm volatile("" : "+v"(most));
        Raw<TIO, V, LINES> o;
        o.put(lam);
        o.store(dX + at - (size_t)l * d);
        o.put(dg);
        o.store(dG + at - (size_t)l * d);
    }
    if (!isinf(most)) return;
    run_start<V>(y, t, lds, lam);
#pragma unroll 1
    for (int l = 0; l < n; ++l) {
        const bool first = first_token && l == n - 1;
        Raw<TIO, V, LINES> a, b, c;
        reload(l, a, b);
        c.zero();
        if (!first) c.load(Z + at - (size_t)(l + 1) * d);
        next<true>(a, b, lam);
        b.put(lam);
        b.store(dX + at - (size_t)l * d);
        a.load(G + at - (size_t)l * d);
        float dg[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float before = c.at(i);
            if (first) before = h0 ? h0[(size_t)t.row * d + t.c0 + i] : 0.f;
            const float g2 = a.at(i) * kLog2e, back = token<true>(g2, 0.f, lam[i]);
            dg[i] = g2 <= kLowest ? 0.f : back * before;
            if (dh0 && first) dh0[(size_t)t.row * d + t.c0 + i] = back;
        }
        b.put(dg);
        b.store(dG + at - (size_t)l * d);
    }
}

// Few tokens: a thread runs V channels through all of them, 8 tokens' loads at a time.
template <typename TIO, int V>
__global__ __launch_bounds__(kThreads) void gated_step_kernel(
    const TIO* __restrict__ X, const TIO* __restrict__ G, const float* h0, TIO* __restrict__ Z,
    float* h_out, int T, int d, int groups, long long n, bool own)
{
    constexpr int L = 8;
    const long long k = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (k >= n) return;
    const long long row = k / groups;
    const int group = (int)(k - row * groups), c0 = min(group * V, d - V);
    const int skip = own ? group * V - c0 : 0;
    float h[V];
    auto start = [&]() {
#pragma unroll
        for (int i = 0; i < V; ++i) h[i] = h0 ? h0[row * d + c0 + i] : 0.f;
    };
    start();
    float most = largest(0.f, h);
    const size_t first = (size_t)row * T * d + c0;
    size_t at = first;
    for (int t0 = 0; t0 < T; t0 += L, at += (size_t)L * d) {
        Raw<TIO, V, false> x[L], g[L];
#pragma unroll
        for (int l = 0; l < L; ++l) {
            if (t0 + l < T) {
                g[l].load(G + at + (size_t)l * d);
                x[l].load(X + at + (size_t)l * d);
            }
        }
#pragma unroll
        for (int l = 0; l < L; ++l) {
            if (t0 + l >= T) break;
            next<false>(g[l], x[l], h);
            most = largest(most, h);
            Raw<TIO, V, false> z;
            z.put(h);
            z.store_from(Z + at + (size_t)l * d, skip);
        }
    }
    if (isinf(most)) {
        start();
        at = first;
#pragma unroll 1
        for (int l = 0; l < T; ++l, at += d) {
            Raw<TIO, V, false> a, b;
            a.load(G + at);
            b.load(X + at);
            next<true>(a, b, h);
            b.put(h);
            b.store_from(Z + at, skip);
        }
    }
    if (h_out) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i >= skip) h_out[row * d + c0 + i] = h[i];
    }
}

long long tiles_of(const Layout& y, int T, int L)
{
    return (T + (long long)y.rows * L - 1) / ((long long)y.rows * L);
}

// Workgroups of 512 threads where they hold a row's tokens in one tile and ones of 256 do not: no
// chain to clear and to wait for.  bf16, d = 64, with 512 and with 256: 96 rows of 512 tokens,
// forward 11.3 and 14.3 us, backward 14.9 and 17.1; 256 rows 12.9 and 16.4, 18.0 and 21.2.  (Rows
// of two tiles and more gain nothing from 512: 96 x 2048 22.7 and 20.5 us.)  The backward kernel's
// registers allow one such workgroup a compute unit, so it takes them up to 256: 384 rows of 512
// are 31.3 and 25.9 us.
bool one_tile_of_512(const Layout& y256, const Layout& y512, bool bf16, int T, int L)
{
    return y256.V == (bf16 ? 8 : 4) && tiles_of(y256, T, L) > 1 && tiles_of(y512, T, L) == 1;
}

Layout fwd_layout(int T, int d, bool bf16)
{
    const Layout y = layout_of(d, bf16, 256), z = layout_of(d, bf16, 512);
    return one_tile_of_512(y, z, bf16, T, kRunFwd) ? z : y;
}

Layout bwd_layout(int BH, int T, int d, bool bf16)
{
    const Layout y = layout_of(d, bf16, 256), z = layout_of(d, bf16, 512);
    return one_tile_of_512(y, z, bf16, T, kRunBwd) && (long long)BH * z.blocks <= 256 ? z : y;
}

// Rows of one launch: a grid has room for fewer than 2^32 threads (a row of T d <= 2^34 has fewer
// than 2^30).  The rows beyond take further launches, one after the other in the same workspace.
constexpr long long kMostThreads = 0x7fffffff;

int rows_of(const Layout& y, int BH, long long tiles)
{
    return (int)std::min<long long>(BH, kMostThreads / (y.threads * (long long)y.blocks * tiles));
}

// p + n, or nullptr
template <typename T> T* shifted(T* p, size_t n) { return p ? p + n : nullptr; }

// Sets up the chain of a launch: the number of workgroups.
unsigned prepare(const Layout& y, int BH, int T, int L, void* ws, Chain& c, int& tiles, int& seqs,
                 hipStream_t s)
{
    const long long nt = tiles_of(y, T, L), ns = (long long)BH * y.blocks;
    tiles = (int)nt;
    seqs = (int)ns;
    c = Chain{};
    if (nt > 1) {
        const size_t bytes = chain_bytes(ns, nt, y.width, &c, ws);
        const size_t n = (bytes + 15) / 16, zeros = up256(4 * (size_t)kTicket * ns) / 16;
        hipLaunchKernelGGL(gated_clear_kernel,
                           dim3((unsigned)std::min<size_t>(2048, (n + kThreads - 1) / kThreads)),
                           dim3(kThreads), 0, s, (uint4*)ws, zeros, n);
    }
    return (unsigned)(nt * ns);
}

template <typename TIO, int V, int NT, bool LINES>
hipError_t fwd_nt(const GatedArgs& a, const Layout& y, hipStream_t s)
{
    const int per = rows_of(y, a.BH, tiles_of(y, a.T, kRunFwd));
    const bool in_place = a.h0 && a.h0 == a.h_out;
    for (long long row = 0; row < a.BH; row += per) {
        const size_t h = (size_t)row * a.d, at = h * a.T;
        const int rows = (int)std::min<long long>(per, a.BH - row);
        Chain c;
        int tiles, seqs;
        const unsigned grid = prepare(y, rows, a.T, kRunFwd, a.workspace, c, tiles, seqs, s);
        hipLaunchKernelGGL((gated_fwd_kernel<TIO, V, NT, LINES>), dim3(grid), dim3(NT), 0, s,
                           (const TIO*)a.X + at, (const TIO*)a.G + at, shifted(a.h0, h),
                           (TIO*)a.Z + at, shifted(a.h_out, h), a.T, a.d, tiles, seqs, y, c,
                           in_place);
    }
    return hipGetLastError();
}

template <typename TIO, int V, int NT, bool LINES>
hipError_t bwd_nt(const GatedBwdArgs& a, const Layout& y, hipStream_t s)
{
    const int per = rows_of(y, a.BH, tiles_of(y, a.T, kRunBwd));
    for (long long row = 0; row < a.BH; row += per) {
        const size_t h = (size_t)row * a.d, at = h * a.T;
        const int rows = (int)std::min<long long>(per, a.BH - row);
        Chain c;
        int tiles, seqs;
        const unsigned grid = prepare(y, rows, a.T, kRunBwd, a.workspace, c, tiles, seqs, s);
        hipLaunchKernelGGL((gated_bwd_kernel<TIO, V, NT, LINES>), dim3(grid), dim3(NT), 0, s,
                           (const TIO*)a.G + at, (const TIO*)a.Z + at, shifted(a.h0, h),
                           (const TIO*)a.dZ + at, shifted(a.dh_T, h), (TIO*)a.dX + at,
                           (TIO*)a.dG + at, shifted(a.dh0, h), a.T, a.d, tiles, seqs, y, c);
    }
    return hipGetLastError();
}

template <typename TIO, int V>
hipError_t fwd_v(const GatedArgs& a, const Layout& y, hipStream_t s)
{
    if constexpr (V * sizeof(TIO) == 16) {
        if (y.threads == 512)
            return y.lines ? fwd_nt<TIO, V, 512, true>(a, y, s) : fwd_nt<TIO, V, 512, false>(a, y, s);
        if (y.lines) return fwd_nt<TIO, V, 256, true>(a, y, s);
    }
    return fwd_nt<TIO, V, 256, false>(a, y, s);
}

template <typename TIO, int V>
hipError_t bwd_v(const GatedBwdArgs& a, const Layout& y, hipStream_t s)
{
    if constexpr (V * sizeof(TIO) == 16) {
        if (y.threads == 512)
            return y.lines ? bwd_nt<TIO, V, 512, true>(a, y, s) : bwd_nt<TIO, V, 512, false>(a, y, s);
        if (y.lines) return bwd_nt<TIO, V, 256, true>(a, y, s);
    }
    return bwd_nt<TIO, V, 256, false>(a, y, s);
}

template <typename TIO, int V>
hipError_t step_v(const GatedArgs& a, hipStream_t s)
{
    const int groups = (a.d + V - 1) / V;
    const long long per = kMostThreads / groups;
    const bool own = a.h0 && a.h0 == a.h_out;
    for (long long row = 0; row < a.BH; row += per) {
        const size_t h = (size_t)row * a.d, at = h * a.T;
        const long long n = std::min<long long>(per, a.BH - row) * groups;
        hipLaunchKernelGGL((gated_step_kernel<TIO, V>), dim3((unsigned)((n + kThreads - 1) / kThreads)),
                           dim3(kThreads), 0, s, (const TIO*)a.X + at, (const TIO*)a.G + at,
                           shifted(a.h0, h), (TIO*)a.Z + at, shifted(a.h_out, h), a.T, a.d, groups,
                           n, own);
    }
    return hipGetLastError();
}

// f(integral V) for the layout's V
#define GATED_BY_WIDTH(V, call)                                                          \
    switch (V) {                                                                         \
    case 1: { constexpr int W = 1; return call; }                                        \
    case 2: { constexpr int W = 2; return call; }                                        \
    case 4: { constexpr int W = 4; return call; }                                        \
    default: break;                                                                      \
    }

}  // namespace

size_t gated_workspace(int BH, int T, int d, bool bf16)
{
    size_t n = 0;
    auto add = [&](const Layout& y, int L) {
        const long long tiles = tiles_of(y, T, L);
        if (tiles > 1)
            n = std::max(n, chain_bytes((long long)rows_of(y, BH, tiles) * y.blocks, tiles, y.width,
                                        nullptr, nullptr));
    };
    add(fwd_layout(T, d, bf16), kRunFwd);
    add(bwd_layout(BH, T, d, bf16), kRunBwd);
    return n;
}

hipError_t launch_gated_step(const GatedArgs& a, hipStream_t s)
{
    const int V = layout_of(a.d, a.bf16, 256).V;
    if (a.bf16) {
        GATED_BY_WIDTH(V, (step_v<uint16_t, W>(a, s)))
        return step_v<uint16_t, 8>(a, s);
    }
    GATED_BY_WIDTH(V, (step_v<float, W>(a, s)))
    return hipErrorInvalidValue;
}

// The serial kernel also takes short rows: a tile of them is mostly empty, and costs its
// latencies all the same.  bf16, d = 64, serial / tiles: 1000 rows of 16 tokens 9.0 / 12.8 us, of
// 32 13.9 / 12.8; 10000 rows of 16 16 / 79, of 32 35 / 79, of 64 62 / 80.
hipError_t launch_gated_fwd(const GatedArgs& a, hipStream_t s)
{
    const Layout y = fwd_layout(a.T, a.d, a.bf16);
    const long long threads = (long long)a.BH * ((a.d + y.V - 1) / y.V);
    if (a.T <= 16 || (a.T <= 64 && threads >= 1 << 15)) return launch_gated_step(a, s);
    if (a.bf16) {
        GATED_BY_WIDTH(y.V, (fwd_v<uint16_t, W>(a, y, s)))
        return fwd_v<uint16_t, 8>(a, y, s);
    }
    GATED_BY_WIDTH(y.V, (fwd_v<float, W>(a, y, s)))
    return hipErrorInvalidValue;
}

hipError_t launch_gated_bwd(const GatedBwdArgs& a, hipStream_t s)
{
    const Layout y = bwd_layout(a.BH, a.T, a.d, a.bf16);
    if (a.bf16) {
        GATED_BY_WIDTH(y.V, (bwd_v<uint16_t, W>(a, y, s)))
        return bwd_v<uint16_t, 8>(a, y, s);
    }
    GATED_BY_WIDTH(y.V, (bwd_v<float, W>(a, y, s)))
    return hipErrorInvalidValue;
}

}  // namespace ttt
