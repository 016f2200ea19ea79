// Internal launchers of the gated delta rule.  The C ABI (api_delta.cpp) validates every
// argument before calling these; they only size grids and launch.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ttt {

constexpr int kDeltaMostDk = 128, kDeltaMostDv = 256;

struct DeltaArgs {
    const void *K, *Q, *V;   // tokens of [B, Hk, T, dk], the same, [B, H, T, dv]
    const float* eta;        // [B, H, T] or nullptr
    float eta_scalar;
    const float* g;          // [B, H, T] or nullptr (no decay)
    const float* W0;         // [B, H, dv, dk] or nullptr (zero)
    void* Z;
    float* W_out;            // or nullptr
    int B, H, Hk, T, dk, dv;
    bool tokens_first;       // [B, T, H, d] instead of [B, H, T, d]
    bool bf16;
    void* workspace;
};
hipError_t launch_delta_fwd(const DeltaArgs& a, hipStream_t s);
// token after token, the state in registers (no workspace)
hipError_t launch_delta_step(const DeltaArgs& a, hipStream_t s);
size_t delta_fwd_workspace(int B, int H, int Hk, int T, int dk, int dv, bool bf16);

struct DeltaBwdArgs {
    DeltaArgs f;             // the forward call's inputs
    const void* dZ;
    const float* dW_T;       // or nullptr
    void *dK, *dQ, *dV;
    float *deta, *dg;        // or nullptr
    float* dW0;              // or nullptr
};
hipError_t launch_delta_bwd(const DeltaBwdArgs& a, hipStream_t s);
size_t delta_bwd_workspace(int B, int H, int Hk, int T, int dk, int dv, bool bf16);

// ---- what the kernels of one pass over some of the heads are given --------------
struct Record;
typedef uint32_t quad __attribute__((ext_vector_type(4)));
typedef float float4x __attribute__((ext_vector_type(4)));

// segments of a sequence, chunks of each, 32 columns a workgroup (or 64)
struct DeltaCut {
    int segments, chunks;
    bool narrow;
};

struct DeltaPass {
    DeltaArgs f;
    int head0, heads;        // heads of values, counted through the batch: whole groups
    int chunks;              // of 64 tokens
    int dvp;                 // dv up to a multiple of 32
    Record* records;         // [heads][chunks]
    // S, its transpose (backward) and P (or its transpose): tiles, or operands in parts
    float4x *S, *St, *P;
    float *states, *cotangents;   // [heads][chunks][DK][dvp]: W^T before a chunk, D^T after it
    float *U, *F;            // [heads][chunks][64][dvp]
    DeltaCut cut;
    float *ends, *ends_back; // [heads][segments][DK][dvp]: states and their gradients past a segment
    float* transitions;      // [heads][segments][DK][DK]
};
// decays, S and P (transposed: S, its transpose and P's) of every chunk
hipError_t launch_delta_prepare(const DeltaPass& p, bool backward, hipStream_t s);
// the scan over the chunks; with `o` both scans of a backward pass, which keep states, U, D and F
hipError_t launch_delta_scans(const DeltaPass& p, const DeltaBwdArgs* o, hipStream_t s);
DeltaCut delta_cut(int heads, int chunks, int dv, int dk, bool backward);
// features of a head as the kernels hold them
inline int delta_padded_dk(int dk) { return dk <= 32 ? 32 : dk <= 64 ? 64 : 128; }

}  // namespace ttt
