// Internal launchers of the operators around the scan (gated recurrence, RMS norm,
// gradient clipping: validated by the C ABI in api_block.cpp; group norm, dropout: in
// api_delta.cpp).  Arguments are valid here; these only size grids and launch.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>

namespace ttt {

// Gated linear recurrence over BH rows of [T, d], T d <= 2^34; any d.
struct GatedArgs {
    const void* X;
    const void* G;
    const float* h0;       // [BH, d] or nullptr (zero)
    void* Z;
    float* h_out;          // [BH, d] or nullptr; may be h0
    int BH, T, d;
    int bf16;
    void* workspace;
};
hipError_t launch_gated_fwd(const GatedArgs& a, hipStream_t s);
// the same by one thread per channel group, serial over the tokens (no workspace)
hipError_t launch_gated_step(const GatedArgs& a, hipStream_t s);

struct GatedBwdArgs {
    const void* G;
    const void* Z;
    const float* h0;       // [BH, d] or nullptr
    const void* dZ;
    const float* dh_T;     // [BH, d] or nullptr
    void* dX;
    void* dG;
    float* dh0;            // [BH, d] or nullptr
    int BH, T, d;
    int bf16;
    void* workspace;
};
hipError_t launch_gated_bwd(const GatedBwdArgs& a, hipStream_t s);
size_t gated_workspace(int BH, int T, int d, bool bf16);

// Root-mean-square norm over rows of D features.
struct RmsArgs {
    const void* X;
    const void* residual;  // or nullptr
    const float* weight;   // or nullptr (ones)
    float eps;
    void* Y;               // I/O type, or e4m3 bytes where scale is set
    float* scale;          // [rows] or nullptr
    void* R;               // or nullptr
    long long rows;
    int D;
    int bf16;
};
hipError_t launch_rmsnorm_fwd(const RmsArgs& a, hipStream_t s);

struct RmsBwdArgs {
    const void* R;
    const float* weight;   // or nullptr
    const void* dY;
    const void* dR;        // or nullptr
    float eps;
    void* dX;
    float* dweight;        // or nullptr
    long long rows;
    int D;
    int bf16;
    void* workspace;
};
hipError_t launch_rmsnorm_bwd(const RmsBwdArgs& a, hipStream_t s);
size_t rmsnorm_bwd_workspace(long long rows, int D, bool bf16);

// Norm over many tensors and their scaling (host arrays of n entries).
struct ClipArgs {
    int n;
    const void* const* grads;
    void* const* outs;     // or nullptr
    const long long* sizes;
    const int* dtypes;
    float max_norm, eps;
    float* norm;
    void* workspace;
};
hipError_t launch_clip(const ClipArgs& a, hipStream_t s);
size_t clip_workspace();

// Group norm with an activation over channels-last tensors [N, S, C] (act: ttt_act).
struct GroupArgs {
    const void* X;
    const float *weight, *bias;   // [C] or nullptr
    float eps;
    void* Y;
    float *mean, *rstd;           // [N, G]
    long long N, S;
    int C, G, act;
    int bf16;
    void* workspace;
};
hipError_t launch_groupnorm_fwd(const GroupArgs& a, hipStream_t s);
size_t groupnorm_fwd_workspace(long long N, long long S, int C, int G, bool bf16);

struct GroupBwdArgs {
    const void *X, *dY;
    const float *weight, *bias, *mean, *rstd;
    void* dX;
    float *dweight, *dbias;       // [C] or nullptr
    long long N, S;
    int C, G, act;
    int bf16;
    void* workspace;
};
hipError_t launch_groupnorm_bwd(const GroupBwdArgs& a, hipStream_t s);
size_t groupnorm_bwd_workspace(long long N, long long S, int C, int G, bool bf16);

// Dropout by a counter-based generator, with the residual's addition.
struct DropoutArgs {
    const void* X;
    const void* residual;         // or nullptr
    void* Y;
    long long n;
    const long long* rng;         // device: seed, first counter
    unsigned threshold;           // of 2^32
    float scale;
    int bf16;
};
hipError_t launch_dropout(const DropoutArgs& a, hipStream_t s);

}  // namespace ttt
