// Internal launchers of the operators around the scan (gated recurrence, RMS norm,
// gradient clipping).  The C ABI (api_block.cpp) validates every argument before calling
// these; they only size grids and launch.
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

}  // namespace ttt
