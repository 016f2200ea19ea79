// C ABI of the operators around the scan: gated recurrence, RMS norm, gradient
// clipping (declared in include/ttt.h).  As in api.cpp every argument is checked here
// before any HIP call, and a failed check enqueues nothing.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "block_launch.h"
#include "host_checks.h"
#include "ttt.h"

using namespace ttt;

namespace {

constexpr int kMostFeatures = 1 << 26;

bool gated_dims_ok(int B, int H, int T, int d, int io_dtype)
{
    if (B <= 0 || H <= 0 || T <= 0 || d <= 0 || !dtype_ok(io_dtype)) return false;
    // token and feature counts with room in an int, rows inside 2^31, one row inside a grid, every
    // element index inside 2^60
    if (T > 1 << 30 || d > kMostFeatures || (long long)T * d > 1ll << 34) return false;
    const long double rows = (long double)B * H;
    return rows * T * d < 1.0e18L && rows < 2.0e9L;
}

bool rms_dims_ok(long long rows, int D)
{
    return rows >= 0 && D > 0 && D <= kMostFeatures && (long double)rows * D < 1.0e18L;
}

size_t elem_bytes(int io_dtype) { return io_dtype == TTT_DTYPE_BF16 ? 2 : 4; }

int gated_fwd_checked(const void* X, const void* G, const float* h0, void* Z, float* h_out, int B,
                      int H, int T, int d, int io_dtype, GatedArgs& a)
{
    if (!X || !G || !Z) return TTT_ERR_INVALID_ARG;
    if (!aligned(X, 16) || !aligned(G, 16) || !aligned(Z, 16) || !aligned(h0, 16) ||
        !aligned(h_out, 16))
        return TTT_ERR_INVALID_ARG;
    if (!gated_dims_ok(B, H, T, d, io_dtype)) return TTT_ERR_INVALID_ARG;
    const size_t state = (size_t)B * H * d, n = state * T * elem_bytes(io_dtype);
    if (overlap(Z, n, X, n) || overlap(Z, n, G, n)) return TTT_ERR_INVALID_ARG;
    if ((h0 && overlap(Z, n, h0, 4 * state)) || (h_out && overlap(Z, n, h_out, 4 * state)))
        return TTT_ERR_INVALID_ARG;
    if (h_out && (overlap(h_out, 4 * state, X, n) || overlap(h_out, 4 * state, G, n)))
        return TTT_ERR_INVALID_ARG;
    // the same place or none: a shifted overlap would hand one channel's state to another
    if (h0 && h_out && h0 != h_out && overlap(h0, 4 * state, h_out, 4 * state))
        return TTT_ERR_INVALID_ARG;
    a.X = X; a.G = G; a.h0 = h0; a.Z = Z; a.h_out = h_out;
    a.BH = B * H; a.T = T; a.d = d; a.bf16 = io_dtype == TTT_DTYPE_BF16;
    a.workspace = nullptr;
    return TTT_OK;
}

}  // namespace

extern "C" {

size_t ttt_gated_workspace_bytes(int B, int H, int T, int d, int io_dtype)
{
    if (!gated_dims_ok(B, H, T, d, io_dtype)) return 0;
    return gated_workspace(B * H, T, d, io_dtype == TTT_DTYPE_BF16);
}

int ttt_gated_fwd(const void* X, const void* G, const float* h0, void* Z, float* h_out, int B,
                  int H, int T, int d, int io_dtype, void* workspace, size_t workspace_bytes,
                  void* stream)
{
    GatedArgs a;
    const int rc = gated_fwd_checked(X, G, h0, Z, h_out, B, H, T, d, io_dtype, a);
    if (rc != TTT_OK) return rc;
    const size_t need = gated_workspace(a.BH, T, d, a.bf16);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
        return TTT_ERR_WORKSPACE;
    a.workspace = workspace;
    return launch_status(launch_gated_fwd(a, reinterpret_cast<hipStream_t>(stream)));
}

int ttt_gated_step(const void* X, const void* G, float* h, void* Z, int B, int H, int n, int d,
                   int io_dtype, void* stream)
{
    if (!h) return TTT_ERR_INVALID_ARG;
    GatedArgs a;
    const int rc = gated_fwd_checked(X, G, h, Z, h, B, H, n, d, io_dtype, a);
    if (rc != TTT_OK) return rc;
    return launch_status(launch_gated_step(a, reinterpret_cast<hipStream_t>(stream)));
}

int ttt_gated_bwd(const void* G, const void* Z, const float* h0, const void* dZ,
                  const float* dh_T, void* dX, void* dG, float* dh0, int B, int H, int T, int d,
                  int io_dtype, void* workspace, size_t workspace_bytes, void* stream)
{
    if (!G || !Z || !dZ || !dX || !dG) return TTT_ERR_INVALID_ARG;
    if (!aligned(G, 16) || !aligned(Z, 16) || !aligned(dZ, 16) || !aligned(dX, 16) ||
        !aligned(dG, 16) || !aligned(h0, 16) || !aligned(dh_T, 16) || !aligned(dh0, 16))
        return TTT_ERR_INVALID_ARG;
    if (!gated_dims_ok(B, H, T, d, io_dtype)) return TTT_ERR_INVALID_ARG;
    const size_t state = (size_t)B * H * d, n = state * T * elem_bytes(io_dtype);
    const struct { const void* p; size_t n; } in[] = {{G, n}, {Z, n}, {dZ, n}, {h0, 4 * state},
                                                      {dh_T, 4 * state}},
                                              out[] = {{dX, n}, {dG, n}, {dh0, 4 * state}};
    for (int i = 0; i < 3; ++i) {
        if (!out[i].p) continue;
        for (const auto& q : in)
            if (q.p && overlap(out[i].p, out[i].n, q.p, q.n)) return TTT_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (out[j].p && overlap(out[i].p, out[i].n, out[j].p, out[j].n))
                return TTT_ERR_INVALID_ARG;
    }
    const size_t need = gated_workspace(B * H, T, d, io_dtype == TTT_DTYPE_BF16);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
        return TTT_ERR_WORKSPACE;

    GatedBwdArgs a;
    a.G = G; a.Z = Z; a.h0 = h0; a.dZ = dZ; a.dh_T = dh_T; a.dX = dX; a.dG = dG; a.dh0 = dh0;
    a.BH = B * H; a.T = T; a.d = d; a.bf16 = io_dtype == TTT_DTYPE_BF16;
    a.workspace = workspace;
    return launch_status(launch_gated_bwd(a, reinterpret_cast<hipStream_t>(stream)));
}

static int rmsnorm_fwd(const void* X, const void* residual, const float* weight, float eps,
                       void* Y, float* scale, bool q8, void* R, long long rows, int D,
                       int io_dtype, void* stream)
{
    if (!rms_dims_ok(rows, D) || !dtype_ok(io_dtype)) return TTT_ERR_INVALID_ARG;
    if (!std::isnormal(eps) || !(eps > 0.f)) return TTT_ERR_INVALID_ARG;
    if (rows == 0) return TTT_OK;
    if (!X || !Y || (q8 && !scale)) return TTT_ERR_INVALID_ARG;
    if (!aligned(X, 16) || !aligned(residual, 16) || !aligned(Y, 16) || !aligned(R, 16) ||
        !aligned(weight, 4) || !aligned(scale, 4))
        return TTT_ERR_INVALID_ARG;
    const size_t n = (size_t)rows * D * elem_bytes(io_dtype), ny = q8 ? (size_t)rows * D : n;
    // an output may stand at an input's place only element for element
    const bool y_at_x = !q8 && Y == X;
    if ((!y_at_x && overlap(Y, ny, X, n)) || (residual && overlap(Y, ny, residual, n)))
        return TTT_ERR_INVALID_ARG;
    if (R && (overlap(R, n, Y, ny) || (R != X && overlap(R, n, X, n)) ||
              (residual && R != residual && overlap(R, n, residual, n))))
        return TTT_ERR_INVALID_ARG;
    if (weight && (overlap(weight, 4 * (size_t)D, Y, ny) || (R && overlap(weight, 4 * (size_t)D, R, n))))
        return TTT_ERR_INVALID_ARG;
    if (q8) {
        const size_t ns = 4 * (size_t)rows;
        if (overlap(scale, ns, X, n) || overlap(scale, ns, Y, ny) ||
            (residual && overlap(scale, ns, residual, n)) || (R && overlap(scale, ns, R, n)) ||
            (weight && overlap(scale, ns, weight, 4 * (size_t)D)))
            return TTT_ERR_INVALID_ARG;
    }

    RmsArgs a;
    a.X = X; a.residual = residual; a.weight = weight; a.eps = eps; a.Y = Y; a.scale = scale;
    a.R = R; a.rows = rows; a.D = D; a.bf16 = io_dtype == TTT_DTYPE_BF16;
    return launch_status(launch_rmsnorm_fwd(a, reinterpret_cast<hipStream_t>(stream)));
}

int ttt_rmsnorm_fwd(const void* X, const void* residual, const float* weight, float eps, void* Y,
                    void* R, long long rows, int D, int io_dtype, void* stream)
{
    return rmsnorm_fwd(X, residual, weight, eps, Y, nullptr, false, R, rows, D, io_dtype, stream);
}

int ttt_rmsnorm_q8_fwd(const void* X, const void* residual, const float* weight, float eps,
                       void* Y8, float* scale, void* R, long long rows, int D, int io_dtype,
                       void* stream)
{
    return rmsnorm_fwd(X, residual, weight, eps, Y8, scale, true, R, rows, D, io_dtype, stream);
}

size_t ttt_rmsnorm_bwd_workspace_bytes(long long rows, int D, int io_dtype)
{
    if (!rms_dims_ok(rows, D) || !dtype_ok(io_dtype)) return 0;
    return rmsnorm_bwd_workspace(rows, D, io_dtype == TTT_DTYPE_BF16);
}

int ttt_rmsnorm_bwd(const void* R, const float* weight, const void* dY, const void* dR, float eps,
                    void* dX, float* dweight, long long rows, int D, int io_dtype,
                    void* workspace, size_t workspace_bytes, void* stream)
{
    if (!rms_dims_ok(rows, D) || !dtype_ok(io_dtype)) return TTT_ERR_INVALID_ARG;
    if (!std::isnormal(eps) || !(eps > 0.f)) return TTT_ERR_INVALID_ARG;
    if (rows > 0 && (!R || !dY || !dX)) return TTT_ERR_INVALID_ARG;
    if (!aligned(R, 16) || !aligned(dY, 16) || !aligned(dR, 16) || !aligned(dX, 16) ||
        !aligned(weight, 4) || !aligned(dweight, 4))
        return TTT_ERR_INVALID_ARG;
    const size_t n = (size_t)rows * D * elem_bytes(io_dtype), nw = 4 * (size_t)D;
    if (rows > 0) {
        if (overlap(dX, n, R, n) || (dX != dY && overlap(dX, n, dY, n)) ||
            (dR && dX != dR && overlap(dX, n, dR, n)) || (weight && overlap(dX, n, weight, nw)))
            return TTT_ERR_INVALID_ARG;
        if (dweight && (overlap(dweight, nw, R, n) || overlap(dweight, nw, dY, n) ||
                        overlap(dweight, nw, dX, n) || (dR && overlap(dweight, nw, dR, n))))
            return TTT_ERR_INVALID_ARG;
    }
    if (dweight && weight && overlap(dweight, nw, weight, nw)) return TTT_ERR_INVALID_ARG;
    const size_t need = rmsnorm_bwd_workspace(rows, D, io_dtype == TTT_DTYPE_BF16);
    if (dweight && need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
        return TTT_ERR_WORKSPACE;
    if (rows == 0 && !dweight) return TTT_OK;

    RmsBwdArgs a;
    a.R = R; a.weight = weight; a.dY = dY; a.dR = dR; a.eps = eps; a.dX = dX;
    a.dweight = dweight; a.rows = rows; a.D = D; a.bf16 = io_dtype == TTT_DTYPE_BF16;
    a.workspace = workspace;
    return launch_status(launch_rmsnorm_bwd(a, reinterpret_cast<hipStream_t>(stream)));
}

size_t ttt_clip_workspace_bytes(void) { return clip_workspace(); }

int ttt_clip_grad_norm(int n, const void* const* grads, void* const* outs,
                       const long long* sizes, const int* dtypes, float max_norm, float eps,
                       float* norm, void* workspace, size_t workspace_bytes, void* stream)
{
    if (n < 0 || (n > 0 && (!grads || !sizes || !dtypes)) || !norm || !aligned(norm, 4))
        return TTT_ERR_INVALID_ARG;
    if (!(max_norm >= 0.f) || !(eps > 0.f) || !std::isfinite(eps)) return TTT_ERR_INVALID_ARG;
    struct Range { uintptr_t lo, hi; bool out; int i; };
    std::vector<Range> ranges;
    try {
        ranges.reserve(2 * (size_t)n);
        long double total = 0;
        for (int i = 0; i < n; ++i) {
            if (sizes[i] < 0 || !dtype_ok(dtypes[i])) return TTT_ERR_INVALID_ARG;
            if (sizes[i] == 0) continue;
            total += sizes[i];
            if (total >= 1.0e18L) return TTT_ERR_INVALID_ARG;
            const size_t e = elem_bytes(dtypes[i]), bytes = (size_t)sizes[i] * e;
            if (!grads[i] || !aligned(grads[i], e)) return TTT_ERR_INVALID_ARG;
            const uintptr_t g = reinterpret_cast<uintptr_t>(grads[i]);
            if (overlap(grads[i], bytes, norm, 4)) return TTT_ERR_INVALID_ARG;
            if (!outs) continue;
            if (!outs[i] || !aligned(outs[i], e)) return TTT_ERR_INVALID_ARG;
            const uintptr_t o = reinterpret_cast<uintptr_t>(outs[i]);
            ranges.push_back({o, o + bytes, true, i});
            if (o != g) ranges.push_back({g, g + bytes, false, i});
            if (overlap(outs[i], bytes, norm, 4)) return TTT_ERR_INVALID_ARG;
        }
    } catch (const std::bad_alloc&) {
        return TTT_ERR_INVALID_ARG;
    }
    // in address order, no output may reach into what follows it or start inside what
    // came before; inputs may overlap each other
    std::sort(ranges.begin(), ranges.end(),
              [](const Range& x, const Range& y) { return x.lo < y.lo; });
    uintptr_t end_out = 0, end_any = 0;
    for (const Range& r : ranges) {
        if (r.lo < end_out || (r.out && r.lo < end_any)) return TTT_ERR_INVALID_ARG;
        end_any = std::max(end_any, r.hi);
        if (r.out) end_out = std::max(end_out, r.hi);
    }
    if (!workspace || workspace_bytes < clip_workspace() || !aligned(workspace, 256))
        return TTT_ERR_WORKSPACE;

    ClipArgs a;
    a.n = n; a.grads = grads; a.outs = outs; a.sizes = sizes; a.dtypes = dtypes;
    a.max_norm = max_norm; a.eps = eps; a.norm = norm; a.workspace = workspace;
    return launch_status(launch_clip(a, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
