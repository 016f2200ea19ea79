// C ABI of the gated delta rule, group norm and dropout (declared in include/ttt.h).  As in
// api.cpp every argument is checked here before any HIP call, and a failed check enqueues
// nothing.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "block_launch.h"
#include "delta_launch.h"
#include "host_checks.h"
#include "ttt.h"

using namespace ttt;

namespace {

size_t elem_bytes(int io_dtype) { return io_dtype == TTT_DTYPE_BF16 ? 2 : 4; }

// an output and what it must not share memory with
struct Span {
    const void* p;
    size_t n;
};

// no output over an input or another output
template <int NO, int NI>
bool apart(const Span (&out)[NO], const Span (&in)[NI])
{
    for (int i = 0; i < NO; ++i) {
        if (!out[i].p) continue;
        for (const Span& q : in)
            if (q.p && overlap(out[i].p, out[i].n, q.p, q.n)) return false;
        for (int j = 0; j < i; ++j)
            if (out[j].p && overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return false;
    }
    return true;
}

int delta_dims(int B, int H, int Hk, int T, int dk, int dv, int io_dtype)
{
    if (B <= 0 || H <= 0 || Hk <= 0 || T <= 0 || dk <= 0 || dv <= 0 || !dtype_ok(io_dtype) || H % Hk)
        return TTT_ERR_INVALID_ARG;
    if (dk > kDeltaMostDk || dv > kDeltaMostDv) return TTT_ERR_UNSUPPORTED;
    // token counts with room in an int; 16-row blocks of states, and the chunks of the heads that
    // share keys, inside a grid (2^32 threads of 256 a workgroup)
    const long double heads = (long double)B * H, most = 16777216.0L;
    if (T > 1 << 30 || heads * ((dv + 15) / 16) >= most || (long double)(H / Hk) * ((T + 63) / 64) >= most)
        return TTT_ERR_INVALID_ARG;
    return TTT_OK;
}

// Few tokens go token by token: no preparing kernel, no workspace.  (us a call, by token and by
// chunk: 8 x 12 heads of 64 features, 17 tokens 15.6 and 19.5, 24 tokens 20.0 and 19.6; 1 x 32 of
// 128, 16 tokens 19.5 and 20.3, 24 tokens 27 and 20; 64 x 16 of 64, 17 tokens 35 and 50.)
bool delta_by_token(int T) { return T <= 16; }

struct DeltaSizes {
    size_t keys, values, scalars, state;    // bytes
};

int delta_checked(const void* K, const void* Q, const void* V, const float* eta, float eta_scalar,
                  const float* g, const float* W0, int B, int H, int Hk, int T, int dk, int dv, int layout,
                  int io_dtype, DeltaArgs& a, DeltaSizes& n)
{
    if (!K || !Q || !V) return TTT_ERR_INVALID_ARG;
    if (!aligned(K, 16) || !aligned(Q, 16) || !aligned(V, 16) || !aligned(W0, 16) || !aligned(eta, 4) ||
        !aligned(g, 4))
        return TTT_ERR_INVALID_ARG;
    if (layout != TTT_LAYOUT_BHTD && layout != TTT_LAYOUT_BTHD) return TTT_ERR_INVALID_ARG;
    if (!eta && !std::isfinite(eta_scalar)) return TTT_ERR_INVALID_ARG;
    const int rc = delta_dims(B, H, Hk, T, dk, dv, io_dtype);
    if (rc != TTT_OK) return rc;
    const size_t e = elem_bytes(io_dtype), tokens = (size_t)B * T;
    n.keys = tokens * Hk * dk * e;
    n.values = tokens * H * dv * e;
    n.scalars = tokens * H * 4;
    n.state = (size_t)B * H * dv * dk * 4;
    a = DeltaArgs();
    a.K = K; a.Q = Q; a.V = V; a.eta = eta; a.eta_scalar = eta_scalar; a.g = g; a.W0 = W0;
    a.Z = nullptr; a.W_out = nullptr;
    a.B = B; a.H = H; a.Hk = Hk; a.T = T; a.dk = dk; a.dv = dv;
    a.tokens_first = layout == TTT_LAYOUT_BTHD;
    a.bf16 = io_dtype == TTT_DTYPE_BF16;
    a.workspace = nullptr;
    return TTT_OK;
}

int delta_outputs(DeltaArgs& a, const DeltaSizes& n, void* Z, float* W_out)
{
    if (!Z || !aligned(Z, 16) || !aligned(W_out, 16)) return TTT_ERR_INVALID_ARG;
    const Span out[] = {{Z, n.values}, {W_out, n.state}};
    // the state may stand at its own place, which is read before it is written
    const Span in[] = {{a.K, n.keys}, {a.Q, n.keys}, {a.V, n.values}, {a.eta, n.scalars}, {a.g, n.scalars},
                       {a.W0 == W_out ? nullptr : a.W0, n.state}};
    if (!apart(out, in)) return TTT_ERR_INVALID_ARG;
    if (a.W0 && overlap(Z, n.values, a.W0, n.state)) return TTT_ERR_INVALID_ARG;
    a.Z = Z;
    a.W_out = W_out;
    return TTT_OK;
}

bool group_dims_ok(long long N, long long S, int C, int G, int io_dtype)
{
    if (N < 0 || S < 0 || C <= 0 || G <= 0 || C % G || C > 1 << 20 || !dtype_ok(io_dtype)) return false;
    // every element index inside 2^59; groups of rows, and rows by 256 channels, in an int (the
    // kernels' grids go on along further axes from 2^22 workgroups on)
    return (long double)N * S * C < 5.0e17L && (long double)N * G < 2147483648.0L &&
           (long double)N * ((C + 255) / 256) < 2147483648.0L;
}

bool act_ok(int act) { return act == TTT_ACT_NONE || act == TTT_ACT_SILU || act == TTT_ACT_GELU; }

bool workspace_ok(const void* p, size_t have, size_t need)
{
    return need == 0 || (p && have >= need && aligned(p, 256));
}

}  // namespace

extern "C" {

size_t ttt_delta_workspace_bytes(int B, int H, int Hk, int T, int dk, int dv, int io_dtype)
{
    if (delta_dims(B, H, Hk, T, dk, dv, io_dtype) != TTT_OK || delta_by_token(T)) return 0;
    return delta_fwd_workspace(B, H, Hk, T, dk, dv, io_dtype == TTT_DTYPE_BF16);
}

int ttt_delta_fwd(const void* K, const void* Q, const void* V, const float* eta, float eta_scalar,
                  const float* g, const float* W0, void* Z, float* W_out, int B, int H, int Hk, int T,
                  int dk, int dv, int layout, int io_dtype, void* workspace, size_t workspace_bytes,
                  void* stream)
{
    DeltaArgs a;
    DeltaSizes n;
    int rc = delta_checked(K, Q, V, eta, eta_scalar, g, W0, B, H, Hk, T, dk, dv, layout, io_dtype, a, n);
    if (rc == TTT_OK) rc = delta_outputs(a, n, Z, W_out);
    if (rc != TTT_OK) return rc;
    if (delta_by_token(T)) return launch_status(launch_delta_step(a, reinterpret_cast<hipStream_t>(stream)));
    if (!workspace_ok(workspace, workspace_bytes, delta_fwd_workspace(B, H, Hk, T, dk, dv, a.bf16)))
        return TTT_ERR_WORKSPACE;
    a.workspace = workspace;
    return launch_status(launch_delta_fwd(a, reinterpret_cast<hipStream_t>(stream)));
}

int ttt_delta_step(const void* K, const void* Q, const void* V, const float* eta, float eta_scalar,
                   const float* g, float* W, void* Z, int B, int H, int Hk, int n, int dk, int dv,
                   int layout, int io_dtype, void* stream)
{
    if (!W) return TTT_ERR_INVALID_ARG;
    DeltaArgs a;
    DeltaSizes sizes;
    int rc = delta_checked(K, Q, V, eta, eta_scalar, g, W, B, H, Hk, n, dk, dv, layout, io_dtype, a, sizes);
    if (rc == TTT_OK) rc = delta_outputs(a, sizes, Z, W);
    if (rc != TTT_OK) return rc;
    return launch_status(launch_delta_step(a, reinterpret_cast<hipStream_t>(stream)));
}

size_t ttt_delta_bwd_workspace_bytes(int B, int H, int Hk, int T, int dk, int dv, int io_dtype)
{
    if (delta_dims(B, H, Hk, T, dk, dv, io_dtype) != TTT_OK) return 0;
    return delta_bwd_workspace(B, H, Hk, T, dk, dv, io_dtype == TTT_DTYPE_BF16);
}

int ttt_delta_bwd(const void* K, const void* Q, const void* V, const float* eta, float eta_scalar,
                  const float* g, const float* W0, const void* dZ, const float* dW_T, void* dK, void* dQ,
                  void* dV, float* deta, float* dg, float* dW0, int B, int H, int Hk, int T, int dk, int dv,
                  int layout, int io_dtype, void* workspace, size_t workspace_bytes, void* stream)
{
    DeltaBwdArgs a;
    DeltaSizes n;
    const int rc =
        delta_checked(K, Q, V, eta, eta_scalar, g, W0, B, H, Hk, T, dk, dv, layout, io_dtype, a.f, n);
    if (rc != TTT_OK) return rc;
    if (!dZ || !dK || !dQ || !dV) return TTT_ERR_INVALID_ARG;
    if (!aligned(dZ, 16) || !aligned(dW_T, 16) || !aligned(dK, 16) || !aligned(dQ, 16) || !aligned(dV, 16) ||
        !aligned(dW0, 16) || !aligned(deta, 4) || !aligned(dg, 4))
        return TTT_ERR_INVALID_ARG;
    const Span out[] = {{dK, n.keys}, {dQ, n.keys}, {dV, n.values}, {deta, n.scalars}, {dg, n.scalars},
                        {dW0, n.state}};
    const Span in[] = {{K, n.keys}, {Q, n.keys}, {V, n.values}, {eta, n.scalars}, {g, n.scalars},
                       {W0, n.state}, {dZ, n.values}, {dW_T, n.state}};
    if (!apart(out, in)) return TTT_ERR_INVALID_ARG;
    if (!workspace_ok(workspace, workspace_bytes, delta_bwd_workspace(B, H, Hk, T, dk, dv, a.f.bf16)))
        return TTT_ERR_WORKSPACE;
    a.f.workspace = workspace;
    a.dZ = dZ; a.dW_T = dW_T; a.dK = dK; a.dQ = dQ; a.dV = dV; a.deta = deta; a.dg = dg; a.dW0 = dW0;
    return launch_status(launch_delta_bwd(a, reinterpret_cast<hipStream_t>(stream)));
}

size_t ttt_groupnorm_workspace_bytes(long long N, long long S, int C, int G, int io_dtype)
{
    if (!group_dims_ok(N, S, C, G, io_dtype) || N == 0 || S == 0) return 0;
    return groupnorm_fwd_workspace(N, S, C, G, io_dtype == TTT_DTYPE_BF16);
}

int ttt_groupnorm_fwd(const void* X, const float* weight, const float* bias, float eps, int act, void* Y,
                      float* mean, float* rstd, long long N, long long S, int C, int G, int io_dtype,
                      void* workspace, size_t workspace_bytes, void* stream)
{
    if (!group_dims_ok(N, S, C, G, io_dtype) || !act_ok(act)) return TTT_ERR_INVALID_ARG;
    if (!std::isnormal(eps) || !(eps > 0.f)) return TTT_ERR_INVALID_ARG;
    if (N == 0 || S == 0) return TTT_OK;
    if (!X || !Y || !mean || !rstd) return TTT_ERR_INVALID_ARG;
    if (!aligned(X, 16) || !aligned(Y, 16) || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(mean, 4) ||
        !aligned(rstd, 4))
        return TTT_ERR_INVALID_ARG;
    const size_t n = (size_t)N * S * C * elem_bytes(io_dtype), per = 4 * (size_t)C, st = 4 * (size_t)N * G;
    const Span out[] = {{Y, n}, {mean, st}, {rstd, st}};
    const Span in[] = {{X == Y ? nullptr : X, n}, {weight, per}, {bias, per}};
    if (!apart(out, in) || overlap(mean, st, X, n) || overlap(rstd, st, X, n)) return TTT_ERR_INVALID_ARG;
    GroupArgs a;
    a.X = X; a.weight = weight; a.bias = bias; a.eps = eps; a.Y = Y; a.mean = mean; a.rstd = rstd;
    a.N = N; a.S = S; a.C = C; a.G = G; a.act = act; a.bf16 = io_dtype == TTT_DTYPE_BF16;
    a.workspace = workspace;
    if (!workspace_ok(workspace, workspace_bytes, groupnorm_fwd_workspace(N, S, C, G, a.bf16)))
        return TTT_ERR_WORKSPACE;
    return launch_status(launch_groupnorm_fwd(a, reinterpret_cast<hipStream_t>(stream)));
}

size_t ttt_groupnorm_bwd_workspace_bytes(long long N, long long S, int C, int G, int io_dtype)
{
    if (!group_dims_ok(N, S, C, G, io_dtype) || N == 0 || S == 0) return 0;
    return groupnorm_bwd_workspace(N, S, C, G, io_dtype == TTT_DTYPE_BF16);
}

int ttt_groupnorm_bwd(const void* X, const float* weight, const float* bias, int act, const float* mean,
                      const float* rstd, const void* dY, void* dX, float* dweight, float* dbias, long long N,
                      long long S, int C, int G, int io_dtype, void* workspace, size_t workspace_bytes,
                      void* stream)
{
    if (!group_dims_ok(N, S, C, G, io_dtype) || !act_ok(act)) return TTT_ERR_INVALID_ARG;
    if (!aligned(weight, 4) || !aligned(bias, 4) || !aligned(mean, 4) || !aligned(rstd, 4) ||
        !aligned(dweight, 4) || !aligned(dbias, 4))
        return TTT_ERR_INVALID_ARG;
    const bool empty = N == 0 || S == 0;
    const size_t n = (size_t)N * S * C * elem_bytes(io_dtype), per = 4 * (size_t)C, st = 4 * (size_t)N * G;
    if (!empty) {
        if (!X || !mean || !rstd || !dY || !dX) return TTT_ERR_INVALID_ARG;
        if (!aligned(X, 16) || !aligned(dY, 16) || !aligned(dX, 16)) return TTT_ERR_INVALID_ARG;
    }
    const Span out[] = {{empty ? nullptr : dX, n}, {dweight, per}, {dbias, per}};
    const Span in[] = {{X == dX ? nullptr : X, n}, {dY == dX ? nullptr : dY, n}, {weight, per}, {bias, per},
                       {mean, st}, {rstd, st}};
    if (!apart(out, in)) return TTT_ERR_INVALID_ARG;
    for (const float* sums : {dweight, dbias})
        if (sums && !empty && (overlap(sums, per, X, n) || overlap(sums, per, dY, n))) return TTT_ERR_INVALID_ARG;
    GroupBwdArgs a;
    a.X = X; a.dY = dY; a.weight = weight; a.bias = bias; a.mean = mean; a.rstd = rstd;
    a.dX = dX; a.dweight = dweight; a.dbias = dbias;
    a.N = N; a.S = S; a.C = C; a.G = G; a.act = act; a.bf16 = io_dtype == TTT_DTYPE_BF16;
    a.workspace = workspace;
    if (!empty && !workspace_ok(workspace, workspace_bytes, groupnorm_bwd_workspace(N, S, C, G, a.bf16)))
        return TTT_ERR_WORKSPACE;
    return launch_status(launch_groupnorm_bwd(a, reinterpret_cast<hipStream_t>(stream)));
}

int ttt_dropout(const void* X, const void* residual, void* Y, long long n, double p, const long long* rng,
                int io_dtype, void* stream)
{
    if (n < 0 || n > 1ll << 59 || !dtype_ok(io_dtype) || !(p >= 0.0) || !(p < 1.0)) return TTT_ERR_INVALID_ARG;
    if (n == 0) return TTT_OK;
    if (!X || !Y || !rng) return TTT_ERR_INVALID_ARG;
    if (!aligned(X, 16) || !aligned(residual, 16) || !aligned(Y, 16) || !aligned(rng, 8))
        return TTT_ERR_INVALID_ARG;
    const size_t bytes = (size_t)n * elem_bytes(io_dtype);
    if ((X != Y && overlap(Y, bytes, X, bytes)) ||
        (residual && residual != Y && overlap(Y, bytes, residual, bytes)) || overlap(Y, bytes, rng, 16))
        return TTT_ERR_INVALID_ARG;
    DropoutArgs a;
    a.X = X; a.residual = residual; a.Y = Y; a.n = n; a.rng = rng;
    a.threshold = (unsigned)std::min(std::llrint(p * 4294967296.0), 4294967295ll);
    a.scale = (float)(1.0 / (1.0 - p));
    a.bf16 = io_dtype == TTT_DTYPE_BF16;
    return launch_status(launch_dropout(a, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
