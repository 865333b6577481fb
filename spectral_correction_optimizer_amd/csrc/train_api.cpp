// C entries of the training-step operators (include/scopt.h): arguments are checked before
// any GPU work, then the launchers of train.hpp enqueue.
#include <hip/hip_runtime.h>

#include "internal.hpp"
#include "scopt.h"
#include "train.hpp"

using namespace scopt;

namespace {

#define HIP_TRY(expr)                                                                      \
    do {                                                                                   \
        hipError_t e_ = (expr);                                                            \
        if (e_ != hipSuccess)                                                              \
            return fail(SC_ERR_HIP, "%s failed: %s (%s:%d)", #expr, hipGetErrorString(e_), \
                        __FILE__, __LINE__);                                               \
    } while (0)
#define SC_TRY(expr)          \
    do {                      \
        int rc_ = (expr);     \
        if (rc_) return rc_;  \
    } while (0)

constexpr int64_t kMaxTokens = (int64_t)1 << 31;  // embedding gradient: half of it, its indexes are 32-bit
constexpr int64_t kMaxVocab = (int64_t)1 << 22;
constexpr int kMaxEmbedH = 1 << 24;
constexpr int64_t kMaxEmbedTasks = ((int64_t)1 << 26) - 4;  // of 64 threads: a launch has fewer than 2^32
constexpr int kNormMaxH = 16384;
constexpr int64_t kMaxProduct = (int64_t)1 << 21;  // sizes of a product's operands
constexpr int64_t kXentLimit = (int64_t)4 << 30;
constexpr int64_t kMaxPairs = (int64_t)1 << 20;
constexpr int kMaxTensors = 1 << 20;
constexpr int64_t kMaxGrad = (int64_t)1 << 48;  // elements of all gradients

int check_dtype(sc_dtype dtype) {
    if (dtype != SC_F32 && dtype != SC_BF16) return fail(SC_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    return SC_OK;
}
int check_size(const char* what, int64_t n, int64_t lo, int64_t hi) {
    if (n < lo || n > hi)
        return fail(SC_ERR_SHAPE, "%s = %lld out of range [%lld, %lld]", what, (long long)n, (long long)lo,
                    (long long)hi);
    return SC_OK;
}
int check_ptr(const char* what, const void* p, uintptr_t align) {
    if (!p) return fail(SC_ERR_INVALID_ARG, "%s is NULL", what);
    if ((uintptr_t)p & (align - 1))
        return fail(SC_ERR_INVALID_ARG, "%s is not %d-byte aligned", what, (int)align);
    return SC_OK;
}
uintptr_t elem(sc_dtype dtype) { return dtype == SC_BF16 ? 2 : 4; }
int check_workspace(const void* p, int64_t have, int64_t need) {
    if (have < need)
        return fail(SC_ERR_INVALID_ARG, "workspace of %lld bytes, %lld needed", (long long)have, (long long)need);
    return need > 0 ? check_ptr("workspace", p, 16) : SC_OK;
}
int check_embed(int64_t T, int64_t V, int H) {
    SC_TRY(check_size("T", T, 0, kMaxTokens - 1));
    SC_TRY(check_size("V", V, 1, kMaxVocab));
    return check_size("H", H, 1, kMaxEmbedH);
}
int check_embed_grad(int64_t T, int64_t V, int H) {
    SC_TRY(check_size("T", T, 0, kMaxTokens / 2 - 1));
    SC_TRY(check_embed(T, V, H));
    return check_size("(T / 32 + V / 8) * ceil(H / 512)", embed_grad_plan(T, V, H).tasks, 0, kMaxEmbedTasks);
}
int check_rows(int64_t T, int H, int maxH) {
    SC_TRY(check_size("T", T, 0, kMaxTokens - 1));
    return check_size("H", H, 1, maxH);
}
int check_xent(sc_dtype dtype, int64_t T, int64_t V, int H, int64_t limit) {
    SC_TRY(check_dtype(dtype));
    SC_TRY(check_size("T", T, 0, kMaxProduct - 1));
    SC_TRY(check_size("V", V, 1, kMaxProduct - 1));
    SC_TRY(check_size("H", H, 1, 65535));
    if (limit < 0) return fail(SC_ERR_INVALID_ARG, "negative limit");
    return SC_OK;
}
int check_wgrad(sc_dtype dtype, int64_t T, int64_t N, int H) {
    SC_TRY(check_dtype(dtype));
    SC_TRY(check_size("T", T, 0, kMaxProduct - 1));
    SC_TRY(check_size("N", N, 1, kMaxProduct - 1));
    return check_size("H", H, 1, kMaxProduct - 1);
}
// Arguments that the losses of tokens share
int check_token_loss(sc_dtype dtype, const void* h, const void* W, const int64_t* targets, int64_t T, int64_t V, int H,
                     const float* logp, const void* dh, const void* dW) {
    SC_TRY(check_ptr("dW", dW, elem(dtype)));
    if (T == 0) return SC_OK;
    SC_TRY(check_ptr("h", h, 16));
    SC_TRY(check_ptr("W", W, 16));
    SC_TRY(check_ptr("targets", targets, 8));
    SC_TRY(check_ptr("logp", logp, 4));
    return check_ptr("dh", dh, elem(dtype));
}
int check_grads(int n, const sc_dtype* dtypes, const int64_t* sizes) {
    if (n < 0 || n > kMaxTensors) return fail(SC_ERR_INVALID_ARG, "%d tensors", n);
    if (n > 0 && (!dtypes || !sizes)) return fail(SC_ERR_INVALID_ARG, "dtypes or sizes is NULL");
    int64_t all = 0;
    for (int i = 0; i < n; ++i) {
        SC_TRY(check_dtype(dtypes[i]));
        SC_TRY(check_size("a tensor's size", sizes[i], 0, kMaxGrad));
        all += sizes[i];
        SC_TRY(check_size("elements of all tensors", all, 0, kMaxGrad));
    }
    return SC_OK;
}
int check_tensors(const char* what, int n, const sc_dtype* dtypes, const int64_t* sizes, const void* const* p) {
    if (n > 0 && !p) return fail(SC_ERR_INVALID_ARG, "%s is NULL", what);
    for (int i = 0; i < n; ++i)
        if (sizes[i] > 0) SC_TRY(check_ptr(what, p[i], elem(dtypes[i])));
    return SC_OK;
}

}  // namespace

extern "C" {

int sc_embed(sc_dtype dtype, const void* table, const int64_t* ids, int64_t T, int64_t V, int H, float scale,
             void* out, void* stream) {
    SC_TRY(check_dtype(dtype));
    SC_TRY(check_embed(T, V, H));
    if (T == 0) return SC_OK;
    SC_TRY(check_ptr("table", table, elem(dtype)));
    SC_TRY(check_ptr("ids", ids, 8));
    SC_TRY(check_ptr("out", out, elem(dtype)));
    HIP_TRY(launch_embed(dtype == SC_BF16, table, ids, T, V, H, scale, out, (hipStream_t)stream));
    return SC_OK;
}

int sc_embed_grad_workspace(int64_t T, int64_t V, int H, int64_t* bytes) {
    SC_TRY(check_embed_grad(T, V, H));
    if (!bytes) return fail(SC_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = embed_grad_plan(T, V, H).bytes;
    return SC_OK;
}

int sc_embed_grad(sc_dtype dtype, const void* dy, const int64_t* ids, int64_t T, int64_t V, int H, float scale,
                  void* dW, void* workspace, int64_t workspace_bytes, void* stream) {
    SC_TRY(check_dtype(dtype));
    SC_TRY(check_embed_grad(T, V, H));
    const EmbedGradPlan p = embed_grad_plan(T, V, H);
    if (T > 0) {
        SC_TRY(check_ptr("dy", dy, elem(dtype)));
        SC_TRY(check_ptr("ids", ids, 8));
    }
    SC_TRY(check_ptr("dW", dW, elem(dtype)));
    SC_TRY(check_workspace(workspace, workspace_bytes, p.bytes));
    HIP_TRY(launch_embed_grad(p, dtype == SC_BF16, dy, ids, scale, dW, workspace, (hipStream_t)stream));
    return SC_OK;
}

int sc_act_pack(sc_dtype dtype, const void* x, int64_t T, int H, int8_t* q, uint8_t* e, void* stream) {
    SC_TRY(check_dtype(dtype));
    SC_TRY(check_rows(T, H, kMaxEmbedH));
    if (T == 0) return SC_OK;
    SC_TRY(check_ptr("x", x, elem(dtype)));
    SC_TRY(check_ptr("q", q, 1));
    SC_TRY(check_ptr("e", e, 1));
    HIP_TRY(launch_act_pack(dtype == SC_BF16, x, T, H, q, e, (hipStream_t)stream));
    return SC_OK;
}

int sc_act_unpack(sc_dtype dtype, const int8_t* q, const uint8_t* e, int64_t T, int H, void* x, void* stream) {
    SC_TRY(check_dtype(dtype));
    SC_TRY(check_rows(T, H, kMaxEmbedH));
    if (T == 0) return SC_OK;
    SC_TRY(check_ptr("q", q, 1));
    SC_TRY(check_ptr("e", e, 1));
    SC_TRY(check_ptr("x", x, elem(dtype)));
    HIP_TRY(launch_act_unpack(dtype == SC_BF16, q, e, T, H, x, (hipStream_t)stream));
    return SC_OK;
}

int sc_rmsnorm(sc_dtype dtype, const void* x, const void* residual, const void* gain, float eps, int64_t T, int H,
               void* h, void* y, float* rstd, int8_t* q, uint8_t* e, void* stream) {
    SC_TRY(check_dtype(dtype));
    SC_TRY(check_rows(T, H, kNormMaxH));
    if (!(eps >= 0.0f)) return fail(SC_ERR_INVALID_ARG, "eps must be >= 0");
    if (T == 0) return SC_OK;
    SC_TRY(check_ptr("x", x, elem(dtype)));
    if (residual) SC_TRY(check_ptr("residual", residual, elem(dtype)));
    SC_TRY(check_ptr("gain", gain, elem(dtype)));
    if (h) SC_TRY(check_ptr("h", h, elem(dtype)));
    SC_TRY(check_ptr("y", y, elem(dtype)));
    SC_TRY(check_ptr("rstd", rstd, 4));
    if (!q != !e) return fail(SC_ERR_INVALID_ARG, "q and e go together");
    HIP_TRY(launch_rmsnorm(dtype == SC_BF16, x, residual, gain, eps, T, H, h, y, rstd, q, e, (hipStream_t)stream));
    return SC_OK;
}

int sc_rmsnorm_grad_workspace(int64_t T, int H, int64_t* bytes) {
    SC_TRY(check_rows(T, H, kNormMaxH));
    if (!bytes) return fail(SC_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 4 * rmsnorm_grad_parts(T, H) * H;
    return SC_OK;
}

int sc_rmsnorm_grad(sc_dtype dtype, const void* dy, const void* gain, const float* rstd, const int8_t* q,
                    const uint8_t* e, const void* dh, int64_t T, int H, void* dx, float* dgain, void* workspace,
                    int64_t workspace_bytes, void* stream) {
    SC_TRY(check_dtype(dtype));
    SC_TRY(check_rows(T, H, kNormMaxH));
    SC_TRY(check_ptr("dgain", dgain, 4));
    if (T > 0) {
        SC_TRY(check_ptr("dy", dy, elem(dtype)));
        SC_TRY(check_ptr("gain", gain, elem(dtype)));
        SC_TRY(check_ptr("rstd", rstd, 4));
        SC_TRY(check_ptr("q", q, 1));
        SC_TRY(check_ptr("e", e, 1));
        if (dh) SC_TRY(check_ptr("dh", dh, elem(dtype)));
        SC_TRY(check_ptr("dx", dx, elem(dtype)));
    }
    SC_TRY(check_workspace(workspace, workspace_bytes, 4 * rmsnorm_grad_parts(T, H) * H));
    HIP_TRY(launch_rmsnorm_grad(dtype == SC_BF16, dy, gain, rstd, q, e, dh, T, H, dx, dgain, (float*)workspace,
                                (hipStream_t)stream));
    return SC_OK;
}

int sc_act_wgrad_workspace(sc_dtype dtype, int64_t T, int64_t N, int H, int64_t* bytes) {
    SC_TRY(check_wgrad(dtype, T, N, H));
    if (!bytes) return fail(SC_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = wgrad_plan(dtype == SC_BF16, T, N, H).bytes;
    return SC_OK;
}

int sc_act_wgrad(sc_dtype dtype, const void* dy, const int8_t* q, const uint8_t* e, const void* gain, int64_t T,
                 int64_t N, int H, void* dW, void* workspace, int64_t workspace_bytes, void* stream) {
    SC_TRY(check_wgrad(dtype, T, N, H));
    const WgradPlan p = wgrad_plan(dtype == SC_BF16, T, N, H);
    if (T > 0) {
        SC_TRY(check_ptr("dy", dy, 16));
        SC_TRY(check_ptr("q", q, 1));
        SC_TRY(check_ptr("e", e, 1));
    }
    if (gain) SC_TRY(check_ptr("gain", gain, elem(dtype)));
    SC_TRY(check_ptr("dW", dW, elem(dtype)));
    SC_TRY(check_workspace(workspace, workspace_bytes, p.bytes));
    HIP_TRY(launch_act_wgrad(p, dy, q, e, gain, dW, workspace, (hipStream_t)stream));
    return SC_OK;
}

int sc_xent_workspace(sc_dtype dtype, int64_t T, int64_t V, int H, int64_t limit, int64_t* bytes) {
    SC_TRY(check_xent(dtype, T, V, H, limit));
    if (!bytes) return fail(SC_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = xent_plan(dtype == SC_BF16, T, V, H, limit ? limit : kXentLimit).bytes;
    return SC_OK;
}

int sc_xent(sc_dtype dtype, const void* h, const void* W, const int64_t* targets, int64_t T, int64_t V, int H,
            int64_t limit, float* loss, float* mean, void* dh, void* dW, void* workspace, int64_t workspace_bytes,
            void* stream) {
    SC_TRY(check_xent(dtype, T, V, H, limit));
    const XentPlan p = xent_plan(dtype == SC_BF16, T, V, H, limit ? limit : kXentLimit);
    if (T > 0) {
        SC_TRY(check_ptr("h", h, 16));
        SC_TRY(check_ptr("targets", targets, 8));
        SC_TRY(check_ptr("loss", loss, 4));
        SC_TRY(check_ptr("dh", dh, elem(dtype)));
        SC_TRY(check_ptr("W", W, 16));
    }
    SC_TRY(check_ptr("mean", mean, 4));
    SC_TRY(check_ptr("dW", dW, elem(dtype)));
    SC_TRY(check_workspace(workspace, workspace_bytes, p.bytes));
    HIP_TRY(launch_xent(p, h, W, targets, loss, mean, dh, dW, workspace, (hipStream_t)stream));
    return SC_OK;
}

int sc_token_logp_workspace(sc_dtype dtype, int64_t T, int64_t V, int H, int64_t* bytes) {
    SC_TRY(check_xent(dtype, T, V, H, 0));
    if (!bytes) return fail(SC_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = token_loss_plan(dtype == SC_BF16, T, V, H, 0, false).bytes;
    return SC_OK;
}

int sc_token_logp(sc_dtype dtype, const void* h, const void* W, const int64_t* targets, int64_t T, int64_t V, int H,
                  float* logp, void* workspace, int64_t workspace_bytes, void* stream) {
    SC_TRY(check_xent(dtype, T, V, H, 0));
    const TokenLossPlan p = token_loss_plan(dtype == SC_BF16, T, V, H, 0, false);
    if (T == 0) return SC_OK;
    SC_TRY(check_ptr("h", h, 16));
    SC_TRY(check_ptr("W", W, 16));
    SC_TRY(check_ptr("targets", targets, 8));
    SC_TRY(check_ptr("logp", logp, 4));
    SC_TRY(check_workspace(workspace, workspace_bytes, p.bytes));
    HIP_TRY(launch_token_logp(p, h, W, targets, logp, workspace, (hipStream_t)stream));
    return SC_OK;
}

int sc_token_loss_workspace(sc_dtype dtype, int64_t T, int64_t V, int H, int64_t limit, int64_t* bytes) {
    SC_TRY(check_xent(dtype, T, V, H, limit));
    if (!bytes) return fail(SC_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = token_loss_plan(dtype == SC_BF16, T, V, H, limit ? limit : kXentLimit, true).bytes;
    return SC_OK;
}

int sc_policy_loss(sc_dtype dtype, const void* h, const void* W, const int64_t* targets, const float* old_logp,
                   const float* advantages, const float* ref_logp, const float* weights, int64_t T, int64_t V, int H,
                   float clip_low, float clip_high, float kl, int64_t limit, float* loss, float* total,
                   float* kl_mean, float* clipped, float* logp, void* dh, void* dW, void* workspace,
                   int64_t workspace_bytes, void* stream) {
    SC_TRY(check_xent(dtype, T, V, H, limit));
    if (!(clip_low >= 0.0f && clip_low <= 1.0f)) return fail(SC_ERR_INVALID_ARG, "clip_low must be in [0, 1]");
    if (!(clip_high >= 0.0f)) return fail(SC_ERR_INVALID_ARG, "clip_high must be >= 0");
    if (!(kl >= 0.0f && kl <= 3.402823466e38f)) return fail(SC_ERR_INVALID_ARG, "kl must be finite and >= 0");
    SC_TRY(check_token_loss(dtype, h, W, targets, T, V, H, logp, dh, dW));
    if (T > 0) {
        SC_TRY(check_ptr("old_logp", old_logp, 4));
        SC_TRY(check_ptr("advantages", advantages, 4));
        SC_TRY(check_ptr("loss", loss, 4));
        if (weights) SC_TRY(check_ptr("weights", weights, 4));
        if (ref_logp) SC_TRY(check_ptr("ref_logp", ref_logp, 4));
        if (!ref_logp && (kl > 0.0f || kl_mean)) return fail(SC_ERR_INVALID_ARG, "kl needs ref_logp");
    }
    if (kl_mean) SC_TRY(check_ptr("kl_mean", kl_mean, 4));
    SC_TRY(check_ptr("total", total, 4));
    SC_TRY(check_ptr("clipped", clipped, 4));
    const TokenLossPlan p = token_loss_plan(dtype == SC_BF16, T, V, H, limit ? limit : kXentLimit, true);
    SC_TRY(check_workspace(workspace, workspace_bytes, p.bytes));
    const PolicyArgs a{old_logp, advantages, ref_logp, weights, 1.0 - (double)clip_low, 1.0 + (double)clip_high, kl,
                       loss, total, kl_mean, clipped, logp};
    HIP_TRY(launch_policy_loss(p, h, W, targets, a, dh, dW, workspace, (hipStream_t)stream));
    return SC_OK;
}

int sc_preference_loss(sc_dtype dtype, const void* h, const void* W, const int64_t* targets, const int64_t* starts,
                       const float* ref_logp, int64_t pairs, int64_t T, int64_t V, int H, float beta, float margin,
                       float smoothing, int average, int64_t limit, float* loss, float* mean, float* rewards,
                       float* logp, void* dh, void* dW, void* workspace, int64_t workspace_bytes, void* stream) {
    SC_TRY(check_xent(dtype, T, V, H, limit));
    SC_TRY(check_size("pairs", pairs, 0, kMaxPairs));
    if (!(beta >= 0.0f && beta <= 3.402823466e38f)) return fail(SC_ERR_INVALID_ARG, "beta must be finite and >= 0");
    if (margin != margin) return fail(SC_ERR_INVALID_ARG, "margin is NaN");
    if (!(smoothing >= 0.0f && smoothing <= 1.0f)) return fail(SC_ERR_INVALID_ARG, "smoothing must be in [0, 1]");
    SC_TRY(check_token_loss(dtype, h, W, targets, T, V, H, logp, dh, dW));
    if (ref_logp) SC_TRY(check_ptr("ref_logp", ref_logp, 4));
    if (pairs > 0) {
        SC_TRY(check_ptr("starts", starts, 8));
        SC_TRY(check_ptr("loss", loss, 4));
        SC_TRY(check_ptr("rewards", rewards, 4));
    }
    SC_TRY(check_ptr("mean", mean, 4));
    const TokenLossPlan p = token_loss_plan(dtype == SC_BF16, T, V, H, limit ? limit : kXentLimit, true);
    SC_TRY(check_workspace(workspace, workspace_bytes, p.bytes));
    const PreferenceArgs a{starts, ref_logp, pairs, beta, margin, smoothing, average != 0, loss, mean, rewards, logp};
    HIP_TRY(launch_preference_loss(p, h, W, targets, a, dh, dW, workspace, (hipStream_t)stream));
    return SC_OK;
}

int sc_layernorm(sc_dtype dtype, const void* x, const void* residual, const void* gain, const void* bias, float eps,
                 int64_t T, int H, void* h, void* y, float* mean, float* rstd, int8_t* q, uint8_t* e, void* stream) {
    SC_TRY(check_dtype(dtype));
    SC_TRY(check_rows(T, H, kNormMaxH));
    if (!(eps >= 0.0f)) return fail(SC_ERR_INVALID_ARG, "eps must be >= 0");
    if (T == 0) return SC_OK;
    SC_TRY(check_ptr("x", x, elem(dtype)));
    if (residual) SC_TRY(check_ptr("residual", residual, elem(dtype)));
    SC_TRY(check_ptr("gain", gain, elem(dtype)));
    if (bias) SC_TRY(check_ptr("bias", bias, elem(dtype)));
    if (h) SC_TRY(check_ptr("h", h, elem(dtype)));
    SC_TRY(check_ptr("y", y, elem(dtype)));
    SC_TRY(check_ptr("mean", mean, 4));
    SC_TRY(check_ptr("rstd", rstd, 4));
    if (!q != !e) return fail(SC_ERR_INVALID_ARG, "q and e go together");
    HIP_TRY(launch_layernorm(dtype == SC_BF16, x, residual, gain, bias, eps, T, H, h, y, mean, rstd, q, e,
                             (hipStream_t)stream));
    return SC_OK;
}

int sc_layernorm_grad_workspace(int64_t T, int H, int64_t* bytes) {
    SC_TRY(check_rows(T, H, kNormMaxH));
    if (!bytes) return fail(SC_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 8 * layernorm_grad_parts(T, H) * H;
    return SC_OK;
}

int sc_layernorm_grad(sc_dtype dtype, const void* dy, const void* gain, const float* rstd, const int8_t* q,
                      const uint8_t* e, const void* h, const float* mean, const void* dh, int64_t T, int H, void* dx,
                      float* dgain, float* dbias, void* workspace, int64_t workspace_bytes, void* stream) {
    SC_TRY(check_dtype(dtype));
    SC_TRY(check_rows(T, H, kNormMaxH));
    SC_TRY(check_ptr("dgain", dgain, 4));
    if (dbias) SC_TRY(check_ptr("dbias", dbias, 4));
    if (T > 0) {
        SC_TRY(check_ptr("dy", dy, elem(dtype)));
        SC_TRY(check_ptr("gain", gain, elem(dtype)));
        SC_TRY(check_ptr("rstd", rstd, 4));
        if (!q != !e || !h != !mean || !q == !h)
            return fail(SC_ERR_INVALID_ARG, "either q and e or h and mean are given");
        if (h) {
            SC_TRY(check_ptr("h", h, elem(dtype)));
            SC_TRY(check_ptr("mean", mean, 4));
        }
        if (dh) SC_TRY(check_ptr("dh", dh, elem(dtype)));
        SC_TRY(check_ptr("dx", dx, elem(dtype)));
    }
    SC_TRY(check_workspace(workspace, workspace_bytes, 8 * layernorm_grad_parts(T, H) * H));
    HIP_TRY(launch_layernorm_grad(dtype == SC_BF16, dy, gain, rstd, mean, q, e, h, dh, T, H, dx, dgain, dbias,
                                  (float*)workspace, (hipStream_t)stream));
    return SC_OK;
}

int sc_grad_sumsq_workspace(int n, const sc_dtype* dtypes, const int64_t* sizes, int64_t* bytes) {
    SC_TRY(check_grads(n, dtypes, sizes));
    if (!bytes) return fail(SC_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 8 * grad_sumsq_parts(GradTensors{n, dtypes, sizes, nullptr, nullptr});
    return SC_OK;
}

int sc_grad_sumsq(int n, const sc_dtype* dtypes, const int64_t* sizes, const void* const* grads, double* sumsq,
                  void* workspace, int64_t workspace_bytes, void* stream) {
    SC_TRY(check_grads(n, dtypes, sizes));
    SC_TRY(check_tensors("a gradient", n, dtypes, sizes, grads));
    SC_TRY(check_ptr("sumsq", sumsq, 8));
    const GradTensors g{n, dtypes, sizes, grads, nullptr};
    SC_TRY(check_workspace(workspace, workspace_bytes, 8 * grad_sumsq_parts(g)));
    HIP_TRY(launch_grad_sumsq(g, sumsq, (double*)workspace, (hipStream_t)stream));
    return SC_OK;
}

int sc_clip_grads(int n, const sc_dtype* dtypes, const int64_t* sizes, const void* const* grads, void* const* out,
                  const double* sumsq, float max_norm, float* norm, float* scale, void* stream) {
    SC_TRY(check_grads(n, dtypes, sizes));
    SC_TRY(check_tensors("a gradient", n, dtypes, sizes, grads));
    SC_TRY(check_tensors("an output", n, dtypes, sizes, out));
    if (!(max_norm >= 0.0f)) return fail(SC_ERR_INVALID_ARG, "max_norm must be >= 0");
    SC_TRY(check_ptr("sumsq", sumsq, 8));
    SC_TRY(check_ptr("norm", norm, 4));
    SC_TRY(check_ptr("scale", scale, 4));
    HIP_TRY(launch_clip(GradTensors{n, dtypes, sizes, grads, out}, sumsq, 1, max_norm, norm, scale,
                        (hipStream_t)stream));
    return SC_OK;
}

int sc_clip_norm(int n, const sc_dtype* dtypes, const int64_t* sizes, const void* const* grads, void* const* out,
                 float max_norm, float* norm, float* scale, void* workspace, int64_t workspace_bytes, void* stream) {
    SC_TRY(check_grads(n, dtypes, sizes));
    SC_TRY(check_tensors("a gradient", n, dtypes, sizes, grads));
    SC_TRY(check_tensors("an output", n, dtypes, sizes, out));
    if (!(max_norm >= 0.0f)) return fail(SC_ERR_INVALID_ARG, "max_norm must be >= 0");
    SC_TRY(check_ptr("norm", norm, 4));
    SC_TRY(check_ptr("scale", scale, 4));
    const GradTensors g{n, dtypes, sizes, grads, out};
    SC_TRY(check_workspace(workspace, workspace_bytes, 8 * grad_sumsq_parts(g)));
    HIP_TRY(launch_clip_norm(g, max_norm, norm, scale, (double*)workspace, (hipStream_t)stream));
    return SC_OK;
}

}  // extern "C"
