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

}  // extern "C"
