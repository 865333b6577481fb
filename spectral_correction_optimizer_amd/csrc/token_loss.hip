// Losses of given tokens' log-probabilities over a large vocabulary, with their gradients:
//
//   s[t][v] = h[t] . W[v],  logp[t] = s[t][y_t] - log sum_v exp(s[t][v])
//   policy:  r = exp(logp - old),  L[t] = -min(r A, clip(r, lo, hi) A) + kl k3,
//            k3 = exp(x) - x - 1 with x = ref - logp;  total = sum of w[t] L[t]
//   preference, sequences 2 p (chosen) and 2 p + 1 (rejected) of each pair:  R = beta times the sum (or
//            mean) of logp - ref over the sequence's counted tokens,  z = R[2 p] - R[2 p + 1] - margin,
//            L[p] = -(1 - e) log sigmoid(z) - e log sigmoid(-z);  mean over the pairs
//   either:  d[t][v] = c[t] (exp(logp of v) - [v = y_t]) with c[t] = -(derivative by logp[t]),
//            dh = d W,  dW = d^T h
//
// A token whose target lies outside [0, V) is not counted.  Prompts and padding are most of such a
// batch, so the counted tokens' rows are put together first, on the device (token_rows_kernel), and
// the products run over as many rows as there are (TpArgs::live); the products are cross entropy's.
// What is a token's or a pair's is computed in 64 bits: a KL term is a difference near zero, and a
// sequence's log-probability a long sum.
#include <cmath>

#include "common.hpp"
#include "internal.hpp"
#include "train.hpp"

namespace scopt {

struct Tails {
    TpTailQuery q[3];  // dh, dW, and dW of the last piece
};

// The counted tokens in order: rows[c] = t, place[t] = c (-1 where not counted), their targets; logp and
// loss (or NULL) of the others are 0, and coef starts at 0.  One workgroup, eight tokens a thread
// and turn: a turn's positions are the sums over the threads before.
__global__ __launch_bounds__(1024) void token_rows_kernel(const int64_t* __restrict__ targets, int64_t T, int64_t V,
                                                          int* __restrict__ live, int* __restrict__ rows,
                                                          int* __restrict__ place, int64_t* __restrict__ kept,
                                                          float* __restrict__ coef, float* __restrict__ logp,
                                                          float* __restrict__ loss, const Tails q,
                                                          TpTail* __restrict__ tails) {
    __shared__ int sums[2][16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int base = 0, turn = 0;
    for (int64_t t0 = 0; t0 < T; t0 += 8192, turn ^= 1) {
        const int64_t first = t0 + 8 * threadIdx.x;
        int64_t y[8];
        int n = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = gld(targets + (first + i < T ? first + i : T - 1));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (first + i >= T || y[i] >= V) y[i] = -1;
            n += y[i] >= 0;
        }
        int upto = n;  // of this wavefront's threads up to this one
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int x = __shfl_up(upto, o);
            upto += lane >= o ? x : 0;
        }
        if (lane == 63) sums[turn][wave] = upto;
        __syncthreads();
        int c = base + upto - n;
#pragma unroll
        for (int w = 0; w < 16; ++w) {
            c += w < wave ? sums[turn][w] : 0;
            base += sums[turn][w];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t t = first + i;
            if (t >= T) break;
            if (y[i] >= 0) {
                gst(rows + c, (int)t);
                gst(kept + c, y[i]);
                if (coef) gst(coef + c, 0.0f);
                gst(place + t, c++);
            } else {
                gst(place + t, -1);
                gst(logp + t, 0.0f);
                if (loss) gst(loss + t, 0.0f);
            }
        }
    }
    if (threadIdx.x == 0) gst(live, base);
    if (!tails || wave >= 3) return;
    // how the gradients' products are dealt out: a wavefront a product, a lane a number of parts
    const TpTailQuery& p = q.q[wave];
    const int tiles = p.tiles(base), total = p.total(base), rest = tiles % p.slots;
    int best = p.ns(rest, total, lane + 1), splits = lane + 1;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int ns = __shfl_xor(best, o), s = __shfl_xor(splits, o);
        const bool less = ns < best || (ns == best && s < splits);
        best = less ? ns : best;
        splits = less ? s : splits;
    }
    if (lane == 0) {
        gst(&tails[wave].full, tiles - rest);
        gst(&tails[wave].rest, rest);
        gst(&tails[wave].splits, splits);
    }
}

// The policy's losses and the coefficients of its logit gradients.  One workgroup: sums in a fixed
// order.
__global__ __launch_bounds__(1024) void policy_kernel(const int* __restrict__ live, const int* __restrict__ rows,
                                                      PolicyArgs a, float* __restrict__ coef) {
    __shared__ double red[16];
    const int n = gld(live);
    const double share = n > 0 ? 1.0 / n : 1.0;
    double total = 0.0, kl = 0.0, stopped = 0.0;
#pragma unroll 4
    for (int c = threadIdx.x; c < n; c += 1024) {
        const int64_t t = gld(rows + c);
        const double lp = gld(a.logp + t), A = gld(a.advantages + t);
        const double r = exp(lp - (double)gld(a.old_logp + t));
        const double w = a.weights ? (double)gld(a.weights + t) : share;
        const bool high = A > 0.0 && r > a.hi, low = A < 0.0 && r < a.lo;
        double L = -A * (high ? a.hi : low ? a.lo : r);
        double g = high || low ? 0.0 : A * r;
        if (a.ref_logp) {
            const double x = (double)gld(a.ref_logp + t) - lp, up = expm1(x);
            kl += up - x;
            if (a.kl != 0.0f) {
                L += (double)a.kl * (up - x);
                g += (double)a.kl * up;
            }
        }
        stopped += high || low ? 1.0 : 0.0;
        total += w != 0.0 ? w * L : 0.0;  // a token of weight 0 counts for nothing, finite or not
        gst(a.loss + t, (float)L);
        gst(coef + c, w != 0.0 ? (float)(g * w) : 0.0f);
    }
    total = block_sum_f64(total, red);
    kl = block_sum_f64(kl, red);
    stopped = block_sum_f64(stopped, red);
    if (threadIdx.x == 0) {
        gst(a.total, (float)total);
        if (a.kl_mean) gst(a.kl_mean, (float)(kl * share));
        gst(a.clipped, (float)(stopped * share));
    }
}

// A workgroup a pair: both sequences' sums, the pair's loss, and its tokens' coefficients.
__global__ __launch_bounds__(1024) void preference_kernel(const int* __restrict__ place, int64_t T, PreferenceArgs a,
                                                          float* __restrict__ coef) {
    __shared__ double red[16];
    const int64_t pair = blockIdx.x;
    int64_t at[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int64_t s = gld(a.starts + 2 * pair + i);
        at[i] = s < 0 ? 0 : s < T ? s : T;
    }
    double reward[2], share[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        double sum = 0.0, n = 0.0;
#pragma unroll 4
        for (int64_t t = at[k] + threadIdx.x; t < at[k + 1]; t += 1024) {
            const bool counted = gld(place + t) >= 0;
            const double x = (double)gld(a.logp + t) - (a.ref_logp ? (double)gld(a.ref_logp + t) : 0.0);
            sum += counted ? x : 0.0;
            n += counted ? 1.0 : 0.0;
        }
        sum = block_sum_f64(sum, red);
        n = block_sum_f64(n, red);
        share[k] = a.average && n > 0.0 ? 1.0 / n : 1.0;
        reward[k] = (double)a.beta * sum * share[k];
    }
    const double e = a.smoothing, z = reward[0] - reward[1] - (double)a.margin;
    const double tail = exp(-fabs(z)), soft = log1p(tail);  // log(1 + exp(-|z|))
    const double win = (z > 0.0 ? 1.0 : tail) / (1.0 + tail), lose = (z > 0.0 ? tail : 1.0) / (1.0 + tail);
    // -log sigmoid(z) = max(-z, 0) + soft; a weight of 0 leaves the other term alone
    const double L = (e < 1.0 ? (1.0 - e) * (fmax(-z, 0.0) + soft) : 0.0) + (e > 0.0 ? e * (fmax(z, 0.0) + soft) : 0.0);
    const double g = (double)a.beta / (double)a.pairs * ((1.0 - e) * lose - e * win);
    if (threadIdx.x == 0) {
        gst(a.loss + pair, (float)(z == z ? L : z));
        if (a.pairs == 1) gst(a.mean, (float)(z == z ? L : z));
        gst(a.rewards + 2 * pair, (float)reward[0]);
        gst(a.rewards + 2 * pair + 1, (float)reward[1]);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float c = (float)((k ? -g : g) * share[k]);
        for (int64_t t = at[k] + threadIdx.x; t < at[k + 1]; t += 1024) {
            const int r = gld(place + t);
            if (r >= 0) gst(coef + r, c);
        }
    }
}

__global__ __launch_bounds__(1024) void pair_mean_kernel(const float* __restrict__ loss, int64_t pairs,
                                                         float* __restrict__ mean) {
    __shared__ double red[16];
    double s = 0.0;
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < pairs; i += 1024) s += (double)gld(loss + i);
    s = block_sum_f64(s, red);
    if (threadIdx.x == 0) gst(mean, pairs > 0 ? (float)(s / (double)pairs) : 0.0f);
}

TokenLossPlan token_loss_plan(bool bf16, int64_t T, int64_t V, int64_t H, int64_t limit, bool gradients) {
    TokenLossPlan p{};
    p.x = xent_plan(bf16, T, V, H, limit, gradients, true);
    p.gradients = gradients;
    int64_t o = p.x.bytes;
    auto take = [&](int64_t bytes) {
        const int64_t at = o;
        o += (bytes + 255) / 256 * 256;
        return at;
    };
    p.o_live = take(4);
    p.o_rows = take(4 * T);
    p.o_place = take(4 * T);
    p.o_targets = take(8 * T);
    p.o_coef = take(4 * T);
    p.bytes = o;
    return p;
}

#define SC_RUN(expr)                          \
    do {                                      \
        const hipError_t e_ = (expr);         \
        if (e_ != hipSuccess) return e_;      \
    } while (0)

namespace {
// The counted tokens' rows, the operands, and every token's log-probability
hipError_t forward(const TokenLossPlan& p, XentRun& run, const void* h, const void* W, const int64_t* targets,
                   float* logp, float* loss, void* dh, void* workspace, hipStream_t st) {
    run.p = &p.x;
    run.h = h;
    run.W = W;
    run.ws = (char*)workspace;
    run.st = st;
    int *live = run.at<int>(p.o_live), *rows = run.at<int>(p.o_rows), *place = run.at<int>(p.o_place);
    int64_t* kept = run.at<int64_t>(p.o_targets);
    float* coef = run.at<float>(p.o_coef);
    run.targets = kept;
    run.live = live;
    run.rows = rows;
    run.place = place;
    run.coef = coef;
    const Tails tails = {{p.x.dh.tail, p.x.dw.tail, p.x.dw_last.tail}};
    hipLaunchKernelGGL(token_rows_kernel, dim3(1), dim3(1024), 0, st, targets, p.x.T, p.x.V, live, rows, place, kept,
                       coef, logp, loss, tails, p.gradients ? run.at<TpTail>(p.x.o_tails) : nullptr);
    SC_RUN(hipGetLastError());
    SC_RUN(run.operands(dh));
    SC_RUN(run.logits());
    return run.log_sums(nullptr, logp);
}
}  // namespace

hipError_t launch_token_logp(const TokenLossPlan& p, const void* h, const void* W, const int64_t* targets,
                             float* logp, void* workspace, hipStream_t st) {
    if (p.x.T == 0) return hipSuccess;
    XentRun run;
    return forward(p, run, h, W, targets, logp, nullptr, nullptr, workspace, st);
}

hipError_t launch_policy_loss(const TokenLossPlan& p, const void* h, const void* W, const int64_t* targets,
                              const PolicyArgs& a, void* dh, void* dW, void* workspace, hipStream_t st) {
    if (p.x.T == 0) {
        SC_RUN(launch_zero(a.total, 4, st));
        if (a.kl_mean) SC_RUN(launch_zero(a.kl_mean, 4, st));
        SC_RUN(launch_zero(a.clipped, 4, st));
        return launch_zero(dW, p.x.V * p.x.H * (p.x.bf16 ? 2 : 4), st);
    }
    XentRun run;
    SC_RUN(forward(p, run, h, W, targets, a.logp, a.loss, dh, workspace, st));
    hipLaunchKernelGGL(policy_kernel, dim3(1), dim3(1024), 0, st, run.live, run.rows, a, run.at<float>(p.o_coef));
    SC_RUN(hipGetLastError());
    return run.gradients(dh, dW);
}

hipError_t launch_preference_loss(const TokenLossPlan& p, const void* h, const void* W, const int64_t* targets,
                                  const PreferenceArgs& a, void* dh, void* dW, void* workspace, hipStream_t st) {
    XentRun run;
    if (p.x.T > 0) SC_RUN(forward(p, run, h, W, targets, a.logp, nullptr, dh, workspace, st));
    if (a.pairs > 0) {
        hipLaunchKernelGGL(preference_kernel, dim3((unsigned)a.pairs), dim3(1024), 0, st, run.place, p.x.T, a,
                           (float*)((char*)workspace + p.o_coef));
        SC_RUN(hipGetLastError());
    }
    if (a.pairs != 1) {
        hipLaunchKernelGGL(pair_mean_kernel, dim3(1), dim3(1024), 0, st, a.loss, a.pairs, a.mean);
        SC_RUN(hipGetLastError());
    }
    if (p.x.T == 0) return launch_zero(dW, p.x.V * p.x.H * (p.x.bf16 ? 2 : 4), st);
    return run.gradients(dh, dW);
}
#undef SC_RUN

}  // namespace scopt
