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
// The three products bound both losses at many tokens, reading W and writing dW at few.  Policy of 8192 tokens,
// 4096 of them counted, 131072 x 2048 in bfloat16: logits 2.01 ms (1090 TFLOP/s), dh 1.64 (1340), dW 1.83 (1200),
// all else 0.09, the call 5.51 to 5.65; of 1000 tokens, 700 counted, 50021 x 1001 in float32 1.27 to 1.29 ms: logits
// 0.26 ms in three float16 products, dh 0.41 and dW 0.43 in six, planes 0.14 and the gradients of the logits 0.08.
// Preference of a pair of 96 tokens, 32000 x 2048: logits 45 us (2.9 TB/s; 34 where no exponentials are kept behind a
// write of as much), dh 28 and dW 30 (4.4 TB/s), five small launches 30.  (Tiles are chosen by T: 60 counted tokens of
// 1000 take 182 us, alone 134.)
#include <cmath>

#include "common.hpp"
#include "internal.hpp"
#include "planes.hpp"
#include "train.hpp"

namespace scopt {

struct Tails {
    TpTailQuery q[5];  // XentPlan::tails
};
// What the counted tokens' rows are told in: rows[c] = t, place[t] = c (-1 where not counted), their targets; logp and
// loss (or NULL) of the others are 0, and coef starts at 0.
struct Rows {
    const int64_t* targets;
    int64_t T, V;
    int *live, *rows, *place;
    int64_t* kept;
    float *coef, *logp, *loss;
    TpTail* tails;
    Tails q;
};

// The next eight tokens' targets, -1 where not counted; returns how many are
__device__ __forceinline__ int targets_of(const Rows& a, int64_t first, int64_t (&y)[8]) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = gld(a.targets + (first + i < a.T ? first + i : a.T - 1));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (first + i >= a.T || y[i] >= a.V) y[i] = -1;
        n += y[i] >= 0;
    }
    return n;
}
__device__ __forceinline__ void tell_rows(const Rows& a, int64_t first, const int64_t (&y)[8], int c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t t = first + i;
        if (t >= a.T) break;
        if (y[i] >= 0) {
            gst(a.rows + c, (int)t);
            gst(a.kept + c, y[i]);
            gst(a.coef + c, 0.0f);
            gst(a.place + t, c++);
        } else {
            gst(a.place + t, -1);
            gst(a.logp + t, 0.0f);
            if (a.loss) gst(a.loss + t, 0.0f);
        }
    }
}
// How the products are dealt out: a wavefront takes one after the other, a lane a number of parts.
__device__ __forceinline__ void tell_tails(const Rows& a, int live) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (threadIdx.x == 0) gst(a.live, live);
    for (int i = wave; i < 5; i += blockDim.x / 64) {
        const TpTailQuery& p = a.q.q[i];
        const int tiles = p.tiles(live), total = p.total(live), rest = tiles % p.slots;
        int best = p.ns(tiles, total, lane + 1), splits = lane + 1;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int ns = __shfl_xor(best, o), s = __shfl_xor(splits, o);
            const bool less = ns < best || (ns == best && s < splits);
            best = less ? ns : best;
            splits = less ? s : splits;
        }
        if (lane == 0) {
            gst(&a.tails[i].full, tiles - rest);
            gst(&a.tails[i].rest, rest);
            gst(&a.tails[i].splits, splits);
        }
    }
}
// This wavefront's sum of n up to each lane
__device__ __forceinline__ int wave_scan(int n) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int x = __shfl_up(n, o);
        n += lane >= o ? x : 0;
    }
    return n;
}

// One workgroup, eight tokens a thread and turn: a turn's positions are the sums over the threads before.
__global__ __launch_bounds__(1024) void token_rows_kernel(const Rows a) {
    __shared__ int sums[2][16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int base = 0, turn = 0;
    for (int64_t t0 = 0; t0 < a.T; t0 += 8192, turn ^= 1) {
        const int64_t first = t0 + 8 * threadIdx.x;
        int64_t y[8];
        const int n = targets_of(a, first, y), upto = wave_scan(n);
        if (lane == 63) sums[turn][wave] = upto;
        __syncthreads();
        int c = base + upto - n;
#pragma unroll
        for (int w = 0; w < 16; ++w) {
            c += w < wave ? sums[turn][w] : 0;
            base += sums[turn][w];
        }
        tell_rows(a, first, y, c);
    }
    tell_tails(a, base);
}

// The same and h's bfloat16 operand in one launch, for up to kFewRows tokens: every workgroup finds all positions by
// itself.  (64 tokens x 2048: 6.5 us, the two kernels 3.7 and 4.4; 8192 tokens, half of them counted: 26 us, 18
// and 17 as two.)
constexpr int64_t kFewRows = 8192;
template <typename E, int ENDS>
__global__ __launch_bounds__(256) void few_rows_kernel(const Rows a, const E* __restrict__ h, int H,
                                                       uint16_t* __restrict__ dst, int64_t ld, int64_t plane,
                                                       E* __restrict__ cleared) {
    __shared__ int sums[2][4];
    __shared__ int16_t place[kFewRows];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int base = 0, turn = 0;
    for (int64_t t0 = 0; t0 < a.T; t0 += 2048, turn ^= 1) {
        const int64_t first = t0 + 8 * threadIdx.x;
        int64_t y[8];
        const int n = targets_of(a, first, y), upto = wave_scan(n);
        if (lane == 63) sums[turn][wave] = upto;
        __syncthreads();
        int c = base + upto - n;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            c += w < wave ? sums[turn][w] : 0;
            base += sums[turn][w];
        }
        int at = c;
#pragma unroll
        for (int i = 0; i < 8; ++i) place[first + i] = (int16_t)(y[i] >= 0 ? at++ : -1);
        if (blockIdx.x == (unsigned)(t0 / 2048) % gridDim.x) tell_rows(a, first, y, c);
    }
    if (blockIdx.x == 0) tell_tails(a, base);
    __syncthreads();
    planes_of_rows<E, ENDS>(
        h, a.T, H, dst, ld, plane, cleared, [&](int64_t r) { return (int64_t)place[r]; }, [](int64_t) { return true; });
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
    __shared__ double red[4][16];
    const int64_t pair = blockIdx.x;
    int64_t at[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int64_t s = gld(a.starts + 2 * pair + i);
        at[i] = s < 0 ? 0 : s < T ? s : T;
    }
    double v[4] = {0.0, 0.0, 0.0, 0.0};  // sums and counts
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll 4
        for (int64_t t = at[k] + threadIdx.x; t < at[k + 1]; t += 1024) {
            const bool counted = gld(place + t) >= 0;
            const double x = (double)gld(a.logp + t) - (a.ref_logp ? (double)gld(a.ref_logp + t) : 0.0);
            v[k] += counted ? x : 0.0;
            v[2 + k] += counted ? 1.0 : 0.0;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) v[i] += __shfl_xor(v[i], o);
        if ((threadIdx.x & 63) == 0) red[i][threadIdx.x >> 6] = v[i];
    }
    __syncthreads();
    double reward[2], share[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        double sum = 0.0, n = 0.0;
#pragma unroll
        for (int w = 0; w < 16; ++w) {
            sum += red[k][w];
            n += red[2 + k][w];
        }
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
hipError_t forward(const TokenLossPlan& p, XentRun& run, bool gradients, const void* h, const void* W,
                   const int64_t* targets, float* logp, float* loss, void* dh, void* workspace, hipStream_t st) {
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
    const Rows r{targets, p.x.T, p.x.V, live, rows, place, kept, coef, logp, loss,
                 run.at<TpTail>(p.x.o_tails),
                 {{p.x.tails[0], p.x.tails[1], p.x.tails[2], p.x.tails[3], p.x.tails[4]}}};
    run.gradients_follow = gradients;
    if (p.x.T <= kFewRows && !p.x.half) {
        const int64_t groups = p.x.T * (p.x.Hh / 8);
        const int64_t blocks = (groups + 256 * kGroups - 1) / (256 * kGroups);
        const dim3 grid((unsigned)(blocks < 1024 ? blocks : 1024));
        auto few = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, r, (const uint16_t*)h, (int)p.x.H,
                               run.at<uint16_t>(p.x.o_h), p.x.Hh, p.x.T * p.x.Hh, (uint16_t*)dh);
        };
        switch (row_ends(p.x.H)) {
            case ROW_WHOLE: few(few_rows_kernel<uint16_t, ROW_WHOLE>); break;
            case ROW_CUT: few(few_rows_kernel<uint16_t, ROW_CUT>); break;
            case ROW_SHORT: few(few_rows_kernel<uint16_t, ROW_SHORT>); break;
        }
        SC_RUN(hipGetLastError());
    } else {
        hipLaunchKernelGGL(token_rows_kernel, dim3(1), dim3(1024), 0, st, r);
        SC_RUN(hipGetLastError());
        SC_RUN(run.h_operand(dh));
    }
    SC_RUN(run.w_planes());
    SC_RUN(run.row_references());
    SC_RUN(run.logits());
    return run.log_sums(nullptr, logp);
}
}  // namespace

hipError_t launch_token_logp(const TokenLossPlan& p, const void* h, const void* W, const int64_t* targets,
                             float* logp, void* workspace, hipStream_t st) {
    if (p.x.T == 0) return hipSuccess;
    XentRun run;
    return forward(p, run, false, h, W, targets, logp, nullptr, nullptr, workspace, st);
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
    SC_RUN(forward(p, run, true, h, W, targets, a.logp, a.loss, dh, workspace, st));
    hipLaunchKernelGGL(policy_kernel, dim3(1), dim3(1024), 0, st, run.live, run.rows, a, run.at<float>(p.o_coef));
    SC_RUN(hipGetLastError());
    return run.gradients(dh, dW);
}

hipError_t launch_preference_loss(const TokenLossPlan& p, const void* h, const void* W, const int64_t* targets,
                                  const PreferenceArgs& a, void* dh, void* dW, void* workspace, hipStream_t st) {
    XentRun run;
    if (p.x.T > 0) SC_RUN(forward(p, run, true, h, W, targets, a.logp, nullptr, dh, workspace, st));
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
