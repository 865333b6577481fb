// Softmax cross entropy over a large vocabulary with its gradients, the logits held in pieces:
//
//   s[t][v] = h[t] . W[v],  lse[t] = log sum_v exp(s[t][v]),  loss[t] = lse[t] - s[t][y_t]
//   mean = sum of loss over the counted t / count
//   d[t][v] = (exp(s[t][v] - lse[t]) - [v = y_t]) / count   (0 where t is not counted)
//   dh = d W,  dW = d^T h
//
// A token whose target lies outside [0, V) is not counted: loss 0, no gradient.
//
// The products run on the matrix cores (tile_product.hpp); they are the cost at large T
// (3 products of 2 T V H operations), reading W and writing dW at small T.  The vocabulary
// goes by in pieces:
//   - If one piece (the whole vocabulary) fits the limit, a T x V matrix is kept: the logits product
//     leaves exponentials relative to each tile's row maximum (16 bits; float32 operands: the
//     logits in float32, beside d's planes 10 bytes an entry), xent_dlogits_kernel turns them into d
//     once every row's sum is known, and the two gradient products read d: three products.
//   - Otherwise no matrix of logits exists: a first pass over the pieces takes only the row sums, and
//     a second one recomputes each piece's logits straight into d: four products, and memory for one
//     piece only.
// 8192 tokens, 131072 x 2048 in bfloat16, kept: logits 3.9 ms (1130 TFLOP/s), d 0.85 ms (5.1 TB/s), dh
// 3.3 ms (1330), dW 3.7 ms (1190), the call 11.7 to 11.9 ms.  In pieces of 1 GiB or 256 MiB 15.0 ms, of 64 MiB
// 16.4 ms (the gradients' sums over the pieces); 32768 tokens, in pieces by default, 59 ms.  Float32, 4096
// tokens, 50021 x 1024: kept 7.2 ms, in pieces of 256 MiB 8.9 ms.
// Of the factor 1 / count, d takes the power of two next below, which is exact: its products with the
// largest states then stay within float32's range as their mean does (0.4% of the call's time); the
// gradients' stores apply the rest.  The matrix cores take d in bfloat16, half a step of its own
// value off (2^-8): two planes would double the gradient products.  An exponential kept between
// the passes adds 2^-10 (tp_pack_unit; 0.4% of the call's time).  Errors of dW against 64 bits at 64
// tokens, 32000 x 2048, relative to its norm: 0.0019 in the rows of targets, 0.0024 in the others,
// where exponentials kept in bfloat16 made it 0.0029; the rounding of dW alone is 0.0017.  The
// target's entry is formed from the float32 logit, as there the subtraction cancels.  In float32 d is
// split exactly into three planes.
// The losses of given tokens (token_loss.hip) share all this: their rows are the counted tokens, and each has a factor
// of its own, which in bfloat16 goes onto its row of dh and its row of h before dW (one rounding more; rows of dW
// against 64 bits 0.0024 of their norm off where a target is met once, dh 0.0017, the rounding of the outputs
// alone 0.0017), so that what is kept can be relative to any power of two of the row (XentPlan::by_row): where that
// is known before the logits, no pass turns exponentials into d.  The factor also undoes the rounding of the target's
// entry, the largest, and moves the row's other entries together by that much, 2^-8 of themselves at most.
#include <cmath>

#include "log_sums.hpp"
#include "tile_product.hpp"

namespace scopt {

namespace {
constexpr int64_t kAlign = 256;
int64_t up(int64_t n, int64_t a) { return (n + a - 1) / a * a; }
}  // namespace

__global__ __launch_bounds__(1024) void xent_lse_kernel(const LogSums a, const int64_t* __restrict__ targets, int64_t V,
                                                        float* __restrict__ loss) {
    __shared__ float red[16][64];
    log_sums<64>(a, a.T, (int64_t)blockIdx.x * 64, red, [&](int64_t t, float logp) {
        gst(loss + t, tp_target(targets, V, t) >= 0 ? -logp : 0.0f);
    });
}
// of counted tokens: 16 rows a workgroup, as 64 threads take a row's tiles
__global__ __launch_bounds__(1024) void token_lse_kernel(const LogSums a, const int* __restrict__ live,
                                                         const int* __restrict__ rows, float* __restrict__ logp) {
    __shared__ float red[16][16];
    const int64_t end = gld(live);
    if ((int64_t)blockIdx.x * 16 >= end) return;
    log_sums<16>(a, end, (int64_t)blockIdx.x * 16, red, [&](int64_t t, float lp) { gst(logp + gld(rows + t), lp); });
}

// The power of two that a token's exponentials are kept relative to (XentPlan::by_row): its target's, whose logit is
// formed here for that alone, so that none is smaller there than its probability is.  A wavefront a row.
__global__ __launch_bounds__(256) void row_reference_kernel(const int* __restrict__ live,
                                                            const uint16_t* __restrict__ h, int64_t ldh,
                                                            const uint16_t* __restrict__ W, int64_t ldw,
                                                            const int64_t* __restrict__ targets, int H,
                                                            float* __restrict__ ref) {
    const int64_t t = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
    if (t >= gld(live)) return;
    const uint16_t *a = h + t * ldh, *b = W + gld(targets + t) * ldw;
    float s = 0.0f;
#pragma unroll 4
    for (int i = 8 * (threadIdx.x & 63); i < H; i += 512) {
        const v4u x = *(const SC_GLOBAL v4u*)(a + i), y = *(const SC_GLOBAL v4u*)(b + i);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            s = fmaf(bf16_lo(x[k]), bf16_lo(y[k]), s);
            s = fmaf(bf16_hi(x[k]), bf16_hi(y[k]), s);
        }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
    // (none for a logit past 2^16, whose last bits are the order of its sum)
    if ((threadIdx.x & 63) == 0)
        gst(ref + t, fabsf(s) < 0x1p16f ? ceilf(s * kLog2e) : __builtin_nanf(""));
}
// Whether all of a row's tiles are kept relative to its reference: no tile's own is above the next power of two
// of the row's sum by more than one.
__device__ __forceinline__ bool kept_by_row(float lse, float row_ref) {
    return tp_by_row(fmaf(lse, kLog2e, 3.0f), row_ref);
}
// softmax - onehot at a token's target, as the logit gradients of live tokens hold it
__device__ __forceinline__ float target_entry(float target_logit, float lse) {
    return __builtin_amdgcn_exp2f((target_logit - lse) * kLog2e) - 1.0f;
}
// 256 threads: row t's factor, coef times what bfloat16's rounding took from the target's entry, and its H states
// times that.  A coefficient of 0 gives zeros, whatever the states are.  d's row is softmax - onehot times 2^up;
// returns its target's entry.
__device__ __forceinline__ float scale_row(int64_t t, float coef, float up, const float* target_logit, const float* lse,
                                           float* factor, const uint16_t* from, uint16_t* to, int64_t H) {
    const float q = target_entry(gld(target_logit + t), gld(lse + t)), unit = __builtin_amdgcn_exp2f(up);
    const float r = bf16_to_f32(f32_to_bf16(q * unit));
    const float c = coef != 0.0f && r != 0.0f ? coef * (q / r) : coef / unit;
    if (threadIdx.x == 0) gst(factor + t, c);
    for (int64_t i = 8 * threadIdx.x; i < H; i += 8 * 256) {
        const v4u w = *(const SC_GLOBAL v4u*)(from + t * H + i);
        v4u o;
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = coef != 0.0f ? pack_bf16x2(bf16_lo(w[k]) * c, bf16_hi(w[k]) * c) : 0u;
        *(SC_GLOBAL v4u*)(to + t * H + i) = o;
    }
    return r;
}
// and of float32 operands, whose coefficients are in d: row t of h's three planes becomes one of zeros where coef is 0
__device__ __forceinline__ void clear_row(int64_t t, float coef, uint16_t* h, int64_t plane, int64_t H) {
    if (coef != 0.0f) return;
    for (int64_t i = 8 * threadIdx.x; i < H; i += 8 * 256)
#pragma unroll
        for (int k = 0; k < 3; ++k) *(SC_GLOBAL v4u*)(h + k * plane + t * H + i) = v4u{0, 0, 0, 0};
}
__global__ __launch_bounds__(256) void clear_rows_kernel(const int* __restrict__ live, const float* __restrict__ coef,
                                                         uint16_t* h, int64_t plane, int64_t H) {
    const int64_t t = blockIdx.x;
    if (t < gld(live)) clear_row(t, gld(coef + t), h, plane, H);
}
__global__ __launch_bounds__(256) void scale_rows_kernel(const int* __restrict__ live, const float* __restrict__ coef,
                                                         const float* __restrict__ target_logit,
                                                         const float* __restrict__ lse, float* __restrict__ factor,
                                                         const uint16_t* __restrict__ from, uint16_t* __restrict__ to,
                                                         int64_t H) {
    const int64_t t = blockIdx.x;
    if (t < gld(live)) (void)scale_row(t, gld(coef + t), 0.0f, target_logit, lse, factor, from, to, H);
}

// d from what the logits product kept: exponentials in 16 bits (in place) or float32 logits
// (into three planes).  `chunks` workgroups a row; a thread takes 8 columns at a time.  With coef the row's first
// workgroup also sees to its row of h (EXP: scaled, and d has only coef's zeros).  A row that was kept relative to
// row_ref is softmax - onehot already, but for its target's entry and a factor, which joins coef: where the
// reference is ref, 2^ref / exp(lse).  (8192 tokens, half of them counted, x 131072: 425 us for all rows anew.)
template <bool EXP>
__global__ __launch_bounds__(256) void xent_dlogits_kernel(const float* __restrict__ logits, uint16_t* P,
                                                           int64_t plane, int64_t ldp, int N, int bn,
                                                           int64_t chunk, int chunks,
                                                           const float* __restrict__ smax, int64_t T,
                                                           const float* __restrict__ lse,
                                                           const float* __restrict__ target_logit,
                                                           const int64_t* __restrict__ targets, int64_t V,
                                                           const float* __restrict__ scale_at,
                                                           const int* __restrict__ live,
                                                           const float* __restrict__ coef, float* factor, uint16_t* h,
                                                           int64_t Hh, const float* __restrict__ row_ref) {
    const int64_t t = blockIdx.x / chunks;
    if (live && t >= gld(live)) return;
    float scale = gld(coef ? coef + t : scale_at);
    const float to_row = EXP && row_ref ? gld(row_ref + t) : 0.0f;
    const bool done = EXP && row_ref && kept_by_row(gld(lse + t), to_row);
    if (coef) {
        if (blockIdx.x % chunks == 0) {
            if constexpr (EXP) {
                const float up = done ? fmaf(gld(lse + t), kLog2e, -to_row) : 0.0f;
                const float r = scale_row(t, scale, up, target_logit, lse, factor, h, h, Hh);
                if (done && threadIdx.x == 0) gst(P + t * ldp + gld(targets + t), f32_to_bf16(r));
            } else {
                clear_row(t, scale, h, T * Hh, Hh);
            }
        }
        if (done) return;
        if constexpr (EXP) scale = scale != 0.0f ? 1.0f : 0.0f;
    }
    // a row without weight is one of zeros, whatever its logits are
    const int64_t tgt = scale != 0.0f ? tp_target(targets, V, t) : -1;
    const float ls = gld(lse + t);
    const float ls2 = ls * kLog2e;
    float at_target = 0.0f;
    if (tgt >= 0) at_target = EXP && coef ? target_entry(gld(target_logit + t), ls) :
                                            (expf(gld(target_logit + t) - ls) - 1.0f) * scale;
    const int64_t end = (N + 7) & ~7;  // the products read no further
    const int64_t from = (int64_t)(blockIdx.x % chunks) * chunk, to = from + chunk < end ? from + chunk : end;
    for (int64_t c = from + 8 * threadIdx.x; c < to; c += 8 * 256) {
        uint16_t* p = P + t * ldp + c;
        float v[8];
        if constexpr (EXP) {
            const v4u w = *(const SC_GLOBAL v4u*)p;
            const float ref = gld(smax + (int64_t)(c / bn) * T + t);
            const bool by_row = row_ref && tp_by_row(ref, to_row);
            // (a row's own reference may be below the smallest number where the tile's, 2^64 above it, is not)
            const float x = (by_row ? to_row : ref) - ls2;
            const bool below = by_row && x < -64.0f;
            const float f = __builtin_amdgcn_exp2f(below ? x + 64.0f : x) * scale, low = below ? 0x1p-64f : 1.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = (by_row ? bf16_lo(w[i]) : tp_unit_lo(w[i])) * f * low;
                v[2 * i + 1] = (by_row ? bf16_hi(w[i]) : tp_unit_hi(w[i])) * f * low;
            }
        } else {
            const v4f a = gld4(logits + t * ldp + c), b = gld4(logits + t * ldp + c + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = expf(a[i] - ls) * scale;
                v[4 + i] = expf(b[i] - ls) * scale;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (c + i == tgt) v[i] = at_target;
            if (tgt < 0 || c + i >= N) v[i] = 0.0f;
        }
        const float lo[4] = {v[0], v[1], v[2], v[3]}, hi[4] = {v[4], v[5], v[6], v[7]};
        if constexpr (EXP) {
            *(SC_GLOBAL v4u*)p = v4u{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                     pack_bf16x2(v[6], v[7])};
        } else {
            tp_store_planes(P, 3, plane, t * ldp + c, lo);
            tp_store_planes(P, 3, plane, t * ldp + c + 4, hi);
        }
    }
}

// the mean loss over the counted tokens, summed in a fixed order, and one token's share of it as the
// factor of the gradients' stores (at least 1, below 2) and d's, a power of two
__global__ __launch_bounds__(1024) void xent_mean_kernel(const float* __restrict__ loss,
                                                         const int64_t* __restrict__ targets, int64_t T, int64_t V,
                                                         float* factors, float* mean) {
    __shared__ double red[16];
    double s = 0.0, n = 0.0;
#pragma unroll 4
    for (int64_t t = threadIdx.x; t < T; t += 1024) {
        s += (double)gld(loss + t);
        n += tp_target(targets, V, t) >= 0 ? 1.0 : 0.0;
    }
    s = block_sum_f64(s, red);
    n = block_sum_f64(n, red);
    if (threadIdx.x == 0) {
        n = n > 0.0 ? n : 1.0;
        double scale = 1.0;
        while (scale * n > 1.0) scale *= 0.5;
        gst(factors, (float)(1.0 / (n * scale)));
        gst(factors + 1, (float)scale);
        gst(mean, (float)(s / n));
    }
}

XentPlan xent_plan(bool bf16, int64_t T, int64_t V, int64_t H, int64_t limit, bool gradients,
                   bool live) {
    XentPlan p{};
    p.bf16 = bf16;
    p.T = T;
    p.V = V;
    p.H = H;
    p.planes = !bf16 || H % 8 != 0;
    p.Hp = p.planes ? tp_pad(up(H, 64)) : H;
    p.Hh = tp_pad(up(H, 64));
    const int nseg = bf16 ? 1 : 6;
    p.half = live && !bf16;
    const int logit_seg = p.half ? 3 : nseg;
    // bytes of a vocabulary column: the kept exponentials, or the logits and d's planes
    const int64_t col_kept = T * (bf16 ? 2 : 10), col_piece = T * (bf16 ? 2 : 6);
    p.keep = gradients && up(V, 256) * col_kept <= limit;
    p.piece = V;
    if (gradients && !p.keep) {
        p.piece = limit / col_piece / 256 * 256;
        if (p.piece < 256) p.piece = 256;
        if (p.piece > V) p.piece = V;
    }
    p.pieces = (int)((V + p.piece - 1) / p.piece);
    p.ldp = tp_pad(up(p.piece, 256));  // the logits' tiles are stored whole
    const int64_t last = V - (int64_t)(p.pieces - 1) * p.piece;
    auto logits = [&](int64_t cols, TpTailQuery& tail) {
        return live ? tp_plan_live(TPK_LOGIT_STATS_LIVE, (int)T, (int)cols, (int)H, logit_seg, tail)
                    : tp_plan((int)T, (int)cols, (int)H, nseg, false);
    };
    p.logits = logits(p.piece, p.tails[3]);
    p.logits_last = logits(last, p.tails[4]);
    if (gradients) {
        const bool join = p.pieces > 1;  // sums over pieces have splits of their own
        p.dh = live && !join ? tp_plan_live(TPK_STATES_LIVE, (int)T, (int)H, (int)p.piece, nseg, p.tails[0])
                             : tp_plan((int)T, (int)H, (int)p.piece, nseg, true);
        auto weights = [&](int64_t rows, TpTailQuery& tail) {
            return live ? tp_plan_live(TPK_WEIGHTS_LIVE, (int)rows, (int)H, (int)T, nseg, tail)
                        : tp_plan((int)rows, (int)H, (int)T, nseg, true);
        };
        p.dw = weights(p.piece, p.tails[1]);
        p.dw_last = weights(last, p.tails[2]);
    }
    p.stat_tiles = (int64_t)(p.pieces - 1) * p.logits.tiles_n + p.logits_last.tiles_n;
    int64_t o = 0;
    auto take = [&](int64_t bytes) {
        const int64_t at = o;
        o += up(bytes, kAlign);
        return at;
    };
    const int np = bf16 ? 1 : 3;
    p.o_factors = take(8);
    const bool whole = gradients || !p.half;  // the gradients' operands, or the logits' too
    p.o_h = whole ? take(2 * np * T * p.Hh) : 0;
    p.o_scaled = live && gradients && bf16 && !p.keep ? take(2 * T * p.Hh) : p.o_h;
    p.o_w = p.planes && whole ? take(2 * np * V * p.Hp) : 0;
    if (p.half) {
        p.o_half_h = take(4 * T * p.Hh);
        p.o_half_w = take(4 * V * p.Hp);
        p.o_exp_h = take(4 * T);
        p.o_exp_w = take(4 * up(V, 256));  // (the last tile's columns are read whole)
    }
    p.o_s = !bf16 && p.keep ? take(4 * T * p.ldp) : 0;
    p.o_p = gradients ? take(2 * np * T * p.ldp) : 0;
    p.o_tl = take(4 * T);
    p.o_lse = take(4 * T);
    p.o_smax = take(4 * T * p.stat_tiles);
    p.o_ssum = take(4 * T * p.stat_tiles);
    const bool join = gradients && p.pieces > 1;
    int64_t part = p.dh.part_bytes;
    if (join && part == 0) part = 4 * T * H;
    for (const TpPlan* q : {&p.dw, &p.dw_last, &p.logits, &p.logits_last}) part = part > q->part_bytes ? part : q->part_bytes;
    p.o_part = take(part);
    p.o_dh = join ? take(4 * T * H) : 0;
    if (live) p.o_tails = take(5 * sizeof(TpTail));
    if (live && gradients) p.o_factor = take(4 * T);
    p.by_row = live && bf16 && p.keep && T * V >= 1 << 24;
    if (p.by_row) p.o_ref = take(4 * T);
    p.bytes = o;
    return p;
}

#define SC_RUN(expr)                          \
    do {                                      \
        const hipError_t e_ = (expr);         \
        if (e_ != hipSuccess) return e_;      \
    } while (0)

hipError_t XentRun::h_operand(void* dh) const {
    if (p->half)
        return launch_half_rows((const float*)h, p->T, p->H, p->Hh, at<uint16_t>(p->o_half_h), at<int>(p->o_exp_h),
                                gradients_follow ? at<uint16_t>(p->o_h) : nullptr, st, place, (float*)dh);
    // h is always copied, without the tokens that are not counted or with zeros for them: whatever
    // they hold (a NaN too) reaches no product
    return launch_to_planes(p->bf16, h, p->T, p->H, at<uint16_t>(p->o_h), p->Hh, p->T * p->Hh,
                            rows ? nullptr : targets, p->V, st, place, dh);
}
hipError_t XentRun::w_planes() const {
    if (!p->planes) return hipSuccess;
    if (p->half)
        return launch_half_rows((const float*)W, p->V, p->H, p->Hp, at<uint16_t>(p->o_half_w), at<int>(p->o_exp_w),
                                gradients_follow ? at<uint16_t>(p->o_w) : nullptr, st);
    return launch_to_planes(p->bf16, W, p->V, p->H, at<uint16_t>(p->o_w), p->Hp, p->V * p->Hp, nullptr, 0, st);
}

hipError_t XentRun::row_references() const {
    if (!p->by_row) return hipSuccess;
    hipLaunchKernelGGL(row_reference_kernel, dim3((unsigned)((p->T + 3) / 4)), dim3(256), 0, st, live,
                       at<uint16_t>(p->o_h), p->Hh, w_operand(), p->Hp, targets, (int)up(p->H, 8), at<float>(p->o_ref));
    return hipGetLastError();
}

// planes (A | B << 2) of the six products of two split operands, smallest first
uint64_t XentRun::segments() const { return p->bf16 ? 0 : 0x0 << 20 | 0x4 << 16 | 0x1 << 12 | 0x8 << 8 | 0x5 << 4 | 0x2; }

TpArgs XentRun::logit_args(int i) const {
    TpArgs a;
    const int64_t v0 = (int64_t)i * p->piece;
    a.A = at<uint16_t>(p->o_h);
    a.lda = p->Hh;
    a.a_plane = p->T * p->Hh;
    a.B = w_operand() + v0 * p->Hp;
    a.ldb = p->Hp;
    a.b_plane = p->V * p->Hp;
    a.M = (int)p->T;
    a.N = (int)(p->V - v0 < p->piece ? p->V - v0 : p->piece);
    a.K = (int)up(p->H, 8);
    a.nseg = p->bf16 ? 1 : 6;
    a.segs = segments();
    a.targets = targets;
    a.vocab = p->V;
    a.n_first = v0;
    a.ldp = p->ldp;
    a.p_plane = p->T * p->ldp;
    a.p_planes = p->bf16 ? 1 : 3;
    a.target_logit = at<float>(p->o_tl);
    a.stat_max = at<float>(p->o_smax);
    a.stat_sum = at<float>(p->o_ssum);
    a.stat_first = (int64_t)i * p->logits.tiles_n;
    a.lse = at<float>(p->o_lse);
    a.live = live;
    if (p->by_row) a.row_ref = at<float>(p->o_ref);
    if (p->half) {
        a.A = at<uint16_t>(p->o_half_h);
        a.B = at<uint16_t>(p->o_half_w) + v0 * p->Hp;
        a.nseg = 3;
        a.segs = 0x0 << 8 | 0x4 << 4 | 0x1;  // the products with a second plane, then the largest
        a.a_exp = at<int>(p->o_exp_h);
        a.b_exp = at<int>(p->o_exp_w) + v0;
    }
    return a;
}

hipError_t XentRun::logits() const {
    for (int i = 0; i < p->pieces; ++i) {
        TpArgs a = logit_args(i);
        a.keep = !p->keep ? TP_KEEP_NONE : p->bf16 ? TP_KEEP_EXP : TP_KEEP_LOGIT;
        a.P = p->bf16 ? at<void>(p->o_p) : at<void>(p->o_s);
        a.part = at<float>(p->o_part);
        const bool last = i + 1 == p->pieces;
        a.tail = at<TpTail>(p->o_tails) + (last ? 4 : 3);
        SC_RUN(launch_tile_product(live ? TPK_LOGIT_STATS_LIVE : TPK_LOGIT_STATS, last ? p->logits_last : p->logits, a,
                                   TpSum{}, st));
    }
    return hipSuccess;
}

LogSums XentRun::sums() const {
    return LogSums{at<float>(p->o_smax), at<float>(p->o_ssum), (int)p->stat_tiles, p->keep && p->bf16,
                   at<float>(p->o_tl),   at<float>(p->o_lse),  p->T};
}

hipError_t XentRun::log_sums(float* loss, float* logp) const {
    if (rows)
        hipLaunchKernelGGL(token_lse_kernel, dim3((unsigned)((p->T + 15) / 16)), dim3(1024), 0, st, sums(), live, rows,
                           logp);
    else
        hipLaunchKernelGGL(xent_lse_kernel, dim3((unsigned)((p->T + 63) / 64)), dim3(1024), 0, st, sums(), targets, p->V,
                           loss);
    return hipGetLastError();
}

hipError_t XentRun::gradients(void* dh, void* dW) const {
    const int64_t T = p->T, V = p->V, H = p->H;
    const float* factors = at<float>(p->o_factors);
    uint16_t* P = at<uint16_t>(p->o_p);
    float *part = at<float>(p->o_part), *dhs = at<float>(p->o_dh);
    const int nseg = p->bf16 ? 1 : 6;
    if (coef && p->o_scaled != p->o_h) {
        hipLaunchKernelGGL(scale_rows_kernel, dim3((unsigned)T), dim3(256), 0, st, live, coef, at<float>(p->o_tl),
                           at<float>(p->o_lse), at<float>(p->o_factor), at<uint16_t>(p->o_h),
                           at<uint16_t>(p->o_scaled), p->Hh);
        SC_RUN(hipGetLastError());
    } else if (coef && !p->bf16 && !p->keep) {
        hipLaunchKernelGGL(clear_rows_kernel, dim3((unsigned)T), dim3(256), 0, st, live, coef, at<uint16_t>(p->o_h),
                           T * p->Hh, p->Hh);
        SC_RUN(hipGetLastError());
    }
    for (int i = 0; i < p->pieces; ++i) {
        const int64_t v0 = (int64_t)i * p->piece;
        const int n = (int)(V - v0 < p->piece ? V - v0 : p->piece);
        if (p->keep) {
            // enough workgroups for the chip, at least 2048 columns each
            const int64_t chunk = up((n * T + 4095) / 4096, 2048);
            const int chunks = (int)((n + chunk - 1) / chunk);
            const dim3 grid((unsigned)(chunks * T));
            auto kernel = p->bf16 ? xent_dlogits_kernel<true> : xent_dlogits_kernel<false>;
            hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, p->bf16 ? nullptr : at<float>(p->o_s), P, T * p->ldp,
                               p->ldp, n, p->logits.bn, chunk, chunks, at<float>(p->o_smax), T, at<float>(p->o_lse),
                               at<float>(p->o_tl), targets, V, factors + 1, live, coef,
                               at<float>(p->o_factor), at<uint16_t>(p->o_h), p->Hh,
                               p->by_row ? at<float>(p->o_ref) : nullptr);
            SC_RUN(hipGetLastError());
        } else {
            TpArgs a = logit_args(i);
            a.P = P;
            a.alpha = factors + 1;
            a.coef = coef;
            a.coef_zeros = coef && p->bf16;
            SC_RUN(launch_tile_product(TPK_LOGIT_GRAD, i + 1 < p->pieces ? p->logits : p->logits_last, a, TpSum{}, st));
        }
        TpArgs a;  // dh (+)= d W: k runs over the piece
        a.A = P;
        a.lda = p->ldp;
        a.a_plane = T * p->ldp;
        a.B = w_operand() + v0 * p->Hp;
        a.ldb = p->Hp;
        a.b_plane = V * p->Hp;
        a.M = (int)T;
        a.N = (int)H;
        a.K = n;
        a.nseg = nseg;
        a.segs = segments();
        a.C = dh;
        a.ldc = H;
        a.c_bf16 = p->bf16;
        a.alpha = coef ? nullptr : factors;
        a.coef = coef && p->bf16 ? at<float>(p->o_factor) : nullptr;
        a.tail = at<TpTail>(p->o_tails);
        a.part = part;
        a.live = live;
        a.rows = rows;
        TpSum sum;
        if (p->pieces > 1) {
            sum.acc = i > 0 ? dhs : nullptr;
            sum.out_acc = i + 1 < p->pieces ? dhs : nullptr;
        }
        SC_RUN(launch_tile_product(live && p->pieces == 1 ? TPK_STATES_LIVE : TPK_STATES, p->dh, a, sum, st));
        if (live && p->bf16 && T <= kFewTokens) {
            SC_RUN(launch_few_tokens(P, p->ldp, at<uint16_t>(p->o_scaled), p->Hh, (int)T, live, n, (int)H,
                                     (uint16_t*)dW + v0 * H, st));
            continue;
        }
        TpArgs b;  // dW = d^T h: k runs over the tokens
        b.A = P;
        b.lda = p->ldp;
        b.a_plane = T * p->ldp;
        b.B = at<uint16_t>(p->o_scaled);
        b.ldb = p->Hh;
        b.b_plane = T * p->Hh;
        b.M = n;
        b.N = (int)H;
        b.K = (int)T;
        b.nseg = nseg;
        b.segs = segments();
        b.C = (char*)dW + v0 * H * (p->bf16 ? 2 : 4);
        b.ldc = H;
        b.c_bf16 = p->bf16;
        b.alpha = coef ? nullptr : factors;
        b.part = part;
        b.live = live;
        b.tail = at<TpTail>(p->o_tails) + (i + 1 < p->pieces ? 1 : 2);
        SC_RUN(launch_tile_product(live ? TPK_WEIGHTS_LIVE : TPK_WEIGHTS, i + 1 < p->pieces ? p->dw : p->dw_last, b,
                                   TpSum{}, st));
    }
    return hipSuccess;
}

hipError_t launch_xent(const XentPlan& p, const void* h, const void* W, const int64_t* targets, float* loss,
                       float* mean, void* dh, void* dW, void* workspace, hipStream_t st) {
    if (p.T == 0) {
        SC_RUN(launch_zero(mean, 4, st));
        return launch_zero(dW, p.V * p.H * (p.bf16 ? 2 : 4), st);
    }
    XentRun run;
    run.p = &p;
    run.h = h;
    run.W = W;
    run.targets = targets;
    run.ws = (char*)workspace;
    run.st = st;
    SC_RUN(run.h_operand(nullptr));
    SC_RUN(run.w_planes());
    SC_RUN(run.logits());
    SC_RUN(run.log_sums(loss, nullptr));
    hipLaunchKernelGGL(xent_mean_kernel, dim3(1), dim3(1024), 0, st, loss, targets, p.T, p.V,
                       run.at<float>(p.o_factors), mean);
    SC_RUN(hipGetLastError());
    return run.gradients(dh, dW);
}
#undef SC_RUN

}  // namespace scopt
