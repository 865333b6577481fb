// The tiled products of the training-step operators: instances of the kernel of
// tile_product.hpp, the choice of tile and split, the sum over splits, and the copies of
// operands into bfloat16 planes.
#include "planes.hpp"
#include "rows.hpp"
#include "tile_product.hpp"

namespace scopt {

namespace {
constexpr int kCus = 256;
using Big = TpShape<256, 256, 2, 4, 2, 1>;   // 128 KB of LDS: one workgroup of 8 waves per CU
using Mid = TpShape<128, 128, 2, 2, 2, 2>;   // 64 KB: two workgroups of 4 waves per CU
using Small = TpShape<64, 128, 1, 4, 3, 2>;  // 72 KB: two workgroups of 4 waves per CU
// Logits of few tokens: one row of tiles, deep buffers, and every tile its own order of k
using Few64 = TpShape<64, 128, 1, 4, 4, 1, true>;    // 96 KB: a workgroup of 4 waves per CU
using Few128 = TpShape<128, 128, 2, 2, 3, 1, true>;  // 96 KB: likewise
}  // namespace

// a column's factor
__device__ __forceinline__ float tp_gain(const TpArgs& P, int n) {
    if (!P.gain) return 1.0f;
    return P.gain_bf16 ? Elem<uint16_t>::load((const uint16_t*)P.gain, n) : gld((const float*)P.gain + n);
}

// Sum of the splits' partial products, in split order, with the store's factors.
// acc: an earlier sum that is added (NULL: none); out_acc: the sum is kept there in float32
// instead of being stored.
__global__ __launch_bounds__(256) void tp_reduce_kernel(const TpArgs P, const float* acc, float* out_acc) {
    const int M = P.live_rows ? min(P.M, gld(P.live)) : P.M;
    const int64_t groups = (int64_t)M * ((P.N + 3) / 4);
    const float alpha = P.alpha ? gld(P.alpha) : 1.0f;
    for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < groups; g += (int64_t)gridDim.x * 256) {
        const int64_t m = g / ((P.N + 3) / 4);
        const int n = (int)(g - m * ((P.N + 3) / 4)) * 4;
        const int left = P.N - n;
        const int64_t at = m * P.N + n, stride = (int64_t)M * P.N;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (left >= 4) {
            if (acc) {
                const v4f_any x = *(const SC_GLOBAL v4f_any*)(acc + at);
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] = x[r];
            }
#pragma unroll 8
            for (int s = 0; s < P.splits; ++s) {
                const v4f_any x = *(const SC_GLOBAL v4f_any*)(P.part + s * stride + at);
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] += x[r];
            }
        } else {
            for (int r = 0; r < left; ++r) {
                float sum = acc ? gld(acc + at + r) : 0.0f;
                for (int s = 0; s < P.splits; ++s) sum += gld(P.part + s * stride + at + r);
                v[r] = sum;
            }
        }
        if (out_acc) {
            tp_store(out_acc, 0, at, v, left);
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] *= alpha * tp_gain(P, min(n + r, P.N - 1));
            if (P.coef) {
                const float f = gld(P.coef + m);
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] *= f;
            }
            tp_store(P.C, P.c_bf16, tp_row(P, (int)m) * P.ldc + n, v, left);
        }
    }
}

// Sum of the parts of TP_TAIL's cut tiles, in order, with its stores: four columns a thread.
template <int BM, int BN>
__global__ __launch_bounds__(256) void tp_tail_kernel(const TpArgs P) {
    const TpTail t = {gld(&P.tail->full), gld(&P.tail->rest), gld(&P.tail->splits)};
    if (t.splits == 1) return;
    const int M = P.live_rows ? min(P.M, gld(P.live)) : P.M, tiles_m = (M + BM - 1) / BM;
    constexpr int GROUPS = BM * BN / 4;
    const int64_t stride = (int64_t)t.rest * BM * BN;
    for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < (int64_t)t.rest * GROUPS;
         g += (int64_t)gridDim.x * 256) {
        const int tile = (int)(g / GROUPS), in = (int)(g % GROUPS) * 4;
        int tm, tn;
        tp_tile(t.full + tile, tiles_m, P.tiles_n, tm, tn);
        const int m = tm * BM + in / BN, n = tn * BN + in % BN;
        if (m >= M || n >= P.N) continue;
        const float* p = P.part + (int64_t)tile * BM * BN + in;
        v4f x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
        for (int s = 0; s < t.splits; ++s) x += gld4(p + s * stride);
        const float f = P.coef ? gld(P.coef + m) : 1.0f;
        const float v[4] = {x[0] * f, x[1] * f, x[2] * f, x[3] * f};
        tp_store(P.C, P.c_bf16, tp_row(P, m) * P.ldc + n, v, P.N - n);
    }
}

// TP_STATS of the parts' sums: a wavefront a row of a tile, BN / 64 columns a lane.
template <int BM, int BN>
__global__ __launch_bounds__(256) void tp_stats_tail_kernel(const TpArgs P) {
    constexpr int C = BN / 64;
    static_assert(C == 2 || C == 4, "columns of a lane");
    const TpTail t = {gld(&P.tail->full), gld(&P.tail->rest), gld(&P.tail->splits)};
    if (t.splits == 1) return;
    const int M = min(P.M, gld(P.live)), tiles_m = (M + BM - 1) / BM;
    const int lane = threadIdx.x & 63;
    const int64_t stride = (int64_t)t.rest * BM * BN;
    const bool pow2 = P.keep == TP_KEEP_EXP;
    for (int row = blockIdx.x * 4 + threadIdx.x / 64; row < t.rest * BM; row += gridDim.x * 4) {
        const int tile = row / BM;
        int tm, tn;
        tp_tile(t.full + tile, tiles_m, P.tiles_n, tm, tn);
        const int m = tm * BM + row % BM, n = tn * BN + lane * C;
        if (m >= M) continue;
        const float* p = P.part + (int64_t)row * BN + lane * C;
        float v[C];
#pragma unroll
        for (int c = 0; c < C; ++c) v[c] = 0.0f;
#pragma unroll 4
        for (int s = 0; s < t.splits; ++s) {
            typedef float vec __attribute__((ext_vector_type(C)));
            const vec x = *(const SC_GLOBAL vec*)(p + s * stride);
#pragma unroll
            for (int c = 0; c < C; ++c) v[c] += x[c];
        }
        if (P.a_exp) {
            const int e = gld(P.a_exp + m);
#pragma unroll
            for (int c = 0; c < C; ++c) v[c] = ldexpf(v[c], e + gld(P.b_exp + min(n + c, P.N - 1)));
        }
        float mx = -__builtin_huge_valf();
#pragma unroll
        for (int c = 0; c < C; ++c) mx = fmaxf(mx, v[c]);
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
        const float ref = tp_reference(mx, pow2);
        const int64_t hit = gld(P.targets + m) - P.n_first - n;
        float e[C], z = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            e[c] = pow2 ? __builtin_amdgcn_exp2f(fmaf(v[c], kLog2e, -ref))
                        : __builtin_amdgcn_exp2f((v[c] - ref) * kLog2e);
            z += e[c];
            if (hit == c && n + c < P.N) gst(P.target_logit + m, v[c]);
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) z += __shfl_xor(z, o);
        if (pow2) {
            uint32_t* to = (uint32_t*)((uint16_t*)P.P + (int64_t)m * P.ldp + n);
            const float row_ref = P.row_ref ? gld(P.row_ref + m) : 0.0f;
            const bool by_row = P.row_ref && tp_by_row(ref, row_ref);
            const float unit = __builtin_amdgcn_exp2f(ref - row_ref);
#pragma unroll
            for (int c = 0; c < C; c += 2)
                gst(to + c / 2, by_row ? pack_bf16x2(e[c] * unit, e[c + 1] * unit) : tp_pack_unit(e[c], e[c + 1]));
        } else if (P.keep == TP_KEEP_LOGIT) {
            float* to = (float*)P.P + (int64_t)m * P.ldp + n;
#pragma unroll
            for (int c = 0; c < C; ++c) gst(to + c, v[c]);
        }
        if (lane == 0) {
            const int64_t at = (int64_t)(P.stat_first + tn) * P.M + m;
            gst(P.stat_max + at, mx == -__builtin_huge_valf() ? mx : ref);
            gst(P.stat_sum + at, z);
        }
    }
}

// Choice of tile and split: the least estimated time.  A workgroup's 64-deep step takes
// `step` us with the chip full and a tile `tile` us beside its steps (its first reads, its
// stores); steps come in whole turns of `turn` buffers for every segment.  Fitted to bf16
// products with both operands' rows contiguous, N x H from T tokens; us of the three shapes:
//   8192 x 2048, T 16384:  436, 614, 829    8192 x 8192, T 2048: 317, 336, 429
//   16384 x 4096, T 512:   101, 106, 119    32768 x 2048, T 64:   54,  49,  63
// The same figures choose for the logits (k contiguous, row statistics behind every tile) and for the
// segments of float32 products, which were not fitted.
// A split's partial sums are written and read once more, at about 5 TB/s, by another kernel.
namespace {
struct ShapeTimes {
    int bm, bn, per_cu, turn;
    double step, tile;
};
constexpr ShapeTimes kShapes[5] = {
    {256, 256, 1, 2, 1.70, 12.0}, {128, 128, 2, 2, 1.20, 3.7}, {64, 128, 2, 3, 0.81, 1.2},
    {64, 128, 1, 4, 0.5, 1.2},    {128, 128, 1, 3, 0.8, 3.7}};  // the last two not fitted
}  // namespace

TpPlan tp_plan(int M, int N, int K, int nseg, bool may_split) {
    TpPlan best;
    double best_us = 1e300;
    for (int s = 0; s < 3; ++s) {
        const ShapeTimes& S = kShapes[s];
        const int64_t tm = (M + S.bm - 1) / S.bm, tn = (N + S.bn - 1) / S.bn;
        const int64_t turns = (int64_t)((K + 64 * S.turn - 1) / (64 * S.turn)) * nseg;
        for (int sp = 1; sp <= (may_split ? 64 : 1); sp *= 2) {
            if (sp > 1 && turns / sp < 2) break;
            const int64_t wgs = tm * tn * sp, slots = kCus * S.per_cu;
            const int64_t rounds = (wgs + slots - 1) / slots;
            double us = (double)rounds * ((double)((turns + sp - 1) / sp * S.turn) * S.step + S.tile);
            if (sp > 1) us += 4.0 + 8.0 * sp * (double)M * N / 5e6;
            if (us < best_us) {
                best_us = us;
                best.shape = s;
                best.bm = S.bm;
                best.bn = S.bn;
                best.tiles_m = (int)tm;
                best.tiles_n = (int)tn;
                best.splits = sp;
                best.part_bytes = sp > 1 ? 4ll * sp * M * N : 0;
            }
        }
    }
    return best;
}

// The least time for the most tokens there can be; with fewer of them the last round is cut anew on the device.
TpPlan tp_plan_live(TpKind kind, int M, int N, int K, int nseg, TpTailQuery& tail) {
    const bool live_k = kind == TPK_WEIGHTS_LIVE, logits = kind == TPK_LOGIT_STATS_LIVE;
    const int rounds = logits ? 1 : 2;
    TpPlan best;
    double best_us = 1e300;
    // Few tokens and enough columns for the weights to be read at memory's rate.  (32000 x 2048 that is not in
    // cache: log-probabilities of 64 tokens 42.8 us, with the small tiles 48.5; the loss of a pair of 96 tokens 135
    // and 143.  The order of k makes the difference, not the depth of the buffers: small tiles with it take 42.7.)
    const bool few = logits && M <= 128 && N >= 128 * 128;
    for (int s = few ? (M <= 64 ? 3 : 4) : 0; s < (few ? (M <= 64 ? 4 : 5) : 3); ++s) {
        const ShapeTimes& S = kShapes[s];
        const int slots = kCus * S.per_cu;
        TpTailQuery q;
        q.M = M;
        q.K = K;
        q.live_k = live_k;
        q.bm = S.bm;
        q.turn_k = 64 * S.turn;
        q.tiles_n = (N + S.bn - 1) / S.bn;
        q.nseg = nseg;
        q.slots = slots;
        q.turn_ns = (int)(1000.0 * S.step * S.turn);
        q.tile_ns = (int)(1000.0 * S.tile);
        q.join_ns = 8 * S.bm * S.bn / 5000;  // a tile's partial sums written and read once more, at about 5 TB/s
        const int live = live_k ? K : M, tiles = q.tiles(live), total = q.total(live);
        // what the tokens do not change goes by at about 5 TB/s (the logits of 64 tokens, 32000 x 2048: whole 25 us,
        // cut in two and joined 35)
        const int64_t bytes = live_k ? (int64_t)M * N * (nseg > 1 ? 4 : 2)
                                     : (int64_t)N * K * (nseg == 6 ? 6 : nseg == 3 ? 4 : 2);
        q.pass_ns = (int)(bytes / 5000 < 1 << 30 ? bytes / 5000 : 1 << 30);
        // parts of any number of live tokens, none of fewer than two turns
        const int64_t parts = total < 4 ? 0 : (int64_t)tiles * (total / 2 < 64 ? total / 2 : 64);
        q.most = few ? 0 : (int)(parts < rounds * slots ? parts : rounds * slots);
        int ns = 0x7fffffff;
        for (int p = 1; p <= 64; ++p) ns = q.ns(tiles, total, p) < ns ? q.ns(tiles, total, p) : ns;
        const double us = (double)(tiles / slots) * ((double)total * S.step * S.turn + S.tile) + 1e-3 * ns;
        if (us < best_us) {
            best_us = us;
            best.shape = s;
            best.bm = S.bm;
            best.bn = S.bn;
            best.tiles_m = (M + S.bm - 1) / S.bm;
            best.tiles_n = q.tiles_n;
            best.part_bytes = 4ll * S.bm * S.bn * q.most;
            tail = q;
        }
    }
    return best;
}

namespace {
template <class S>
hipError_t launch_few(const TpPlan& plan, const TpArgs& P, hipStream_t st) {
    auto kernel = P.a_exp ? tile_product_kernel<S, true, true, TP_STATS_TAIL, true>
                          : tile_product_kernel<S, true, true, TP_STATS_TAIL, false>;
    hipLaunchKernelGGL(kernel, dim3(kCus * S::PER_CU), dim3(S::NT), 0, st, P);
    if (plan.part_bytes > 0)
        hipLaunchKernelGGL((tp_stats_tail_kernel<S::BM, S::BN>), dim3(2048), dim3(256), 0, st, P);
    return hipGetLastError();
}
template <class S>
hipError_t launch_tail(TpKind kind, const TpPlan& plan, const TpArgs& P, hipStream_t st) {
    const dim3 grid(kCus * S::PER_CU), blk(S::NT);
    if (kind == TPK_LOGIT_STATS_LIVE && P.a_exp)
        hipLaunchKernelGGL((tile_product_kernel<S, true, true, TP_STATS_TAIL, true>), grid, blk, 0, st, P);
    else if (kind == TPK_LOGIT_STATS_LIVE)
        hipLaunchKernelGGL((tile_product_kernel<S, true, true, TP_STATS_TAIL>), grid, blk, 0, st, P);
    else if (kind == TPK_STATES_LIVE)
        hipLaunchKernelGGL((tile_product_kernel<S, true, false, TP_TAIL>), grid, blk, 0, st, P);
    else
        hipLaunchKernelGGL((tile_product_kernel<S, false, false, TP_TAIL>), grid, blk, 0, st, P);
    if (plan.part_bytes > 0) {
        auto join = kind == TPK_LOGIT_STATS_LIVE ? tp_stats_tail_kernel<S::BM, S::BN> : tp_tail_kernel<S::BM, S::BN>;
        hipLaunchKernelGGL(join, dim3(2048), dim3(256), 0, st, P);
    }
    return hipGetLastError();
}
template <class S>
hipError_t launch_shape(TpKind kind, const TpArgs& P, bool part, hipStream_t st) {
    const int all = P.tiles_m * P.tiles_n * P.splits, most = kCus * S::PER_CU;
    const dim3 grid((unsigned)(all < most ? all : most)), blk(S::NT);
    switch (kind) {
        case TPK_LOGIT_STATS:
            hipLaunchKernelGGL((tile_product_kernel<S, true, true, TP_STATS>), grid, blk, 0, st, P);
            break;
        case TPK_LOGIT_GRAD:
            if (P.a_exp) hipLaunchKernelGGL((tile_product_kernel<S, true, true, TP_GRAD, true>), grid, blk, 0, st, P);
            else hipLaunchKernelGGL((tile_product_kernel<S, true, true, TP_GRAD>), grid, blk, 0, st, P);
            break;
        case TPK_STATES:
            if (part) hipLaunchKernelGGL((tile_product_kernel<S, true, false, TP_PART>), grid, blk, 0, st, P);
            else hipLaunchKernelGGL((tile_product_kernel<S, true, false, TP_STORE>), grid, blk, 0, st, P);
            break;
        case TPK_WEIGHTS:
            if (part) hipLaunchKernelGGL((tile_product_kernel<S, false, false, TP_PART>), grid, blk, 0, st, P);
            else hipLaunchKernelGGL((tile_product_kernel<S, false, false, TP_STORE>), grid, blk, 0, st, P);
            break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}
}  // namespace

hipError_t launch_tp_reduce(const TpArgs& P, const float* acc, float* out_acc, hipStream_t st) {
    const int64_t groups = (int64_t)P.M * ((P.N + 3) / 4);
    const int64_t blocks = (groups + 255) / 256;
    hipLaunchKernelGGL(tp_reduce_kernel, dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, st, P, acc,
                       out_acc);
    return hipGetLastError();
}

hipError_t launch_tile_product(TpKind kind, const TpPlan& plan, TpArgs P, const TpSum& sum, hipStream_t st) {
    P.tiles_m = plan.tiles_m;
    P.tiles_n = plan.tiles_n;
    P.splits = plan.splits;
    P.live_rows = P.live && (kind == TPK_STATES || kind == TPK_STATES_LIVE);
    if (kind == TPK_LOGIT_STATS_LIVE && plan.shape >= 3)
        return plan.shape == 3 ? launch_few<Few64>(plan, P, st) : launch_few<Few128>(plan, P, st);
    if (kind >= TPK_LOGIT_STATS_LIVE)
        return plan.bm == 256   ? launch_tail<Big>(kind, plan, P, st)
               : plan.bm == 128 ? launch_tail<Mid>(kind, plan, P, st)
                                : launch_tail<Small>(kind, plan, P, st);
    const bool part = (kind == TPK_STATES || kind == TPK_WEIGHTS) && (plan.splits > 1 || sum.acc || sum.out_acc);
    hipError_t e = plan.bm == 256   ? launch_shape<Big>(kind, P, part, st)
                   : plan.bm == 128 ? launch_shape<Mid>(kind, P, part, st)
                                    : launch_shape<Small>(kind, P, part, st);
    if (e != hipSuccess || !part) return e;
    return launch_tp_reduce(P, sum.acc, sum.out_acc, st);
}

// zeros, by a kernel: the calls may be captured into a graph
__global__ __launch_bounds__(256) void zero_kernel(uint16_t* p, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        gst(p + i, (uint16_t)0);
}
hipError_t launch_zero(void* p, int64_t bytes, hipStream_t st) {
    const int64_t blocks = (bytes / 2 + 255) / 256;
    if (blocks > 0)
        hipLaunchKernelGGL(zero_kernel, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, st,
                           (uint16_t*)p, bytes / 2);
    return hipGetLastError();
}

// place: where each row goes, or NULL
template <typename E, int ENDS>
__global__ __launch_bounds__(256) void to_planes_kernel(const E* __restrict__ src, int64_t rows, int cols,
                                                        uint16_t* __restrict__ dst, int64_t ld, int64_t plane,
                                                        const int64_t* __restrict__ targets, int64_t vocab,
                                                        const int* __restrict__ place, E* __restrict__ cleared) {
    planes_of_rows<E, ENDS>(
        src, rows, cols, dst, ld, plane, cleared,
        [&](int64_t r) { return place ? gld(place + r) : r; },
        [&](int64_t r) {
            const int64_t t = targets ? gld(targets + r) : 0;
            return t >= 0 && t < vocab;
        });
}

// A wavefront a row; up to 2048 columns stay in registers between its largest magnitude and its planes.
template <int ENDS, bool PLANES>
__global__ __launch_bounds__(256) void half_rows_kernel(const float* __restrict__ src, int64_t rows, int cols, int64_t ld,
                                                        uint16_t* __restrict__ half, int* __restrict__ exps,
                                                        uint16_t* __restrict__ planes, const int* __restrict__ place,
                                                        float* __restrict__ cleared) {
    constexpr int C = 4;
    const int lane = threadIdx.x & 63;
    const int64_t plane = rows * ld;
    for (int64_t r = (int64_t)blockIdx.x * 4 + threadIdx.x / 64; r < rows; r += (int64_t)gridDim.x * 4) {
        const float* from = src + r * cols;
        Group8<float, ENDS> w[C], more[C];
#pragma unroll
        for (int j = 0; j < C; ++j) w[j].load(from, (j * 64 + lane) * 8, cols);
        const int64_t to = place ? gld(place + r) : r;
        if (to < 0) {
            const float none[8] = {};
            if (cleared)
                for (int c = lane * 8; c < cols; c += 512) store8(cleared + r * cols + c, cols - c, none);
            continue;
        }
        float most = 0.0f;
        auto take = [&](const Group8<float, ENDS>& g, int c) __attribute__((always_inline)) {
            float f[8];
            value8(g, c, cols, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float a = fabsf(f[i]);
                most = fmaxf(most, a < __builtin_huge_valf() ? a : 0.0f);
            }
        };
#pragma unroll
        for (int j = 0; j < C; ++j) take(w[j], (j * 64 + lane) * 8);
        for (int c0 = C * 512; c0 < cols; c0 += C * 512) {
#pragma unroll
            for (int j = 0; j < C; ++j) more[j].load(from, c0 + (j * 64 + lane) * 8, cols);
#pragma unroll
            for (int j = 0; j < C; ++j) take(more[j], c0 + (j * 64 + lane) * 8);
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor(most, o));
        const int e = half_exponent(most);
        if (lane == 0) gst(exps + to, -e);
        auto put = [&](const Group8<float, ENDS>& g, int c) __attribute__((always_inline)) {
            if (c >= ld) return;
            float f[8];
            value8(g, c, cols, f);
            v8h h, l;
            split8_half(f, e, h, l);
            uint16_t* o = half + to * ld + c;
            *(SC_GLOBAL v8h*)o = h;
            *(SC_GLOBAL v8h*)(o + plane) = l;
            if constexpr (PLANES) {
                const Split8 s = split8_any(f);
                uint16_t* p = planes + to * ld + c;
                *(SC_GLOBAL v8bf*)p = s.h;
                *(SC_GLOBAL v8bf*)(p + plane) = s.m;
                *(SC_GLOBAL v8bf*)(p + 2 * plane) = s.l;
            }
        };
#pragma unroll
        for (int j = 0; j < C; ++j) put(w[j], (j * 64 + lane) * 8);
        for (int c0 = C * 512; c0 < ld; c0 += C * 512) {
#pragma unroll
            for (int j = 0; j < C; ++j) more[j].load(from, c0 + (j * 64 + lane) * 8, cols);
#pragma unroll
            for (int j = 0; j < C; ++j) put(more[j], c0 + (j * 64 + lane) * 8);
        }
    }
}

hipError_t launch_half_rows(const float* src, int64_t rows, int64_t cols, int64_t ld, uint16_t* half, int* exps,
                            uint16_t* planes, hipStream_t st, const int* place, float* cleared) {
    if (rows <= 0) return hipSuccess;
    const int64_t blocks = (rows + 3) / 4;
    const dim3 grid((unsigned)(blocks < 16384 ? blocks : 16384));
#define SC_HALF(ENDS_)                                                                                              \
    if (planes)                                                                                                    \
        hipLaunchKernelGGL((half_rows_kernel<ENDS_, true>), grid, dim3(256), 0, st, src, rows, (int)cols, ld, half, \
                           exps, planes, place, cleared);                                                          \
    else                                                                                                           \
        hipLaunchKernelGGL((half_rows_kernel<ENDS_, false>), grid, dim3(256), 0, st, src, rows, (int)cols, ld, half, \
                           exps, planes, place, cleared);
    switch (row_ends(cols)) {
        case ROW_WHOLE: SC_HALF(ROW_WHOLE) break;
        case ROW_CUT: SC_HALF(ROW_CUT) break;
        case ROW_SHORT: SC_HALF(ROW_SHORT) break;
    }
#undef SC_HALF
    return hipGetLastError();
}

hipError_t launch_to_planes(bool bf16, const void* src, int64_t rows, int64_t cols, uint16_t* dst, int64_t ld,
                            int64_t plane, const int64_t* targets, int64_t vocab, hipStream_t st, const int* place,
                            void* cleared) {
    const int64_t n = rows * (ld / 8);
    if (n <= 0) return hipSuccess;
    if (!targets) vocab = 1;  // every row counts
    const int64_t blocks = (n + 256 * kGroups - 1) / (256 * kGroups);
    const dim3 grid((unsigned)(blocks < 65536 ? blocks : 65536));
#define SC_PLANES(E_, ENDS_)                                                                                         \
    hipLaunchKernelGGL((to_planes_kernel<E_, ENDS_>), grid, dim3(256), 0, st, (const E_*)src, rows, (int)cols, dst, \
                       ld, plane, targets, vocab, place, (E_*)cleared);
    SC_BY_ENDS(bf16, cols, SC_PLANES)
#undef SC_PLANES
    return hipGetLastError();
}

}  // namespace scopt
