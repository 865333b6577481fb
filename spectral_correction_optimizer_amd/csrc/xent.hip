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
#include <cmath>

#include "tile_product.hpp"

namespace scopt {

namespace {
constexpr int64_t kAlign = 256;
int64_t up(int64_t n, int64_t a) { return (n + a - 1) / a * a; }
}  // namespace

// 64 tokens a workgroup, one a lane, the tiles dealt to 16 wavefronts: a row's log-sum-exp from
// its tiles' references and sums [tile][T], and its loss.  pow2: the references are powers of
// two.  A row of -infinity only has no finite log-sum-exp; like a row with NaN or +infinity
// it gives NaN.
__global__ __launch_bounds__(1024) void xent_lse_kernel(const float* __restrict__ smax,
                                                        const float* __restrict__ ssum, int tiles, int pow2,
                                                        const float* __restrict__ target_logit,
                                                        const int64_t* __restrict__ targets, int64_t T, int64_t V,
                                                        float* __restrict__ lse, float* __restrict__ loss) {
    __shared__ float red[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * 64 + lane, at = t < T ? t : T - 1;
    const float none = -__builtin_huge_valf();
    // a difference of references as a factor; a tile of -infinity has sum 0 (or NaN)
    auto scaled = [&](float s, float r, float to) {
        return r == none ? s : s * (pow2 ? exp2f(r - to) : expf(r - to));
    };
    // sixteen tiles' values in flight, joined to the running reference and sum
    float m = none, z = 0.0f;
    constexpr int U = 16;
    for (int i0 = wave; i0 < tiles; i0 += 16 * U) {
        float r[U], s[U], top = m;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = i0 + 16 * u < tiles ? i0 + 16 * u : tiles - 1;
            r[u] = gld(smax + i * T + at);
            s[u] = gld(ssum + i * T + at);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) top = i0 + 16 * u < tiles ? fmaxf(top, r[u]) : top;
        z = scaled(z, m, top);
        m = top;
#pragma unroll
        for (int u = 0; u < U; ++u) z += i0 + 16 * u < tiles ? scaled(s[u], r[u], m) : 0.0f;
    }
    red[wave][lane] = m;
    __syncthreads();
    float top = none;
#pragma unroll
    for (int w = 0; w < 16; ++w) top = fmaxf(top, red[w][lane]);
    z = scaled(z, m, top);
    m = top;
    __syncthreads();
    red[wave][lane] = z;
    __syncthreads();
    if (wave > 0 || t >= T) return;
    z = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) z += red[w][lane];
    // a power of two's logarithm in two parts: m * ln2 is off by less than 2^-40 of m
    const float base = pow2 ? m * 0.693145751953125f : m, rest = pow2 ? m * 1.42860682030941723e-6f : 0.0f;
    const float logz = m == none ? __builtin_nanf("") : logf(z) + rest;
    const bool counted = tp_target(targets, V, t) >= 0;
    gst(lse + t, base + logz);
    gst(loss + t, counted ? (base - gld(target_logit + t)) + logz : 0.0f);
}

// d from what the logits product kept: exponentials in 16 bits (in place) or float32 logits
// (into three planes).  `chunks` workgroups a row; a thread takes 8 columns at a time.
template <bool EXP>
__global__ __launch_bounds__(256) void xent_dlogits_kernel(const float* __restrict__ logits, uint16_t* P,
                                                           int64_t plane, int64_t ldp, int N, int bn,
                                                           int64_t chunk, int chunks,
                                                           const float* __restrict__ smax, int64_t T,
                                                           const float* __restrict__ lse,
                                                           const float* __restrict__ target_logit,
                                                           const int64_t* __restrict__ targets, int64_t V,
                                                           const float* __restrict__ scale_at) {
    const int64_t t = blockIdx.x / chunks;
    const float scale = gld(scale_at);
    const int64_t tgt = tp_target(targets, V, t);
    const float ls = gld(lse + t);
    const float ls2 = ls * kLog2e;
    const float at_target = tgt >= 0 ? (expf(gld(target_logit + t) - ls) - 1.0f) * scale : 0.0f;
    const int64_t end = (N + 7) & ~7;  // the products read no further
    const int64_t from = (int64_t)(blockIdx.x % chunks) * chunk, to = from + chunk < end ? from + chunk : end;
    for (int64_t c = from + 8 * threadIdx.x; c < to; c += 8 * 256) {
        uint16_t* p = P + t * ldp + c;
        float v[8];
        if constexpr (EXP) {
            const v4u w = *(const SC_GLOBAL v4u*)p;
            const float f = __builtin_amdgcn_exp2f(gld(smax + (int64_t)(c / bn) * T + t) - ls2) * scale;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = tp_unit_lo(w[i]) * f;
                v[2 * i + 1] = tp_unit_hi(w[i]) * f;
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

XentPlan xent_plan(bool bf16, int64_t T, int64_t V, int64_t H, int64_t limit) {
    XentPlan p{};
    p.bf16 = bf16;
    p.T = T;
    p.V = V;
    p.H = H;
    p.planes = !bf16 || H % 8 != 0;
    p.Hp = p.planes ? tp_pad(up(H, 64)) : H;
    p.Hh = tp_pad(up(H, 64));
    const int nseg = bf16 ? 1 : 6;
    // bytes of a vocabulary column: the kept exponentials, or the logits and d's planes
    const int64_t col_kept = T * (bf16 ? 2 : 10), col_piece = T * (bf16 ? 2 : 6);
    p.keep = up(V, 256) * col_kept <= limit;
    p.piece = V;
    if (!p.keep) {
        p.piece = limit / col_piece / 256 * 256;
        if (p.piece < 256) p.piece = 256;
        if (p.piece > V) p.piece = V;
    }
    p.pieces = (int)((V + p.piece - 1) / p.piece);
    p.ldp = tp_pad(up(p.piece, 256));  // the logits' tiles are stored whole
    const int64_t last = V - (int64_t)(p.pieces - 1) * p.piece;
    p.logits = tp_plan((int)T, (int)p.piece, (int)H, nseg, false);
    p.logits_last = tp_plan((int)T, (int)last, (int)H, nseg, false);
    p.dh = tp_plan((int)T, (int)H, (int)p.piece, nseg, true);
    p.dw = tp_plan((int)p.piece, (int)H, (int)T, nseg, true);
    p.dw_last = tp_plan((int)last, (int)H, (int)T, nseg, true);
    p.stat_tiles = (int64_t)(p.pieces - 1) * p.logits.tiles_n + p.logits_last.tiles_n;
    int64_t o = 0;
    auto take = [&](int64_t bytes) {
        const int64_t at = o;
        o += up(bytes, kAlign);
        return at;
    };
    const int np = bf16 ? 1 : 3;
    p.o_factors = take(8);
    p.o_h = take(2 * np * T * p.Hh);
    p.o_w = p.planes ? take(2 * np * V * p.Hp) : 0;
    p.o_s = !bf16 && p.keep ? take(4 * T * p.ldp) : 0;
    p.o_p = take(2 * np * T * p.ldp);
    p.o_tl = take(4 * T);
    p.o_lse = take(4 * T);
    p.o_smax = take(4 * T * p.stat_tiles);
    p.o_ssum = take(4 * T * p.stat_tiles);
    const bool join = p.pieces > 1;
    int64_t part = p.dh.part_bytes;
    if (join && part == 0) part = 4 * T * H;
    part = part > p.dw.part_bytes ? part : p.dw.part_bytes;
    part = part > p.dw_last.part_bytes ? part : p.dw_last.part_bytes;
    p.o_part = take(part);
    p.o_dh = join ? take(4 * T * H) : 0;
    p.bytes = o;
    return p;
}

hipError_t launch_xent(const XentPlan& p, const void* h, const void* W, const int64_t* targets, float* loss,
                       float* mean, void* dh, void* dW, void* workspace, hipStream_t st) {
    char* ws = (char*)workspace;
    const int64_t T = p.T, V = p.V, H = p.H, Hp = p.Hp, Hh = p.Hh;
    const int np = p.bf16 ? 1 : 3;
    float* factors = (float*)(ws + p.o_factors);
    uint16_t* P = (uint16_t*)(ws + p.o_p);
    float* S = (float*)(ws + p.o_s);
    float *tl = (float*)(ws + p.o_tl), *lse = (float*)(ws + p.o_lse);
    float *smax = (float*)(ws + p.o_smax), *ssum = (float*)(ws + p.o_ssum);
    float *part = (float*)(ws + p.o_part), *dhs = (float*)(ws + p.o_dh);
    hipError_t e;
    if (T == 0) {
        if ((e = launch_zero(mean, 4, st)) != hipSuccess) return e;
        return launch_zero(dW, V * H * (p.bf16 ? 2 : 4), st);
    }
#define SC_RUN(expr) \
    if ((e = (expr)) != hipSuccess) return e

    // h is always copied, with zeros for the tokens that are not counted: whatever they hold
    // (a NaN too) reaches no product
    uint16_t* hp = (uint16_t*)(ws + p.o_h);
    const uint16_t* wp = (const uint16_t*)W;
    SC_RUN(launch_to_planes(p.bf16, h, T, H, hp, Hh, T * Hh, targets, V, st));
    if (p.planes) {
        wp = (uint16_t*)(ws + p.o_w);
        SC_RUN(launch_to_planes(p.bf16, W, V, H, (uint16_t*)wp, Hp, V * Hp, nullptr, 0, st));
    }
    // planes (A | B << 2) of the six products of two split operands, smallest first
    const uint64_t segs = p.bf16 ? 0 : 0x0 << 20 | 0x4 << 16 | 0x1 << 12 | 0x8 << 8 | 0x5 << 4 | 0x2;
    const int nseg = p.bf16 ? 1 : 6;

    auto logits = [&](int i) {
        TpArgs a;
        const int64_t v0 = (int64_t)i * p.piece;
        a.A = hp;
        a.lda = Hh;
        a.a_plane = T * Hh;
        a.B = wp + v0 * Hp;
        a.ldb = Hp;
        a.b_plane = V * Hp;
        a.M = (int)T;
        a.N = (int)(V - v0 < p.piece ? V - v0 : p.piece);
        a.K = (int)up(H, 8);
        a.nseg = nseg;
        a.segs = segs;
        a.targets = targets;
        a.vocab = V;
        a.n_first = v0;
        a.ldp = p.ldp;
        a.p_plane = T * p.ldp;
        a.p_planes = np;
        a.target_logit = tl;
        a.stat_max = smax;
        a.stat_sum = ssum;
        a.stat_first = (int64_t)i * p.logits.tiles_n;
        a.lse = lse;
        return a;
    };
    auto logits_plan = [&](int i) -> const TpPlan& { return i + 1 < p.pieces ? p.logits : p.logits_last; };
    for (int i = 0; i < p.pieces; ++i) {
        TpArgs a = logits(i);
        a.keep = !p.keep ? TP_KEEP_NONE : p.bf16 ? TP_KEEP_EXP : TP_KEEP_LOGIT;
        a.P = p.bf16 ? (void*)P : (void*)S;
        SC_RUN(launch_tile_product(TPK_LOGIT_STATS, logits_plan(i), a, TpSum{}, st));
    }
    const int pow2 = p.keep && p.bf16;
    hipLaunchKernelGGL(xent_lse_kernel, dim3((unsigned)((T + 63) / 64)), dim3(1024), 0, st, smax, ssum,
                       (int)p.stat_tiles, pow2, tl, targets, T, V, lse, loss);
    SC_RUN(hipGetLastError());
    hipLaunchKernelGGL(xent_mean_kernel, dim3(1), dim3(1024), 0, st, loss, targets, T, V, factors, mean);
    SC_RUN(hipGetLastError());

    for (int i = 0; i < p.pieces; ++i) {
        const int64_t v0 = (int64_t)i * p.piece;
        const int n = (int)(V - v0 < p.piece ? V - v0 : p.piece);
        if (p.keep) {
            // enough workgroups for the chip, at least 2048 columns each
            const int64_t chunk = up((n * T + 4095) / 4096, 2048);
            const int chunks = (int)((n + chunk - 1) / chunk);
            const dim3 grid((unsigned)(chunks * T));
            if (p.bf16)
                hipLaunchKernelGGL(xent_dlogits_kernel<true>, grid, dim3(256), 0, st, nullptr, P, T * p.ldp, p.ldp, n,
                                   p.logits.bn, chunk, chunks, smax, T, lse, tl, targets, V, factors + 1);
            else
                hipLaunchKernelGGL(xent_dlogits_kernel<false>, grid, dim3(256), 0, st, S, P, T * p.ldp, p.ldp, n,
                                   p.logits.bn, chunk, chunks, smax, T, lse, tl, targets, V, factors + 1);
            SC_RUN(hipGetLastError());
        } else {
            TpArgs a = logits(i);
            a.P = P;
            a.alpha = factors + 1;
            SC_RUN(launch_tile_product(TPK_LOGIT_GRAD, logits_plan(i), a, TpSum{}, st));
        }
        TpArgs a;  // dh (+)= d W: k runs over the piece
        a.A = P;
        a.lda = p.ldp;
        a.a_plane = T * p.ldp;
        a.B = wp + v0 * Hp;
        a.ldb = Hp;
        a.b_plane = V * Hp;
        a.M = (int)T;
        a.N = (int)H;
        a.K = n;
        a.nseg = nseg;
        a.segs = segs;
        a.C = dh;
        a.ldc = H;
        a.c_bf16 = p.bf16;
        a.alpha = factors;
        a.part = part;
        TpSum sum;
        if (p.pieces > 1) {
            sum.acc = i > 0 ? dhs : nullptr;
            sum.out_acc = i + 1 < p.pieces ? dhs : nullptr;
        }
        SC_RUN(launch_tile_product(TPK_STATES, p.dh, a, sum, st));
        TpArgs b;  // dW = d^T h: k runs over the tokens
        b.A = P;
        b.lda = p.ldp;
        b.a_plane = T * p.ldp;
        b.B = hp;
        b.ldb = Hh;
        b.b_plane = T * Hh;
        b.M = n;
        b.N = (int)H;
        b.K = (int)T;
        b.nseg = nseg;
        b.segs = segs;
        b.C = (char*)dW + v0 * H * (p.bf16 ? 2 : 4);
        b.ldc = H;
        b.c_bf16 = p.bf16;
        b.alpha = factors;
        b.part = part;
        SC_RUN(launch_tile_product(TPK_WEIGHTS, i + 1 < p.pieces ? p.dw : p.dw_last, b, TpSum{}, st));
    }
#undef SC_RUN
    return hipSuccess;
}

}  // namespace scopt
