// Layer norm with its gradient:
//
//   h = x + r,  mu = mean(h),  rstd = 1 / sqrt(mean((h - mu)^2) + eps),  n = (h - mu) rstd,  y = n g + b
//   a = dy g,  dx = dh + rstd (a - mean(a) - n mean(a n)),  dg = sum over tokens of dy n,  db = of dy
//
// The gradient reads n from the 8-bit checkpoint that the norm may leave (act.hip), or forms it from
// h, mu and rstd: mu in float32 is half a step off, the same for the whole row, and in a row far from 0 a step is
// much of the deviation (mean 100, deviation 0.001: 0.4%), so the mean of n is taken off again.  Each element passes
// once, so HBM bounds both: the row stays in registers between its sums and the outputs.  65536 x 2048 in bfloat16
// with a residual: norm 197 us (5.5 TB/s), 236 us with the checkpoint (5.1); gradient from the checkpoint 174 us
// (5.4), from h 194 us (5.5); a copy of 1 GiB reaches 5.1.
#include <cmath>

#include "rows.hpp"
#include "internal.hpp"
#include "train.hpp"

namespace scopt {

// The norm's threads of a workgroup (its rows share no barriers), and workgroups of a launch, that further
// rows are dealt to: 2048 are resident at once where a row takes few registers (65536 x 2048 in bfloat16:
// 197 us; a workgroup for each row 244).
constexpr int ln_block(int tpr) { return tpr == 64 ? 256 : tpr; }
constexpr int64_t kLnGrid = 2048;

// The gradient's shapes by row length: threads of a row, its groups of 8 a thread, rows of a workgroup and the
// most workgroups.  Each workgroup leaves two partial rows of float32, so few of them with many rows save
// traffic (2051 x 4100 in float32: 32.0 us with 256 workgroups of 768 threads, 35.1 with 512 of 256 and three groups).
struct LnGradShape {
    int most_h, tpr, c, rows, parts;
};
constexpr LnGradShape kLnGrad[7] = {{512, 64, 1, 4, 512},   {1024, 64, 2, 4, 512},  {2048, 256, 1, 4, 256},
                                    {4096, 256, 2, 2, 256}, {6144, 768, 1, 1, 256}, {8192, 512, 2, 1, 256},
                                    {16384, 512, 4, 1, 256}};
constexpr int ln_grad_shape(int H) {
    int i = 0;
    while (H > kLnGrad[i].most_h) ++i;
    return i;
}

// Sums of N values over the TPR threads of a row, used in turn as act.hip's row_sum.
template <int TPR, int N, typename F>
__device__ __forceinline__ void row_sums(F (&v)[N], F (*red)[TPR / 64][N], int turn) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += __shfl_xor(v[k], o);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int k = 0; k < N; ++k) red[turn][threadIdx.x % TPR / 64][k] = v[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = F(0);
#pragma unroll
        for (int w = 0; w < TPR / 64; ++w)
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] += red[turn][w][k];
    }
}

// Rows are summed and normalised in 64 bits, as the root-mean-square norm's are: a value next to
// the border of two of the checkpoint's steps falls to the side that it belongs to.  The variance is taken
// about the mean, from the registers: nothing cancels.  h may be x or res: a row is stored after its first
// sum, which every thread of the row has loaded for.  Gain and bias stay in registers over the rows of
// a workgroup, and where the registers allow (C <= 2) a row is fetched while the one before it is worked on.
template <typename E, int ENDS, int C> struct LnInput {
    Group8<E, ENDS> x[C], r[C];
};
template <typename E, int ENDS, int TPR, int C, bool KEEP>
__global__ __launch_bounds__(ln_block(TPR)) void layernorm_kernel(const E* x, const E* res,
                                                                          const E* __restrict__ gain,
                                                                          const E* __restrict__ bias, float eps,
                                                                          int64_t T, int H, E* h, E* y, float* mean,
                                                                          float* rstd, int8_t* q, uint8_t* e) {
    constexpr int ROWS = ln_block(TPR) / TPR;
    __shared__ double red[2][TPR / 64][1];
    const int in = threadIdx.x % TPR;
    const int nb = (H + kActBlock - 1) / kActBlock;
    Group8<E, ENDS> gw[C], bw[C];
#pragma unroll
    for (int j = 0; j < C; ++j) gw[j].load(gain, (j * TPR + in) * 8, H);
    if (bias) {
#pragma unroll
        for (int j = 0; j < C; ++j) bw[j].load(bias, (j * TPR + in) * 8, H);
    }
    using Input = LnInput<E, ENDS, C>;
    auto fetch = [&](int64_t t, Input& r) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < C; ++j) r.x[j].load(x + t * H, (j * TPR + in) * 8, H);
        if (res) {
#pragma unroll
            for (int j = 0; j < C; ++j) r.r[j].load(res + t * H, (j * TPR + in) * 8, H);
        }
    };
    constexpr bool AHEAD = C <= 2;
    const int64_t stride = (int64_t)gridDim.x * ROWS;
    int64_t t = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
    Input cur, next;
    if (AHEAD && t < T) fetch(t, next);
    for (; t < T; t += stride) {  // wave-uniform
        if (AHEAD) {
            cur = next;
            if (t + stride < T) fetch(t + stride, next);
        } else {
            fetch(t, cur);
        }
        double v[C][8], s[1] = {0.0};
#pragma unroll
        for (int j = 0; j < C; ++j) {
            float a[8], r[8];
            value8(cur.x[j], (j * TPR + in) * 8, H, a);
            if (res) value8(cur.r[j], (j * TPR + in) * 8, H, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[j][i] = res ? (double)a[i] + (double)r[i] : (double)a[i];
                s[0] += v[j][i];
            }
        }
        row_sums<TPR>(s, red, 0);
        const double mu = s[0] / (double)H;
        s[0] = 0.0;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c = (j * TPR + in) * 8, left = H - c;
            if (h && left > 0) {
                float f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = (float)v[j][i];
                store8(h + t * H + c, left, f);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[j][i] = i < left ? v[j][i] - mu : 0.0;  // the norm of the sum, not of the rounded h
                s[0] = fma(v[j][i], v[j][i], s[0]);
            }
        }
        row_sums<TPR>(s, red, 1);
        const double rs = 1.0 / sqrt(s[0] / (double)H + (double)eps);
        if (in == 0) {
            gst(mean + t, (float)mu);
            gst(rstd + t, (float)rs);
        }
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c = (j * TPR + in) * 8, left = H - c;
            float f[8], g[8], b[8];
            value8(gw[j], c, H, g);
            if (bias) value8(bw[j], c, H, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[j][i] *= rs;
                f[i] = bias ? fmaf((float)v[j][i], g[i], b[i]) : (float)v[j][i] * g[i];
            }
            if (left > 0) store8(y + t * H + c, left, f);
            if constexpr (KEEP) {
                int8_t k[8];
                uint8_t ex;
                act_encode8(v[j], k, ex);
                if (left > 0) {
                    store_q8(q + t * H + c, left, k);
                    if ((in & 3) == 0) gst(e + t * nb + c / kActBlock, ex);
                }
            }
        }
    }
}

// A row's normalised values as fetched: from the checkpoint, or from h with the row's statistics.
template <typename E, int ENDS, bool KEPT, int C> struct LnRow {
    Group8<E, ENDS> dy[C], dh[C];
    GroupQ8<ENDS> q[C];
    float rs;
};
template <typename E, int ENDS, int C> struct LnRow<E, ENDS, false, C> {
    Group8<E, ENDS> dy[C], dh[C], h[C];
    float rs, mu;
};
template <typename E> struct LnGradArgs {
    const E *dy, *gain;
    const float *rstd, *mean;
    const int8_t* q;
    const uint8_t* e;
    const E *h, *dh;
    int64_t T;
    int H;
    E* dx;
    float* partial;
};

// Rows are dealt to the workgroups in turn; each keeps its rows' sums of dy n and dy in registers
// and writes two rows of `partial`, summed in a fixed order by layernorm_dgain_kernel.  Where the
// registers allow (C <= 2) a row is fetched while the one before it is worked on.
template <typename E, int ENDS, int TPR, int C, int ROWS, bool KEPT>
__global__ __launch_bounds__(TPR * ROWS) void layernorm_grad_kernel(const LnGradArgs<E> P) {
    constexpr bool JOINT = ROWS > 1 && TPR > 64;  // the rows share barriers: all of them take every turn
    constexpr int SUMS = !KEPT && JOINT ? 3 : 2;
    __shared__ float red[ROWS][2][TPR / 64][SUMS];
    __shared__ float red_n[ROWS][2][TPR / 64][1];
    __shared__ float sums[ROWS > 1 ? TPR * 16 : 1];
    const int in = threadIdx.x % TPR, row = threadIdx.x / TPR;
    const int H = P.H, nb = (H + kActBlock - 1) / kActBlock;
    const int64_t T = P.T;
    float g[C][8], dg[C][8], db[C][8];
#pragma unroll
    for (int j = 0; j < C; ++j) {
        load8<ENDS>(P.gain, (j * TPR + in) * 8, H, g[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) dg[j][i] = db[j][i] = 0.0f;
    }
    const int64_t stride = (int64_t)gridDim.x * ROWS;
    using Row = LnRow<E, ENDS, KEPT, C>;
    auto fetch = [&](int64_t t, Row& r) __attribute__((always_inline)) {
        r.rs = gld(P.rstd + t);
        if constexpr (!KEPT) r.mu = gld(P.mean + t);
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c = (j * TPR + in) * 8;
            r.dy[j].load(P.dy + t * H, c, H);
            if constexpr (KEPT) r.q[j].load(P.q + t * H, P.e + t * nb, c, H);
            else r.h[j].load(P.h + t * H, c, H);
        }
        if (P.dh) {
#pragma unroll
            for (int j = 0; j < C; ++j) r.dh[j].load(P.dh + t * H, (j * TPR + in) * 8, H);
        }
    };
    constexpr bool AHEAD = C <= 2 && TPR < 1024;
    Row cur, next;
    int64_t t = (int64_t)blockIdx.x * ROWS + row;
    int turn = 0;
    if (AHEAD) fetch(t < T ? t : T - 1, next);
    for (; t - (JOINT ? row : 0) < T; t += stride, turn ^= 1) {
        const bool live = !JOINT || t < T;
        if (AHEAD) {
            cur = next;
            fetch(t + stride < T ? t + stride : T - 1, next);
        } else {
            fetch(live ? t : T - 1, cur);
        }
        float a[C][8], n[C][8], s[SUMS] = {};
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c = (j * TPR + in) * 8;
            value8(cur.dy[j], c, H, a[j]);
            if constexpr (JOINT) {
#pragma unroll
                for (int i = 0; i < 8; ++i) a[j][i] = live ? a[j][i] : 0.0f;
            }
            if constexpr (KEPT) {
                cur.q[j].value(c, H, n[j]);
            } else {
                value8(cur.h[j], c, H, n[j]);
#pragma unroll
                for (int i = 0; i < 8; ++i) n[j][i] = c + i < H ? (n[j][i] - cur.mu) * cur.rs : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dg[j][i] = fmaf(a[j][i], n[j][i], dg[j][i]);
                if constexpr (SUMS > 2) s[2] += n[j][i];
                db[j][i] += a[j][i];
                a[j][i] *= g[j][i];
                s[0] += a[j][i];
                s[1] = fmaf(a[j][i], n[j][i], s[1]);
            }
        }
        // dx may be dy or dh: a cut row's last group overlaps another thread's, so dh has to have
        // arrived before any thread passes the sum
        if constexpr (ENDS == ROW_CUT) {
            if (P.dh) {
#pragma unroll
                for (int j = 0; j < C; ++j) cur.dh[j].arrived();
            }
        }
        row_sums<TPR>(s, red[row], turn);
        const float c0 = s[0] / (float)H;
        float c1 = s[1] / (float)H;
        if constexpr (!KEPT) {
            // What the mean's rounding left in the row comes off: not where it is more than that, as the mean is
            // another one, nor where it is less than the sums' own rounding.  (Rows of their own barriers form the
            // sum where it is needed: 2051 x 4100 in float32 32.1 us, in every row 33.4.)
            const float most = 0x1p-22f * fabsf(cur.mu) * cur.rs;
            if (__builtin_expect(most > 0x1p-20f, 0)) {
                float left[1] = {s[SUMS - 1]};
                if constexpr (SUMS == 2) {
                    left[0] = 0.0f;
#pragma unroll
                    for (int j = 0; j < C; ++j)
#pragma unroll
                        for (int i = 0; i < 8; ++i) left[0] += n[j][i];
                    row_sums<TPR>(left, red_n[row], turn);
                }
                const float mean = left[0] / (float)H, shift = fabsf(mean) <= most ? mean : 0.0f;
                c1 = fmaf(-shift, c0, c1);
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    const int c = (j * TPR + in) * 8;
                    float dy[8];
                    value8(cur.dy[j], c, H, dy);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        n[j][i] -= c + i < H ? shift : 0.0f;
                        dg[j][i] = fmaf(live ? dy[i] : 0.0f, -shift, dg[j][i]);
                    }
                }
            }
        }
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c = (j * TPR + in) * 8, left = H - c;
            float d[8];
            if (P.dh) {
                value8(cur.dh[j], c, H, d);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) d[i] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = fmaf(cur.rs, fmaf(-n[j][i], c1, a[j][i] - c0), d[i]);
            if (left > 0 && live) store8(P.dx + t * H + c, left, d);
        }
    }
    float* out = P.partial + (int64_t)blockIdx.x * 2 * H;
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const int c = (j * TPR + in) * 8;
        if constexpr (ROWS > 1) {
            // the workgroup's rows, one after the other
            for (int w = 0; w < ROWS; ++w) {
                if (row == w) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float* p = sums + (in * 8 + i) * 2;
                        p[0] = w ? p[0] + dg[j][i] : dg[j][i];
                        p[1] = w ? p[1] + db[j][i] : db[j][i];
                    }
                }
                __syncthreads();
            }
            if (row == 0 && H - c > 0) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dg[j][i] = sums[(in * 8 + i) * 2];
                    db[j][i] = sums[(in * 8 + i) * 2 + 1];
                }
                store8(out + c, H - c, dg[j]);
                store8(out + H + c, H - c, db[j]);
            }
            __syncthreads();
        } else if (H - c > 0) {
            store8(out + c, H - c, dg[j]);
            store8(out + H + c, H - c, db[j]);
        }
    }
}

// 16 of the 2 H columns a workgroup, 64 groups of partial rows
__global__ __launch_bounds__(1024) void layernorm_dgain_kernel(const float* __restrict__ partial, int parts, int H,
                                                               float* __restrict__ dgain, float* __restrict__ dbias) {
    __shared__ float red[16][16];
    const int col = threadIdx.x & 15, grp = threadIdx.x >> 4;
    const int c = blockIdx.x * 16 + col;
    float s = 0.0f;
    if (c < 2 * H) {
#pragma unroll 8
        for (int p = grp; p < parts; p += 64) s += gld(partial + (int64_t)p * 2 * H + c);
    }
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if ((threadIdx.x & 63) < 16) red[threadIdx.x >> 6][col] = s;
    __syncthreads();
    if (threadIdx.x < 16 && c < 2 * H) {
        s = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k) s += red[k][col];
        if (c < H) gst(dgain + c, s);
        else if (dbias) gst(dbias + c - H, s);
    }
}

// The norm's threads and groups of 8 a row.  A wavefront takes rows of up to 2048 elements by itself: no
// barriers (65536 x 2048: 197 us in bfloat16, 394 in float32; four wavefronts a row 220 and 421).
template <typename E, int ENDS, int TPR, int C, typename... A>
static void ln_rows(int64_t T, hipStream_t st, int8_t* q, A... args) {
    constexpr int64_t rows = ln_block(TPR) / TPR;
    const int64_t b = (T + rows - 1) / rows;
    const dim3 grid((unsigned)(b < kLnGrid ? b : kLnGrid)), blk(ln_block(TPR));
    if (q) hipLaunchKernelGGL((layernorm_kernel<E, ENDS, TPR, C, true>), grid, blk, 0, st, args...);
    else hipLaunchKernelGGL((layernorm_kernel<E, ENDS, TPR, C, false>), grid, blk, 0, st, args...);
}
template <typename E, int ENDS, typename... A>
static void ln_sizes(int H, int64_t T, A... args) {
    if (ENDS == ROW_SHORT || H <= 512) ln_rows<E, ENDS, 64, 1>(T, args...);
    else if constexpr (ENDS != ROW_SHORT) {
        if (H <= 1024) ln_rows<E, ENDS, 64, 2>(T, args...);
        // (32 rows of 2048: 4.5 us, a wavefront each 7.3)
        else if (H <= 2048 && T <= 1024) ln_rows<E, ENDS, 256, 1>(T, args...);
        else if (H <= 1536) ln_rows<E, ENDS, 64, 3>(T, args...);
        else if (H <= 2048) ln_rows<E, ENDS, 64, 4>(T, args...);
        else if (H <= 4096) ln_rows<E, ENDS, 256, 2>(T, args...);
        else if (H <= 6144) ln_rows<E, ENDS, 256, 3>(T, args...);
        else if (H <= 8192) ln_rows<E, ENDS, 256, 4>(T, args...);
        else ln_rows<E, ENDS, 512, 4>(T, args...);
    }
}
template <typename E, int ENDS, int I>
static void ln_grad_sizes(int H, int parts, hipStream_t st, const LnGradArgs<E>& a) {
    constexpr LnGradShape S = kLnGrad[I];
    if constexpr (I + 1 < 7 && ENDS != ROW_SHORT)
        if (H > S.most_h) return ln_grad_sizes<E, ENDS, I + 1>(H, parts, st, a);
    const dim3 grid((unsigned)parts), blk(S.tpr * S.rows);
    if (a.q) hipLaunchKernelGGL((layernorm_grad_kernel<E, ENDS, S.tpr, S.c, S.rows, true>), grid, blk, 0, st, a);
    else hipLaunchKernelGGL((layernorm_grad_kernel<E, ENDS, S.tpr, S.c, S.rows, false>), grid, blk, 0, st, a);
}

hipError_t launch_layernorm(bool bf16, const void* x, const void* residual, const void* gain, const void* bias,
                            float eps, int64_t T, int H, void* h, void* y, float* mean, float* rstd, int8_t* q,
                            uint8_t* e, hipStream_t st) {
    if (T <= 0) return hipSuccess;
#define SC_NORM(E_, ENDS_)                                                                                      \
    ln_sizes<E_, ENDS_>(H, T, st, q, (const E_*)x, (const E_*)residual, (const E_*)gain, (const E_*)bias, \
                                   eps, T, H, (E_*)h, (E_*)y, mean, rstd, q, e);
    SC_BY_ENDS(bf16, H, SC_NORM)
#undef SC_NORM
    return hipGetLastError();
}

int64_t layernorm_grad_parts(int64_t T, int H) {
    const LnGradShape& S = kLnGrad[ln_grad_shape(H)];
    const int64_t wgs = (T + S.rows - 1) / S.rows;
    return wgs < S.parts ? wgs : S.parts;
}

hipError_t launch_layernorm_grad(bool bf16, const void* dy, const void* gain, const float* rstd, const float* mean,
                                 const int8_t* q, const uint8_t* e, const void* h, const void* dh, int64_t T, int H,
                                 void* dx, float* dgain, float* dbias, float* partial, hipStream_t st) {
    const int parts = (int)layernorm_grad_parts(T, H);
    if (T > 0) {
#define SC_GRAD(E_, ENDS_)                                                                                      \
    LnGradArgs<E_> a{(const E_*)dy, (const E_*)gain, rstd, mean, q, e, (const E_*)h, (const E_*)dh, T, H, (E_*)dx, \
                     partial};                                                                                  \
    ln_grad_sizes<E_, ENDS_, 0>(H, parts, st, a);
        SC_BY_ENDS(bf16, H, SC_GRAD)
#undef SC_GRAD
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    hipLaunchKernelGGL(layernorm_dgain_kernel, dim3((unsigned)((2 * H + 15) / 16)), dim3(1024), 0, st, partial, parts,
                       H, dgain, dbias);
    return hipGetLastError();
}

}  // namespace scopt
