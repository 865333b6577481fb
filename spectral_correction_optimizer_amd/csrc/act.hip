// 8-bit activation checkpoints, the residual root-mean-square norm that writes one, its
// gradient from it, and the weight gradient of a projection whose input it is.
//
//   h = x + r,  rstd = 1 / sqrt(mean(h^2) + eps),  n = h rstd,  y = n g
//   the checkpoint keeps n in 8 bits: blocks of 32 along a row share a power of two,
//     E = max(floor(log2 max|n|), -120), q = round(n 2^(6 - E)) clipped to +-127
//   gradient: a = dy g, c = mean(a n), dx = dh + rstd (a - n c), dg = sum over tokens of dy n
//   weight gradient: dW[o][i] = g[i] sum over tokens of dy[t][o] n[t][i]
//
// The norm, its gradient and the conversions stream each element once and are bound by HBM.
// A wavefront owns a row of up to 1024 elements, a workgroup a longer one; the row stays in
// registers between the sum and the outputs.  The norm's sums are 64-bit, its gradient's float32.
// 65536 x 2048 in bfloat16: norm 220-232 us (5.2-5.5 TB/s), gradient 181 us (5.2 TB/s; without
// the row fetched ahead and with branches around the loads 333 us), checkpoint read 64 us (6.3
// TB/s, partly from cache).
#include <cmath>

#include "rows.hpp"
#include "internal.hpp"
#include "train.hpp"

namespace scopt {

namespace {
int64_t up(int64_t n, int64_t a) { return (n + a - 1) / a * a; }
}  // namespace

// A thread converts kGroups groups of 8 elements.  The four threads of a block of 32 are
// neighbours in a wave, and whole blocks leave the loop together (groups and strides are
// multiples of 4).
template <typename E, int ENDS>
__global__ __launch_bounds__(256) void act_pack_kernel(const E* __restrict__ x, int64_t T, int H, int8_t* q,
                                                       uint8_t* e) {
    const int nb = (H + kActBlock - 1) / kActBlock, per_row = nb * 4;
    const int64_t n = T * per_row;
    const bool small = n < (int64_t)1 << 31;
    for (int64_t g0 = (int64_t)blockIdx.x * 256 * kGroups + threadIdx.x; g0 < n;
         g0 += (int64_t)gridDim.x * 256 * kGroups) {
        Group8<E, ENDS> w[kGroups];
        int64_t t[kGroups];
        int in[kGroups];
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            const int64_t g = g0 + k * 256;
            split_group(g < n ? g : n - 4 + (threadIdx.x & 3), per_row, small, t[k], in[k]);
            w[k].load(x + t[k] * H, in[k] * 8, H);
        }
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            const int c = in[k] * 8;
            float v[8];
            value8(w[k], c, H, v);
            int8_t o[8];
            uint8_t ex;
            act_encode8(v, o, ex);
            if (g0 + k * 256 >= n) continue;
            store_q8(q + t[k] * H + c, H - c, o);
            if ((in[k] & 3) == 0) gst(e + t[k] * nb + in[k] / 4, ex);
        }
    }
}

// ld: columns of a row of x, zeros from H on
template <typename E, int ENDS>
__global__ __launch_bounds__(256) void act_unpack_kernel(const int8_t* __restrict__ q, const uint8_t* __restrict__ e,
                                                         int64_t T, int H, int64_t ld, E* x) {
    const int nb = (H + kActBlock - 1) / kActBlock, per_row = (int)((ld + 7) / 8);
    const int64_t n = T * per_row;
    const bool small = n < (int64_t)1 << 31;
    for (int64_t g0 = (int64_t)blockIdx.x * 256 * kGroups + threadIdx.x; g0 < n;
         g0 += (int64_t)gridDim.x * 256 * kGroups) {
        GroupQ8<ENDS> w[kGroups];
        int64_t t[kGroups];
        int in[kGroups];
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            const int64_t g = g0 + k * 256;
            split_group(g < n ? g : n - 1, per_row, small, t[k], in[k]);
            w[k].load(q + t[k] * H, e + t[k] * nb, in[k] * 8, H);
        }
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            const int c = in[k] * 8;
            float v[8];
            w[k].value(c, H, v);
            if (g0 + k * 256 < n) store8(x + t[k] * ld + c, (int)(ld - c), v);  // bfloat16: exact, 8 significant bits
        }
    }
}

// Sum over the TPR threads of a row: `red` holds a value per wave, twice, and is used in turn
// (`turn`), so that one barrier a row is enough.
template <int TPR, typename F>
__device__ __forceinline__ F row_sum(F v, F (*red)[TPR / 64], int turn) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) red[turn][threadIdx.x >> 6] = v;
        __syncthreads();
        v = F(0);
#pragma unroll
        for (int w = 0; w < TPR / 64; ++w) v += red[turn][w];
    }
    return v;
}

// The rows are normalised in 64 bits (the vector unit's rate for them is float32's, and HBM stays
// the bound): a value next to the border of two of the checkpoint's steps then falls to the
// side that it belongs to, which float32's roundings decided before, a few in a million.
//
// Rows beyond the grid's are taken in turn.  h may be x or res: a row is loaded whole (a cut
// row's last group overlaps another thread's) before row_sum, and stored after it.
template <typename E, int ENDS, int TPR, int C>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void rmsnorm_kernel(const E* x, const E* res,
                                                                        const E* __restrict__ gain, float eps,
                                                                        int64_t T, int H, E* h, E* y, float* rstd,
                                                                        int8_t* q, uint8_t* e) {
    constexpr int ROWS = TPR > 256 ? 1 : 256 / TPR;
    __shared__ double red[2][TPR / 64];
    const int in = threadIdx.x % TPR;
    const int nb = (H + kActBlock - 1) / kActBlock;
    int turn = 0;
    for (int64_t t = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR; t < T;  // wave-uniform
         t += (int64_t)gridDim.x * ROWS, turn ^= 1) {
        Group8<E, ENDS> xw[C], rw[C], gw[C];
#pragma unroll
        for (int j = 0; j < C; ++j) xw[j].load(x + t * H, (j * TPR + in) * 8, H);
        if (res) {
#pragma unroll
            for (int j = 0; j < C; ++j) rw[j].load(res + t * H, (j * TPR + in) * 8, H);
        }
#pragma unroll
        for (int j = 0; j < C; ++j) gw[j].load(gain, (j * TPR + in) * 8, H);
        auto sums = [&](int j, double (&v)[8]) __attribute__((always_inline)) {
            float a[8], r[8];
            value8(xw[j], (j * TPR + in) * 8, H, a);
            if (res) value8(rw[j], (j * TPR + in) * 8, H, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = res ? (double)a[i] + (double)r[i] : (double)a[i];
        };
        double ss = 0.0;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            double v[8];
            sums(j, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fma(v[i], v[i], ss);
        }
        ss = row_sum<TPR>(ss, red, turn);
        const double rs = 1.0 / sqrt(ss / (double)H + (double)eps);
        if (in == 0) gst(rstd + t, (float)rs);
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c = (j * TPR + in) * 8, left = H - c;
            double v[8];
            float f[8], g[8];
            sums(j, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = (float)v[i];
            if (h && left > 0) store8(h + t * H + c, left, f);
            value8(gw[j], c, H, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] *= rs;  // the norm of the sum, not of the rounded h
                f[i] = (float)v[i] * g[i];
            }
            if (left > 0) store8(y + t * H + c, left, f);
            if (q) {
                int8_t k[8];
                uint8_t ex;
                act_encode8(v, k, ex);
                if (left > 0) {
                    store_q8(q + t * H + c, left, k);
                    if ((in & 3) == 0) gst(e + t * nb + c / kActBlock, ex);
                }
            }
        }
    }
}

// Rows are dealt to the workgroups in turn; each keeps its rows' sum of dy n in registers and
// writes one row of `partial`, summed in a fixed order by rmsnorm_dgain_kernel.  Where the
// registers allow (C <= 2) a row is fetched while the one before it is worked on.
template <typename E, int ENDS, int C> struct NormGradRow {
    Group8<E, ENDS> dy[C], dh[C];
    GroupQ8<ENDS> n[C];
    float rs;
};
template <typename E, int ENDS, int TPR, int C>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void rmsnorm_grad_kernel(
    const E* dy, const E* __restrict__ gain, const float* __restrict__ rstd, const int8_t* __restrict__ q,
    const uint8_t* __restrict__ e, const E* dh, int64_t T, int H, E* dx, float* partial) {
    constexpr int ROWS = TPR > 256 ? 1 : 256 / TPR;
    __shared__ float red[2][TPR / 64];
    __shared__ float sums[ROWS > 1 ? TPR * 8 : 1];
    const int in = threadIdx.x % TPR, row = threadIdx.x / TPR;
    const int nb = (H + kActBlock - 1) / kActBlock;
    float g[C][8], dg[C][8];
#pragma unroll
    for (int j = 0; j < C; ++j) {
        load8<ENDS>(gain, (j * TPR + in) * 8, H, g[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) dg[j][i] = 0.0f;
    }
    const int64_t stride = (int64_t)gridDim.x * ROWS;
    auto fetch = [&](int64_t t, NormGradRow<E, ENDS, C>& r) __attribute__((always_inline)) {
        r.rs = gld(rstd + t);
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c = (j * TPR + in) * 8;
            r.dy[j].load(dy + t * H, c, H);
            r.n[j].load(q + t * H, e + t * nb, c, H);
        }
        if (dh) {
#pragma unroll
            for (int j = 0; j < C; ++j) r.dh[j].load(dh + t * H, (j * TPR + in) * 8, H);
        }
    };
    constexpr bool AHEAD = C <= 2;
    NormGradRow<E, ENDS, C> cur, next;
    int64_t t = (int64_t)blockIdx.x * ROWS + row;
    int turn = 0;
    if (AHEAD && t < T) fetch(t, next);
    for (; t < T; t += stride, turn ^= 1) {
        if (AHEAD) {
            cur = next;
            fetch(t + stride < T ? t + stride : t, next);
        } else {
            fetch(t, cur);
        }
        float a[C][8], n[C][8], dot = 0.0f;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            value8(cur.dy[j], (j * TPR + in) * 8, H, a[j]);
            cur.n[j].value((j * TPR + in) * 8, H, n[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dg[j][i] = fmaf(a[j][i], n[j][i], dg[j][i]);
                a[j][i] *= g[j][i];
                dot = fmaf(a[j][i], n[j][i], dot);
            }
        }
        // dx may be dy or dh: a cut row's last group overlaps another thread's, so dh has to have
        // arrived before any thread passes the sum
        if constexpr (ENDS == ROW_CUT) {
            if (dh) {
#pragma unroll
                for (int j = 0; j < C; ++j) cur.dh[j].arrived();
            }
        }
        const float c1 = row_sum<TPR>(dot, red, turn) / (float)H;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c = (j * TPR + in) * 8, left = H - c;
            float d[8];
            if (dh) {
                value8(cur.dh[j], c, H, d);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) d[i] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = fmaf(cur.rs, fmaf(-n[j][i], c1, a[j][i]), d[i]);
            if (left > 0) store8(dx + t * H + c, left, d);
        }
    }
    float* out = partial + (int64_t)blockIdx.x * H;
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const int c = (j * TPR + in) * 8;
        if constexpr (ROWS > 1) {
            // the workgroup's rows, one after the other
            for (int w = 0; w < ROWS; ++w) {
                if (row == w) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) sums[in * 8 + i] = w ? sums[in * 8 + i] + dg[j][i] : dg[j][i];
                }
                __syncthreads();
            }
            if (row == 0 && H - c > 0) {
                float s[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) s[i] = sums[in * 8 + i];
                store8(out + c, H - c, s);
            }
            __syncthreads();
        } else if (H - c > 0) {
            store8(out + c, H - c, dg[j]);
        }
    }
}

// 16 columns a workgroup, 64 groups of partial rows
__global__ __launch_bounds__(1024) void rmsnorm_dgain_kernel(const float* __restrict__ partial, int parts, int H,
                                                             float* __restrict__ dgain) {
    __shared__ float red[16][16];
    const int col = threadIdx.x & 15, grp = threadIdx.x >> 4;
    const int c = blockIdx.x * 16 + col;
    float s = 0.0f;
    if (c < H) {
#pragma unroll 8
        for (int p = grp; p < parts; p += 64) s += gld(partial + (int64_t)p * H + c);
    }
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if ((threadIdx.x & 63) < 16) red[threadIdx.x >> 6][col] = s;
    __syncthreads();
    if (threadIdx.x < 16 && c < H) {
        s = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k) s += red[k][col];
        gst(dgain + c, s);
    }
}

namespace {
dim3 grid_of(int64_t threads) {
    const int64_t b = (threads + 255) / 256;
    return dim3((unsigned)(b < 65536 ? b : 65536));
}
}  // namespace

hipError_t launch_act_pack(bool bf16, const void* x, int64_t T, int H, int8_t* q, uint8_t* e, hipStream_t st) {
    if (T <= 0) return hipSuccess;
    const dim3 grid = grid_of((T * ((H + kActBlock - 1) / kActBlock) * 4 + kGroups - 1) / kGroups);
#define SC_PACK(E_, ENDS_) \
    hipLaunchKernelGGL((act_pack_kernel<E_, ENDS_>), grid, dim3(256), 0, st, (const E_*)x, T, H, q, e);
    SC_BY_ENDS(bf16, H, SC_PACK)
#undef SC_PACK
    return hipGetLastError();
}

static hipError_t unpack_rows(bool bf16, const int8_t* q, const uint8_t* e, int64_t T, int H, int64_t ld, void* x,
                              hipStream_t st) {
    if (T <= 0) return hipSuccess;
    const dim3 grid = grid_of((T * ((ld + 7) / 8) + kGroups - 1) / kGroups);
#define SC_UNPACK(E_, ENDS_) \
    hipLaunchKernelGGL((act_unpack_kernel<E_, ENDS_>), grid, dim3(256), 0, st, q, e, T, H, ld, (E_*)x);
    SC_BY_ENDS(bf16, H, SC_UNPACK)
#undef SC_UNPACK
    return hipGetLastError();
}

hipError_t launch_act_unpack(bool bf16, const int8_t* q, const uint8_t* e, int64_t T, int H, void* x,
                             hipStream_t st) {
    return unpack_rows(bf16, q, e, T, H, H, x, st);
}

// Threads and groups of 8 a row: a wave up to 1024 elements, a workgroup beyond.
template <typename E, int ENDS, int TPR, int C, typename... A>
static void norm_rows(int64_t T, hipStream_t st, A... args) {
    constexpr int64_t rows = TPR > 256 ? 1 : 256 / TPR;
    const int64_t b = (T + rows - 1) / rows;
    hipLaunchKernelGGL((rmsnorm_kernel<E, ENDS, TPR, C>), dim3((unsigned)(b < 1 << 20 ? b : 1 << 20)),
                       dim3(TPR > 256 ? TPR : 256), 0, st, args...);
}
template <typename E, int ENDS, typename... A>
static void norm_ends(int64_t T, int H, hipStream_t st, A... args) {
    if (ENDS == ROW_SHORT || H <= 512) norm_rows<E, ENDS, 64, 1>(T, st, args...);
    else if constexpr (ENDS != ROW_SHORT) {
        if (H <= 1024) norm_rows<E, ENDS, 64, 2>(T, st, args...);
        else if (H <= 2048) norm_rows<E, ENDS, 256, 1>(T, st, args...);
        else if (H <= 4096) norm_rows<E, ENDS, 256, 2>(T, st, args...);
        else if (H <= 6144) norm_rows<E, ENDS, 256, 3>(T, st, args...);
        else if (H <= 8192) norm_rows<E, ENDS, 256, 4>(T, st, args...);
        else norm_rows<E, ENDS, 1024, 2>(T, st, args...);
    }
}

hipError_t launch_rmsnorm(bool bf16, const void* x, const void* residual, const void* gain, float eps, int64_t T,
                          int H, void* h, void* y, float* rstd, int8_t* q, uint8_t* e, hipStream_t st) {
    if (T <= 0) return hipSuccess;
#define SC_NORM(E_, ENDS_)                                                                                     \
    norm_ends<E_, ENDS_>(T, H, st, (const E_*)x, (const E_*)residual, (const E_*)gain, eps, T, H, (E_*)h, (E_*)y, \
                         rstd, q, e);
    SC_BY_ENDS(bf16, H, SC_NORM)
#undef SC_NORM
    return hipGetLastError();
}

// Partial rows of dgain, a workgroup's each: 1024, fewer where a row takes more registers
// (two workgroups of 4 waves run on a CU, or one of 16).
int64_t rmsnorm_grad_parts(int64_t T, int H) {
    const int64_t wgs = H <= 1024 ? (T + 3) / 4 : T, most = H <= 4096 ? 1024 : H <= 8192 ? 512 : 256;
    return wgs < most ? wgs : most;
}

template <typename E, int ENDS, int TPR, int C, typename... A>
static void grad_rows(int parts, hipStream_t st, A... args) {
    hipLaunchKernelGGL((rmsnorm_grad_kernel<E, ENDS, TPR, C>), dim3((unsigned)parts), dim3(TPR > 256 ? TPR : 256), 0,
                       st, args...);
}
template <typename E, int ENDS, typename... A>
static void grad_ends(int parts, int H, hipStream_t st, A... args) {
    if (ENDS == ROW_SHORT || H <= 512) grad_rows<E, ENDS, 64, 1>(parts, st, args...);
    else if constexpr (ENDS != ROW_SHORT) {
        if (H <= 1024) grad_rows<E, ENDS, 64, 2>(parts, st, args...);
        else if (H <= 2048) grad_rows<E, ENDS, 256, 1>(parts, st, args...);
        else if (H <= 4096) grad_rows<E, ENDS, 256, 2>(parts, st, args...);
        else if (H <= 6144) grad_rows<E, ENDS, 256, 3>(parts, st, args...);
        else if (H <= 8192) grad_rows<E, ENDS, 256, 4>(parts, st, args...);
        else grad_rows<E, ENDS, 1024, 2>(parts, st, args...);
    }
}

hipError_t launch_rmsnorm_grad(bool bf16, const void* dy, const void* gain, const float* rstd, const int8_t* q,
                               const uint8_t* e, const void* dh, int64_t T, int H, void* dx, float* dgain,
                               float* partial, hipStream_t st) {
    const int parts = (int)rmsnorm_grad_parts(T, H);
    if (T > 0) {
#define SC_GRAD(E_, ENDS_)                                                                                      \
    grad_ends<E_, ENDS_>(parts, H, st, (const E_*)dy, (const E_*)gain, rstd, q, e, (const E_*)dh, T, H, (E_*)dx, \
                         partial);
        SC_BY_ENDS(bf16, H, SC_GRAD)
#undef SC_GRAD
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    hipLaunchKernelGGL(rmsnorm_dgain_kernel, dim3((unsigned)((H + 15) / 16)), dim3(1024), 0, st, partial, parts, H,
                       dgain);
    return hipGetLastError();
}

// ---- weight gradient ---------------------------------------------------------------------
// The checkpoint is exact in bfloat16 (8 significant bits and a power of two), so it is one
// plane, and a float32 dy takes three products instead of six.

WgradPlan wgrad_plan(bool bf16, int64_t T, int64_t N, int64_t H) {
    WgradPlan p{};
    p.bf16 = bf16;
    p.T = T;
    p.N = N;
    p.H = H;
    p.planes = !bf16 || N % 8 != 0;
    p.Np = p.planes ? tp_pad(up(N, 64)) : N;
    p.Hp = tp_pad(up(H, 64));
    p.prod = tp_plan((int)N, (int)H, (int)T, bf16 ? 1 : 3, true);
    int64_t o = 0;
    auto take = [&](int64_t bytes) {
        const int64_t at = o;
        o += up(bytes, 256);
        return at;
    };
    p.o_n = take(2 * T * p.Hp);
    p.o_dy = p.planes ? take(2 * (bf16 ? 1 : 3) * T * p.Np) : 0;
    p.o_part = take(p.prod.part_bytes);
    p.bytes = o;
    return p;
}

hipError_t launch_act_wgrad(const WgradPlan& p, const void* dy, const int8_t* q, const uint8_t* e, const void* gain,
                            void* dW, void* workspace, hipStream_t st) {
    if (p.T == 0) return launch_zero(dW, p.N * p.H * (p.bf16 ? 2 : 4), st);
    char* ws = (char*)workspace;
    uint16_t* n = (uint16_t*)(ws + p.o_n);
    hipError_t err = unpack_rows(true, q, e, p.T, (int)p.H, p.Hp, n, st);
    if (err != hipSuccess) return err;
    const uint16_t* d = (const uint16_t*)dy;
    if (p.planes) {
        d = (uint16_t*)(ws + p.o_dy);
        if ((err = launch_to_planes(p.bf16, dy, p.T, p.N, (uint16_t*)d, p.Np, p.T * p.Np, nullptr, 0, st)) !=
            hipSuccess)
            return err;
    }
    TpArgs a;
    a.A = d;
    a.lda = p.Np;
    a.a_plane = p.T * p.Np;
    a.B = n;
    a.ldb = p.Hp;
    a.M = (int)p.N;
    a.N = (int)p.H;
    a.K = (int)p.T;
    a.nseg = p.bf16 ? 1 : 3;
    a.segs = p.bf16 ? 0 : 0x0 << 8 | 0x1 << 4 | 0x2;  // lo, mid, hi of dy
    a.C = dW;
    a.ldc = p.H;
    a.c_bf16 = p.bf16;
    a.gain = gain;
    a.gain_bf16 = p.bf16;
    a.part = (float*)(ws + p.o_part);
    return launch_tile_product(TPK_WEIGHTS, p.prod, a, TpSum{}, st);
}

}  // namespace scopt
