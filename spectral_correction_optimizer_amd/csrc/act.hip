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
// A wavefront owns a row of up to 2048 elements, a workgroup a longer one; the row stays in
// registers between the sum and the outputs.  Sums are float32 (the norm's over at most
// 16384 squares, spread over 64 or 256 lanes).
#include <cmath>

#include "rows.hpp"
#include "internal.hpp"
#include "train.hpp"

namespace scopt {

namespace {
int64_t up(int64_t n, int64_t a) { return (n + a - 1) / a * a; }

// sum over the TPR threads of a row; red: one float per wave
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    if constexpr (TPR > 64) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < TPR / 64; ++w) v += red[w];
    }
    return v;
}
}  // namespace

// Every group of 8 elements is a thread's; blocks of a row's end are cut, and the four
// threads of a block are neighbours in a wave.
template <typename E>
__global__ __launch_bounds__(256) void act_pack_kernel(const E* __restrict__ x, int64_t T, int H, int8_t* q,
                                                       uint8_t* e) {
    const int nb = (H + kActBlock - 1) / kActBlock;
    const int64_t groups = T * nb * 4;
    // whole blocks leave the loop together: groups and the stride are multiples of 4
    for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < groups; g += (int64_t)gridDim.x * 256) {
        const int64_t t = g / (nb * 4);
        const int in = (int)(g - t * (nb * 4)), c = in * 8, left = H - c;
        float v[8];
        load8(x + t * H + c, left, v);
        int8_t k[8];
        uint8_t ex;
        act_encode8(v, k, ex);
        store_q8(q + t * H + c, left, k);
        if ((in & 3) == 0) gst(e + t * nb + in / 4, ex);
    }
}

template <typename E>
__global__ __launch_bounds__(256) void act_unpack_kernel(const int8_t* __restrict__ q, const uint8_t* __restrict__ e,
                                                         int64_t T, int H, int64_t ld, E* x) {
    const int nb = (H + kActBlock - 1) / kActBlock, per_row = (int)((ld + 7) / 8);
    const int64_t groups = T * per_row;
    for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < groups; g += (int64_t)gridDim.x * 256) {
        const int64_t t = g / per_row;
        const int c = (int)(g - t * per_row) * 8, left = H - c;
        float v[8];
        if (left > 0) {
            load_q8(q + t * H + c, left, act_step(gld(e + t * nb + c / kActBlock)), v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.0f;
        }
        store8(x + t * ld + c, (int)(ld - c), v);  // bfloat16: exact, 8 significant bits
    }
}

template <typename E, int TPR, int C>
__global__ __launch_bounds__(256) void rmsnorm_kernel(const E* __restrict__ x, const E* __restrict__ res,
                                                      const E* __restrict__ gain, float eps, int64_t T, int H,
                                                      E* h, E* y, float* rstd, int8_t* q, uint8_t* e) {
    __shared__ float red[4];
    const int in = threadIdx.x % TPR;
    const int64_t t = (int64_t)blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
    if (t >= T) return;  // a whole wave, or (TPR 256) no row
    const int nb = (H + kActBlock - 1) / kActBlock;
    float v[C][8];
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const int c = (j * TPR + in) * 8;
        load8(x + t * H + c, H - c, v[j]);
    }
    if (res) {
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c = (j * TPR + in) * 8;
            float r[8];
            load8(res + t * H + c, H - c, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] += r[i];
        }
    }
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(v[j][i], v[j][i], ss);
    ss = row_sum<TPR>(ss, red);
    const float rs = 1.0f / sqrtf(ss / (float)H + eps);
    if (in == 0) gst(rstd + t, rs);
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const int c = (j * TPR + in) * 8, left = H - c;
        if (h && left > 0) store8(h + t * H + c, left, v[j]);
        float g[8], o[8];
        if (left > 0) load8(gain + c, left, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[j][i] *= rs;  // the norm of the float32 sum, not of the rounded h
            o[i] = left > 0 ? v[j][i] * g[i] : 0.0f;
        }
        if (left > 0) store8(y + t * H + c, left, o);
        if (q) {
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

// Rows are dealt to the workgroups in turn; each keeps its rows' sum of dy n in registers and
// writes one row of `partial`, summed in a fixed order by rmsnorm_dgain_kernel.
template <typename E, int TPR, int C>
__global__ __launch_bounds__(256) void rmsnorm_grad_kernel(const E* __restrict__ dy, const E* __restrict__ gain,
                                                           const float* __restrict__ rstd,
                                                           const int8_t* __restrict__ q,
                                                           const uint8_t* __restrict__ e, const E* __restrict__ dh,
                                                           int64_t T, int H, E* dx, float* partial) {
    constexpr int ROWS = 256 / TPR;
    __shared__ float red[4];
    __shared__ float sums[ROWS > 1 ? TPR * 8 : 1];
    const int in = threadIdx.x % TPR, row = threadIdx.x / TPR;
    const int nb = (H + kActBlock - 1) / kActBlock;
    float g[C][8], dg[C][8];
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const int c = (j * TPR + in) * 8;
        load8(gain + c, H - c, g[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) dg[j][i] = 0.0f;
    }
    for (int64_t t = (int64_t)blockIdx.x * ROWS + row; t < T; t += (int64_t)gridDim.x * ROWS) {
        float a[C][8], n[C][8];
        const float rs = gld(rstd + t);
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c = (j * TPR + in) * 8, left = H - c;
            load8(dy + t * H + c, left, a[j]);
            load_q8(q + t * H + c, left, left > 0 ? act_step(gld(e + t * nb + c / kActBlock)) : 0.0f, n[j]);
        }
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dg[j][i] = fmaf(a[j][i], n[j][i], dg[j][i]);
                a[j][i] *= g[j][i];
                dot = fmaf(a[j][i], n[j][i], dot);
            }
        const float c1 = row_sum<TPR>(dot, red) / (float)H;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c = (j * TPR + in) * 8, left = H - c;
            if (left <= 0) continue;
            float d[8];
            if (dh) {
                load8(dh + t * H + c, left, d);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) d[i] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = fmaf(rs, fmaf(-n[j][i], c1, a[j][i]), d[i]);
            store8(dx + t * H + c, left, d);
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

// 64 columns a workgroup, 16 groups of partial rows
__global__ __launch_bounds__(1024) void rmsnorm_dgain_kernel(const float* __restrict__ partial, int parts, int H,
                                                             float* __restrict__ dgain) {
    __shared__ float red[16][64];
    const int lane = threadIdx.x & 63, grp = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + lane;
    float s = 0.0f;
    if (c < H)
        for (int p = grp; p < parts; p += 16) s += gld(partial + (int64_t)p * H + c);
    red[grp][lane] = s;
    __syncthreads();
    if (grp == 0 && c < H) {
        for (int k = 1; k < 16; ++k) s += red[k][lane];
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
    const dim3 grid = grid_of(T * ((H + kActBlock - 1) / kActBlock) * 4);
    if (bf16)
        hipLaunchKernelGGL(act_pack_kernel<uint16_t>, grid, dim3(256), 0, st, (const uint16_t*)x, T, H, q, e);
    else
        hipLaunchKernelGGL(act_pack_kernel<float>, grid, dim3(256), 0, st, (const float*)x, T, H, q, e);
    return hipGetLastError();
}

static hipError_t unpack_rows(bool bf16, const int8_t* q, const uint8_t* e, int64_t T, int H, int64_t ld, void* x,
                              hipStream_t st) {
    if (T <= 0) return hipSuccess;
    const dim3 grid = grid_of(T * ((ld + 7) / 8));
    if (bf16)
        hipLaunchKernelGGL(act_unpack_kernel<uint16_t>, grid, dim3(256), 0, st, q, e, T, H, ld, (uint16_t*)x);
    else
        hipLaunchKernelGGL(act_unpack_kernel<float>, grid, dim3(256), 0, st, q, e, T, H, ld, (float*)x);
    return hipGetLastError();
}

hipError_t launch_act_unpack(bool bf16, const int8_t* q, const uint8_t* e, int64_t T, int H, void* x,
                             hipStream_t st) {
    return unpack_rows(bf16, q, e, T, H, H, x, st);
}

// thread layout of a row: TPR threads, C groups of 8 elements each
#define SC_ROW_LAYOUTS(X)                                             \
    if (H <= 512) { X(64, 1) } else if (H <= 1024) { X(64, 2) }       \
    else if (H <= 2048) { X(64, 4) } else if (H <= 4096) { X(256, 2) } \
    else if (H <= 8192) { X(256, 4) } else { X(256, 8) }

hipError_t launch_rmsnorm(bool bf16, const void* x, const void* residual, const void* gain, float eps, int64_t T,
                          int H, void* h, void* y, float* rstd, int8_t* q, uint8_t* e, hipStream_t st) {
    if (T <= 0) return hipSuccess;
#define SC_NORM_E(TPR_, C_, E_)                                                                              \
    hipLaunchKernelGGL((rmsnorm_kernel<E_, TPR_, C_>), dim3((unsigned)((T + 256 / TPR_ - 1) / (256 / TPR_))), \
                       dim3(256), 0, st, (const E_*)x, (const E_*)residual, (const E_*)gain, eps, T, H, (E_*)h, \
                       (E_*)y, rstd, q, e);
#define SC_NORM(TPR_, C_)                          \
    if (bf16) { SC_NORM_E(TPR_, C_, uint16_t) }    \
    else { SC_NORM_E(TPR_, C_, float) }
    SC_ROW_LAYOUTS(SC_NORM)
#undef SC_NORM
#undef SC_NORM_E
    return hipGetLastError();
}

int64_t rmsnorm_grad_parts(int64_t T, int H) {
    const int64_t wgs = H <= 2048 ? (T + 3) / 4 : T;
    return wgs < 1024 ? wgs : 1024;
}

hipError_t launch_rmsnorm_grad(bool bf16, const void* dy, const void* gain, const float* rstd, const int8_t* q,
                               const uint8_t* e, const void* dh, int64_t T, int H, void* dx, float* dgain,
                               float* partial, hipStream_t st) {
    const int parts = (int)rmsnorm_grad_parts(T, H);
    if (T > 0) {
#define SC_GRAD_E(TPR_, C_, E_)                                                                                 \
    hipLaunchKernelGGL((rmsnorm_grad_kernel<E_, TPR_, C_>), dim3((unsigned)parts), dim3(256), 0, st,            \
                       (const E_*)dy, (const E_*)gain, rstd, q, e, (const E_*)dh, T, H, (E_*)dx, partial);
#define SC_GRAD(TPR_, C_)                          \
    if (bf16) { SC_GRAD_E(TPR_, C_, uint16_t) }    \
    else { SC_GRAD_E(TPR_, C_, float) }
        SC_ROW_LAYOUTS(SC_GRAD)
#undef SC_GRAD
#undef SC_GRAD_E
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    hipLaunchKernelGGL(rmsnorm_dgain_kernel, dim3((unsigned)((H + 63) / 64)), dim3(1024), 0, st, partial, parts, H,
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
    p.Np = p.planes ? up(N, 64) : N;
    p.Hp = up(H, 64);
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
