// The tiled products of the training-step operators: instances of the kernel of
// tile_product.hpp, the choice of tile and split, the sum over splits, and the copies of
// operands into bfloat16 planes.
#include "rows.hpp"
#include "tile_product.hpp"

namespace scopt {

namespace {
constexpr int kCus = 256;
using Big = TpShape<256, 256, 2, 4, 2, 1>;   // 128 KB of LDS: one workgroup of 8 waves per CU
using Mid = TpShape<128, 128, 2, 2, 2, 2>;   // 64 KB: two workgroups of 4 waves per CU
using Small = TpShape<64, 128, 1, 4, 3, 2>;  // 72 KB: two workgroups of 4 waves per CU
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
    const int64_t groups = (int64_t)P.M * ((P.N + 3) / 4);
    const float alpha = P.alpha ? gld(P.alpha) : 1.0f;
    for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < groups; g += (int64_t)gridDim.x * 256) {
        const int64_t m = g / ((P.N + 3) / 4);
        const int n = (int)(g - m * ((P.N + 3) / 4)) * 4;
        const int left = P.N - n;
        const int64_t at = m * P.N + n, stride = (int64_t)P.M * P.N;
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
            tp_store(P.C, P.c_bf16, m * P.ldc + n, v, left);
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
TpPlan tp_plan(int M, int N, int K, int nseg, bool may_split) {
    struct Shape {
        int bm, bn, per_cu, turn;
        double step, tile;
    };
    static const Shape shapes[3] = {
        {256, 256, 1, 2, 1.70, 12.0}, {128, 128, 2, 2, 1.20, 3.7}, {64, 128, 2, 3, 0.81, 1.2}};
    TpPlan best;
    double best_us = 1e300;
    for (int s = 0; s < 3; ++s) {
        const Shape& S = shapes[s];
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

namespace {
template <class S>
hipError_t launch_shape(TpKind kind, const TpArgs& P, bool part, hipStream_t st) {
    const int all = P.tiles_m * P.tiles_n * P.splits, most = kCus * S::PER_CU;
    const dim3 grid((unsigned)(all < most ? all : most)), blk(S::NT);
    switch (kind) {
        case TPK_LOGIT_STATS:
            hipLaunchKernelGGL((tile_product_kernel<S, true, true, TP_STATS>), grid, blk, 0, st, P);
            break;
        case TPK_LOGIT_GRAD:
            hipLaunchKernelGGL((tile_product_kernel<S, true, true, TP_GRAD>), grid, blk, 0, st, P);
            break;
        case TPK_STATES:
            if (part) hipLaunchKernelGGL((tile_product_kernel<S, true, false, TP_PART>), grid, blk, 0, st, P);
            else hipLaunchKernelGGL((tile_product_kernel<S, true, false, TP_STORE>), grid, blk, 0, st, P);
            break;
        case TPK_WEIGHTS:
            if (part) hipLaunchKernelGGL((tile_product_kernel<S, false, false, TP_PART>), grid, blk, 0, st, P);
            else hipLaunchKernelGGL((tile_product_kernel<S, false, false, TP_STORE>), grid, blk, 0, st, P);
            break;
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
    const bool part = (kind == TPK_STATES || kind == TPK_WEIGHTS) && (plan.splits > 1 || sum.acc || sum.out_acc);
    hipError_t e = plan.shape == 0   ? launch_shape<Big>(kind, P, part, st)
                   : plan.shape == 1 ? launch_shape<Mid>(kind, P, part, st)
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

// The exact split of any float32 values (split8 rounds the first part, which overflows from
// 0x1.FFp127 on and leaves infinity - infinity): the first part stays at bfloat16's largest value, and
// an infinity is its own first part, beside zeros.
__device__ __forceinline__ Split8 split8_any(const float (&f)[8]) {
    constexpr float most = 0x1.FEp127f;
    v4u h, m, l;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float first[2], rest[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float x = f[2 * i + u], a = fabsf(x);
            first[u] = a >= 0x1.FFp127f && a < __builtin_huge_valf() ? copysignf(most, x) : x;
        }
        h[i] = pack_bf16x2(first[0], first[1]);
        rest[0] = f[2 * i] - bf16_lo(h[i]);
        rest[1] = f[2 * i + 1] - bf16_hi(h[i]);
#pragma unroll
        for (int u = 0; u < 2; ++u) rest[u] = fabsf(f[2 * i + u]) == __builtin_huge_valf() ? 0.0f : rest[u];
        m[i] = pack_bf16x2(rest[0], rest[1]);
        l[i] = pack_bf16x2(rest[0] - bf16_lo(m[i]), rest[1] - bf16_hi(m[i]));
    }
    return Split8{__builtin_bit_cast(v8bf, h), __builtin_bit_cast(v8bf, m), __builtin_bit_cast(v8bf, l)};
}

// planes[p][r][c]: kGroups groups of eight columns a thread (ld is a multiple of 8)
template <typename E, int ENDS>
__global__ __launch_bounds__(256) void to_planes_kernel(const E* __restrict__ src, int64_t rows, int cols,
                                                        uint16_t* __restrict__ dst, int64_t ld, int64_t plane,
                                                        const int64_t* __restrict__ targets, int64_t vocab) {
    const int per_row = (int)(ld / 8);
    const int64_t n = rows * per_row;
    const bool small = n < (int64_t)1 << 31;
    for (int64_t g0 = (int64_t)blockIdx.x * 256 * kGroups + threadIdx.x; g0 < n;
         g0 += (int64_t)gridDim.x * 256 * kGroups) {
        Group8<E, ENDS> w[kGroups];
        int64_t r[kGroups], tgt[kGroups];
        int in[kGroups];
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            const int64_t g = g0 + k * 256;
            split_group(g < n ? g : n - 1, per_row, small, r[k], in[k]);
            w[k].load(src + r[k] * cols, in[k] * 8, cols);
            tgt[k] = targets ? gld(targets + r[k]) : 0;
        }
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            if (g0 + k * 256 >= n) break;
            uint16_t* o = dst + r[k] * ld + in[k] * 8;
            const bool live = tgt[k] >= 0 && tgt[k] < vocab;
            float f[8];
            value8(w[k], in[k] * 8, cols, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = live ? f[i] : 0.0f;
            if constexpr (sizeof(E) == 2) {
                store8(o, 8, f);  // exact
            } else {
                const Split8 s = split8_any(f);
                *(SC_GLOBAL v8bf*)o = s.h;
                *(SC_GLOBAL v8bf*)(o + plane) = s.m;
                *(SC_GLOBAL v8bf*)(o + 2 * plane) = s.l;
            }
        }
    }
}

hipError_t launch_to_planes(bool bf16, const void* src, int64_t rows, int64_t cols, uint16_t* dst, int64_t ld,
                            int64_t plane, const int64_t* targets, int64_t vocab, hipStream_t st) {
    const int64_t n = rows * (ld / 8);
    if (n <= 0) return hipSuccess;
    if (!targets) vocab = 1;  // every row counts
    const int64_t blocks = (n + 256 * kGroups - 1) / (256 * kGroups);
    const dim3 grid((unsigned)(blocks < 65536 ? blocks : 65536));
#define SC_PLANES(E_, ENDS_)                                                                                         \
    hipLaunchKernelGGL((to_planes_kernel<E_, ENDS_>), grid, dim3(256), 0, st, (const E_*)src, rows, (int)cols, dst, \
                       ld, plane, targets, vocab);
    SC_BY_ENDS(bf16, cols, SC_PLANES)
#undef SC_PLANES
    return hipGetLastError();
}

}  // namespace scopt
