// Tiled products on the bfloat16 matrix cores of gfx950 for the training-step
// operators (cross entropy, weight gradient):
//
//   acc[m][n] = sum over segments s, k of A_s(m, k) * B_s(n, k)
//
// with float32 accumulation.  An operand is a set of bfloat16 planes, stored either
// with k contiguous ([rows][K]) or with the rows contiguous ([K][rows]); a segment names
// one plane of each operand.  bfloat16 operands have one plane and one segment.  A float32
// operand is split exactly into three planes x = hi + mid + lo (common.hpp), and the six
// largest of the nine plane products (three when the other operand is exact in one plane)
// run through the same loop, smallest first, into the same accumulators: the parts left
// out are below 2^-23 of |a b|.
//
// A workgroup owns a BM x BN tile and advances 64 k at a time.  Both operand tiles go
// from memory straight into LDS (16 bytes per lane, no registers), NST buffers deep; each
// wave multiplies a (BM / WVM) x (BN / WVN) part in 16 x 16 x 32 blocks.  Each buffer is
// an array of its own and the loop is unrolled over them, so the reads of one buffer do
// not wait for the loads that fill another.
//
// LDS layouts (16-byte slots permuted within a row by choosing which global chunk each
// lane fetches, so that the matrix operand reads touch every bank once):
//   k contiguous:    [row][64 k], slot = chunk ^ (row & 7) ^ ((row >> 3) & 1); a
//                    fragment is one 16-byte read per lane.
//   rows contiguous: [k][rows], 32-byte blocks, block ^= (k & 3) | ((k >> 3) & 1) << 2;
//                    a fragment is two transposing reads (ds_read_b64_tr_b16: 16 lanes
//                    read four k rows of 16 elements, each lane receives the four k of
//                    one row).
// Bounds: every load goes through a buffer resource that ends at the operand's end, and a
// lane whose chunk lies beyond the operand's rows (or k) gets an offset beyond it: such
// lanes deliver zeros.
#pragma once

#include <type_traits>

#include "common.hpp"
#include "internal.hpp"
#include "train.hpp"

namespace scopt {

typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));

#define SC_LDS __attribute__((address_space(3)))
#define SC_INLINE __attribute__((always_inline))

constexpr uint32_t kTpMaxBytes = 0x7fffffffu;  // largest buffer range (offsets stay below 2^31)
constexpr uint32_t kTpBeyond = 0x80000000u;    // an offset beyond every range

// Loader of one operand's R x 64 tile: offsets are set up once, the base advances.
template <int R, int NT, bool KC>
struct TpLoader {
    static constexpr int NL = R * 8 / NT;  // 16-byte loads per thread and tile
    uint32_t voff[NL];
    int kchunk;  // KC: the k of this lane's chunk within a tile
    __device__ __forceinline__ void init(int64_t ld, int rows, int r0) {
        const int t = threadIdx.x;
        if constexpr (KC) {
            const int r = t >> 3, slot = t & 7;
            const int c = slot ^ (r & 7) ^ ((r >> 3) & 1);
            kchunk = c * 8;
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const int row = r + i * (NT / 8);
                voff[i] = r0 + row < rows ? (uint32_t)(row * ld + c * 8) * 2u : kTpBeyond;
            }
        } else {
            constexpr int CR = R / 8;  // chunks per k row
            kchunk = 0;
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const int k = t / CR + i * (NT / CR), slot = t % CR;
                const int c = slot ^ swz(k) * 2;
                voff[i] = r0 + c * 8 < rows ? (uint32_t)(k * ld + c * 8) * 2u : kTpBeyond;
            }
        }
    }
    static __device__ __forceinline__ int swz(int k) {
        constexpr int MASK = R >= 128 ? 7 : R / 16 - 1;
        return ((k & 3) | (((k >> 3) & 1) << 2)) & MASK;
    }
    // fetch the tile at k0 of a plane into lds; live = false fetches nothing (zeros)
    __device__ __forceinline__ void fetch(const uint16_t* p, int64_t ld, int rows, int K, int r0, int k0,
                                          bool live, uint16_t* lds) const {
        // a row of k ends at a whole chunk (what lies between is zero or meets zeros), and so
        // does a row of rows (the sums of what lies beyond are not stored)
        if (KC) K = (K + 7) & ~7;
        else rows = (rows + 7) & ~7;
        const int64_t first = KC ? (int64_t)r0 * ld + k0 : (int64_t)k0 * ld + r0;
        const int64_t total = KC ? (int64_t)(rows - 1) * ld + K : (int64_t)(K - 1) * ld + rows;
        int64_t bytes = (total - first) * 2;
        bytes = bytes < (int64_t)kTpMaxBytes ? bytes : (int64_t)kTpMaxBytes;
        const __amdgpu_buffer_rsrc_t rs = buf_rsrc(p + first, live && bytes > 0 ? (uint32_t)bytes : 0u);
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            uint32_t v = voff[i];
            if (KC) v = k0 + kchunk < K ? v : kTpBeyond;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (SC_LDS void*)(lds + i * NT * 8 + wave * 512), 16, v, 0,
                                                     0, 0);
        }
    }
};

// Fragment reader of NB 16-row blocks starting at row w0 of a tile (w0 / 16 is a multiple of
// NB, a power of two: a block's offset differs from the first one's by an exclusive or).
template <int R, int NB, bool KC>
struct TpReader {
    int off;
    __device__ __forceinline__ void init(int w0) {
        const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
        if constexpr (KC) {
            const int f = (j & 7) ^ ((j >> 3) & 1);
            off = (w0 + j) * 64 + ((g ^ f) << 3);
        } else {
            const int k = g * 8 + (j >> 2);
            off = k * R + (((w0 / 16) ^ TpLoader<R, 64, false>::swz(k)) << 4) + (j & 3) * 4;
        }
    }
    // The offsets are formed anew where this is called: kept in registers over the loop they
    // would not fit beside the sums.
    __device__ __forceinline__ void renew() { asm volatile("" : "+v"(off)); }
    // the 8 k values (kk * 32 + 8 * (lane / 16) ..) of row w0 + 16 b + lane % 16
    __device__ __forceinline__ v8bf read(const uint16_t* lds, int kk, int b) const {
        if constexpr (KC) {
            return *(const v8bf*)(lds + (off ^ kk << 5) + b * 16 * 64);
        } else {
            const uint16_t* p = lds + (off ^ b << 4) + kk * 32 * R;
            const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((SC_LDS v4s*)p);
            const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((SC_LDS v4s*)(p + 4 * R));
            return __builtin_bit_cast(v8bf, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
    }
};

// ---- epilogue pieces -------------------------------------------------------------------

__device__ __forceinline__ float tp_gain(const TpArgs& P, int n) {
    if (!P.gain) return 1.0f;
    return P.gain_bf16 ? Elem<uint16_t>::load((const uint16_t*)P.gain, n) : gld((const float*)P.gain + n);
}
// four consecutive elements at `at`, the first `left` of them inside the row
__device__ __forceinline__ void tp_store(void* base, int bf16, int64_t at, const float (&v)[4], int left, bool vec) {
    if (bf16) {
        uint16_t* p = (uint16_t*)base + at;
        if (vec) {
            *(SC_GLOBAL v2u*)p = v2u{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (r < left) gst(p + r, f32_to_bf16(v[r]));
        }
    } else {
        float* p = (float*)base + at;
        if (vec) {
            gst4(p, v4f{v[0], v[1], v[2], v[3]});
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (r < left) gst(p + r, v[r]);
        }
    }
}
// four dlogits as one bfloat16 plane, or as the three planes of their float32 values
__device__ __forceinline__ void tp_store_planes(uint16_t* base, int planes, int64_t plane, int64_t at,
                                                const float (&v)[4]) {
    v2u h = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    *(SC_GLOBAL v2u*)(base + at) = h;
    if (planes == 3) {
        const float r0 = v[0] - bf16_lo(h[0]), r1 = v[1] - bf16_hi(h[0]);
        const float r2 = v[2] - bf16_lo(h[1]), r3 = v[3] - bf16_hi(h[1]);
        const v2u m = {pack_bf16x2(r0, r1), pack_bf16x2(r2, r3)};
        const v2u l = {pack_bf16x2(r0 - bf16_lo(m[0]), r1 - bf16_hi(m[0])),
                       pack_bf16x2(r2 - bf16_lo(m[1]), r3 - bf16_hi(m[1]))};
        *(SC_GLOBAL v2u*)(base + plane + at) = m;
        *(SC_GLOBAL v2u*)(base + 2 * plane + at) = l;
    }
}
// the target of a row; -1 where it is no row of the vocabulary
__device__ __forceinline__ int64_t tp_target(const int64_t* targets, int64_t vocab, int64_t m) {
    const int64_t t = gld(targets + m);
    return t >= 0 && t < vocab ? t : -1;
}
constexpr float kLog2e = 1.44269504088896340736f;
// The reference of a tile's exponentials.  TP_KEEP_EXP: the row maximum in powers of two,
// rounded up; otherwise the maximum itself.  A tile whose row is all -infinity takes 0, so
// that its exponentials are 0 and not NaN.
__device__ __forceinline__ float tp_reference(float mx, bool pow2) {
    if (mx == -__builtin_huge_valf()) return 0.0f;
    return pow2 ? ceilf(mx * kLog2e) : mx;
}

// What becomes of a tile's sums.
enum TpEpi {
    TP_STORE = 0,   // C = acc * alpha * gain[n], bfloat16 or float32
    TP_PART = 1,    // float32 sums of one split of k, [split][M][N]
    TP_STATS = 2,   // row maxima and exp sums of the tile; logits kept as P.keep says
    TP_GRAD = 3,    // exp(acc - lse[m]) - [n is m's target], as bfloat16 planes
};

template <int BM_, int BN_, int WVM_, int WVN_, int NST_, int PER_CU_>
struct TpShape {
    static constexpr int BM = BM_, BN = BN_, WVM = WVM_, WVN = WVN_, NST = NST_, PER_CU = PER_CU_;
    static constexpr int NT = 64 * WVM * WVN;
    static constexpr int WAVES = WVM * WVN * PER_CU / 4;  // per SIMD
};

// Tile of a workgroup: every XCD gets a contiguous range of ids, and consecutive ids walk
// groups of 8 row tiles with the rows fastest, so the tiles that run together on an XCD
// form a block of 8 x 4 tiles and share their panels in its L2.
__device__ __forceinline__ void tp_tile(int id, int tiles_m, int tiles_n, int& tm, int& tn) {
    constexpr int GM = 8;
    const int group = id / (GM * tiles_n);
    const int m_first = group * GM;
    const int gm = tiles_m - m_first < GM ? tiles_m - m_first : GM;
    const int in = id - group * GM * tiles_n;
    tm = m_first + in % gm;
    tn = in / gm;
}

template <class S, bool AKC, bool BKC, int EPI>
__global__ __launch_bounds__(S::NT, S::WAVES) void tile_product_kernel(const TpArgs P) {
    constexpr int BM = S::BM, BN = S::BN, NT = S::NT, NST = S::NST;
    constexpr int WM = BM / S::WVM, WN = BN / S::WVN, MI = WM / 16, NI = WN / 16;
    using LA = TpLoader<BM, NT, AKC>;
    using LB = TpLoader<BN, NT, BKC>;
    constexpr int ASZ = BM * 64, BSZ = BN * 64;
    __shared__ __align__(1024) uint16_t a0[ASZ], b0[BSZ], a1[ASZ], b1[BSZ];
    __shared__ __align__(1024) uint16_t a2[NST > 2 ? ASZ : 8], b2[NST > 2 ? BSZ : 8];
    __shared__ __align__(1024) uint16_t a3[NST > 3 ? ASZ : 8], b3[NST > 3 ? BSZ : 8];

    const int tiles = P.tiles_m * P.tiles_n;
    const int id = xcd_remap(blockIdx.x, gridDim.x);
    const int split = id / tiles;
    int tm, tn;
    tp_tile(id - split * tiles, P.tiles_m, P.tiles_n, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = (wave / S::WVN) * WM, wn = (wave % S::WVN) * WN;

    LA la;
    LB lb;
    la.init(P.lda, P.M, m0);
    lb.init(P.ldb, P.N, n0);
    TpReader<BM, MI, AKC> ra;
    TpReader<BN, NI, BKC> rb;
    ra.init(wm);
    rb.init(wn);

    v4f acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

    const int ksteps = (P.K + 63) / 64, total = ksteps * P.nseg;
    const int per = (total + P.splits - 1) / P.splits;
    const int first = split * per, last = min(total, first + per);

    // the step that is fetched next: its segment and k
    int seg = first / ksteps, kst = first - seg * ksteps, fetched = first;
    auto fetch = [&](uint16_t* as, uint16_t* bs) SC_INLINE {
        const bool live = fetched < last;
        const uint32_t planes = live ? (uint32_t)(P.segs >> (4 * seg)) : 0;
        la.fetch(P.A + (planes & 3) * P.a_plane, P.lda, P.M, P.K, m0, kst * 64, live, as);
        lb.fetch(P.B + ((planes >> 2) & 3) * P.b_plane, P.ldb, P.N, P.K, n0, kst * 64, live, bs);
        ++fetched;
        if (++kst == ksteps) {
            kst = 0;
            ++seg;
        }
    };
    // fragments of one 32-deep half of a step, and their products
    struct Frags {
        v8bf a[MI], b[NI];
    };
    auto read = [&](const uint16_t* as, const uint16_t* bs, int kk, Frags& f) SC_INLINE {
        ra.renew();
        rb.renew();
#pragma unroll
        for (int j = 0; j < NI; ++j) f.b[j] = rb.read(bs, kk, j);
#pragma unroll
        for (int i = 0; i < MI; ++i) f.a[i] = ra.read(as, kk, i);
    };
    auto multiply = [&](const Frags& f) SC_INLINE {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j)  // transposed: a lane's four sums are consecutive n
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.b[j], f.a[i], acc[i][j], 0, 0, 0);
    };
    // one half's products with the next half's reads spread between them
    auto interleave = [&]() SC_INLINE {
        constexpr int READS = (AKC ? MI : 2 * MI) + (BKC ? NI : 2 * NI), PRODS = MI * NI;
#pragma unroll
        for (int r = 0; r < READS; ++r) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // an LDS read
            __builtin_amdgcn_sched_group_barrier(0x008, PRODS / READS, 0);
        }
        if constexpr (PRODS % READS) __builtin_amdgcn_sched_group_barrier(0x008, PRODS % READS, 0);
    };
    // every step issues the same number of loads (the ones past the end fetch nothing)
    constexpr int PER = LA::NL + LB::NL;
    Frags f0, f1;
    // On entry the first half of this step's fragments is in f0 (or on its way).
    auto step = [&](uint16_t* as, uint16_t* bs, const uint16_t* an, const uint16_t* bn) SC_INLINE {
        read(as, bs, 1, f1);
        multiply(f0);
        interleave();
        // this wave's loads of the next step have landed and its reads of this step's buffer
        // are done; after the barrier that holds for every wave
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(PER * (NST - 2)) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        fetch(as, bs);
        __builtin_amdgcn_sched_barrier(0);  // the loads go out before the products
        read(an, bn, 0, f0);
        multiply(f1);
        interleave();
        __builtin_amdgcn_sched_barrier(0);
    };
    fetch(a0, b0);
    fetch(a1, b1);
    if constexpr (NST > 2) fetch(a2, b2);
    if constexpr (NST > 3) fetch(a3, b3);
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(PER * (NST - 1)) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    read(a0, b0, 0, f0);
    // whole turns of the buffers: the steps past the end multiply zeros
    for (int s = first; s < last; s += NST) {
        if constexpr (NST == 2) {
            step(a0, b0, a1, b1);
            step(a1, b1, a0, b0);
        } else if constexpr (NST == 3) {
            step(a0, b0, a1, b1);
            step(a1, b1, a2, b2);
            step(a2, b2, a0, b0);
        } else {
            step(a0, b0, a1, b1);
            step(a1, b1, a2, b2);
            step(a2, b2, a3, b3);
            step(a3, b3, a0, b0);
        }
    }
    // loads past the end may still be on their way into LDS
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");

    // Lane l holds, of block (i, j): row m = wm + 16 i + l % 16, columns
    // n = wn + 16 j + 4 (l / 16) + 0..3.
    const int lm = m0 + wm + (lane & 15), ln = n0 + wn + 4 * (lane >> 4);
    const int M = P.M, N = P.N;
    if constexpr (EPI == TP_STORE) {
        const float alpha = P.alpha ? gld(P.alpha) : 1.0f;
        auto store = [&](auto bf16, auto vec) SC_INLINE {
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                const int n = ln + 16 * j;
                float g[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) g[r] = alpha * tp_gain(P, min(n + r, N - 1));
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    const int m = lm + 16 * i;
                    const float v[4] = {acc[i][j][0] * g[0], acc[i][j][1] * g[1], acc[i][j][2] * g[2],
                                        acc[i][j][3] * g[3]};
                    if (m < M && n < N)
                        tp_store(P.C, decltype(bf16)::value, (int64_t)m * P.ldc + n, v, N - n, decltype(vec)::value);
                }
            }
        };
        using T = std::true_type;
        using F = std::false_type;
        if (P.c_bf16) {
            if (P.c_vec) store(T{}, T{});
            else store(T{}, F{});
        } else {
            if (P.c_vec) store(F{}, T{});
            else store(F{}, F{});
        }
    } else if constexpr (EPI == TP_PART) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                const int m = lm + 16 * i, n = ln + 16 * j;
                if (m >= M || n >= N) continue;
                const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                tp_store(P.part, 0, ((int64_t)split * M + m) * N + n, v, N - n, (N & 3) == 0);
            }
    } else if constexpr (EPI == TP_STATS) {
        // row maximum over the tile's columns: registers, the four lanes of a row, the
        // waves beside each other
        float* red = (float*)a0;  // [WVN][BM]
        __syncthreads();
        float mx[MI], sum[MI];
        const bool pow2 = P.keep == TP_KEEP_EXP;
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            float v = -__builtin_huge_valf();
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (ln + 16 * j + r < N) v = fmaxf(v, acc[i][j][r]);
            v = fmaxf(v, __shfl_xor(v, 16));
            v = fmaxf(v, __shfl_xor(v, 32));
            if (lane < 16) red[(wave % S::WVN) * BM + wm + 16 * i + lane] = v;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            float v = red[wm + 16 * i + (lane & 15)];
#pragma unroll
            for (int w = 1; w < S::WVN; ++w) v = fmaxf(v, red[w * BM + wm + 16 * i + (lane & 15)]);
            mx[i] = v;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int m = lm + 16 * i;
            const int64_t tgt = m < M ? tp_target(P.targets, P.vocab, m) - P.n_first : -1;
            const float ref = tp_reference(mx[i], pow2);
            float z = 0.0f;
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                const int n = ln + 16 * j;
                float e[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float s = acc[i][j][r];
                    e[r] = n + r < N ? (pow2 ? __builtin_amdgcn_exp2f(fmaf(s, kLog2e, -ref)) : expf(s - ref)) : 0.0f;
                    z += e[r];
                    if (m < M && n + r < N && n + r == tgt) gst(P.target_logit + m, s);
                }
                if (m < M && n < P.ldp) {
                    if (P.keep == TP_KEEP_EXP)
                        tp_store(P.P, 1, (int64_t)m * P.ldp + n, e, 4, true);
                    else if (P.keep == TP_KEEP_LOGIT) {
                        const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                        tp_store(P.P, 0, (int64_t)m * P.ldp + n, v, 4, true);
                    }
                }
            }
            z += __shfl_xor(z, 16);
            z += __shfl_xor(z, 32);
            sum[i] = z;
            if (lane < 16) red[(wave % S::WVN) * BM + wm + 16 * i + lane] = z;
        }
        __syncthreads();
        if (wave % S::WVN == 0 && lane < 16) {
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                const int m = lm + 16 * i;
                float z = sum[i];
                for (int w = 1; w < S::WVN; ++w) z += red[w * BM + wm + 16 * i + lane];
                if (m < M) {
                    const int64_t at = (int64_t)m * P.stat_ld + P.stat_first + tn;
                    gst(P.stat_max + at, mx[i] == -__builtin_huge_valf() ? mx[i] : tp_reference(mx[i], pow2));
                    gst(P.stat_sum + at, z);
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int m = lm + 16 * i;
            if (m >= M) continue;
            const int64_t tgt = tp_target(P.targets, P.vocab, m);
            const float lse = gld(P.lse + m);
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                const int n = ln + 16 * j;
                if (n >= P.ldp) continue;
                float v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    v[r] = tgt >= 0 && n + r < N ? expf(acc[i][j][r] - lse) - (P.n_first + n + r == tgt ? 1.0f : 0.0f)
                                                 : 0.0f;
                tp_store_planes((uint16_t*)P.P, P.p_planes, P.p_plane, (int64_t)m * P.ldp + n, v);
            }
        }
    }
}

}  // namespace scopt
