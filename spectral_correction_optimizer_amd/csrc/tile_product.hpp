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
// out are below 2^-23 of |a b|.  With HALF the planes are float16: two of them hold 22 bits of a row that a
// power of two takes into their range, three products leave out below 3 2^-22 of |a b| (2^-37 of the
// rows' largest values), and the powers of two come back with the sums.
//
// A workgroup owns a BM x BN tile; buffers in LDS hold 64 k of it.  Both operand tiles go
// from memory straight into LDS (16 bytes per lane, no registers); each wave multiplies a
// (BM / WVM) x (BN / WVN) part in 16 x 16 x 32 blocks, 32 k a step.  A step's fragments are
// read from LDS during the products of the step before it, so a buffer is free, and being
// filled again, one step before its products end.  Each buffer is an array of its own and the
// loop is unrolled over them, so the reads of one buffer do not wait for the loads that fill
// another.
//
// At 256 x 256, 8 waves and two buffers: 1330 TFLOP/s at 8192 x 2048 x 131072 (A with k
// contiguous, B with rows), 1190 at 131072 x 2048 x 8192 (both with rows).  The matrix cores are
// busy for 66 and 61% of the cycles, LDS for a quarter of them without a bank conflict, at a clock
// of 1.85 GHz (2.4 at most).  Tried
// and not kept: four buffers of 32 k (64-byte rows where k is contiguous: 10% slower there),
// fragments that are read in the step that multiplies them (1040), addresses formed in
// every step instead of every turn of the buffers (8% slower), and sums that the register
// allocator places (it moves them about and spills).
//
// LDS layouts (16-byte slots permuted within a row by choosing which global chunk each
// lane fetches, so that the matrix operand reads touch every bank once):
//   k contiguous:    [row][64 k], slot = chunk ^ (row >> 1 & 7); a fragment is one 16-byte
//                    read per lane.  (The hardware takes 16 lanes at a time, in quads that
//                    are not all consecutive; this order has no conflict, row & 7 had.)
//   rows contiguous: [k][rows], 32-byte blocks, block ^= (k & 3) | ((k >> 3) & 1) << 2;
//                    a fragment is two transposing reads (ds_read_b64_tr_b16: 16 lanes
//                    read four k rows of 16 elements, each lane receives the four k of
//                    one row).
// Bounds: every load goes through a buffer resource that ends at the operand's end, so rows
// (k contiguous) or k (rows contiguous) past it deliver zeros.  A chunk past K of a row with k
// contiguous gets an offset beyond the end.  Columns past the rows of a k row deliver that
// row's padding or the next k row: they only reach sums that are not stored.
//
// A workgroup takes tiles in turn, as many workgroups as run at once, and the loads of its
// next tile are under way while the sums of this one are stored.
#pragma once

#include <type_traits>

#include "common.hpp"
#include "internal.hpp"
#include "rows.hpp"
#include "train.hpp"

namespace scopt {

typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));

#define SC_LDS __attribute__((address_space(3)))
#define SC_INLINE __attribute__((always_inline))

constexpr uint32_t kTpMaxBytes = 0x7fffffffu;  // largest buffer range (offsets stay below 2^31)
constexpr uint32_t kTpBeyond = 0x80000000u;    // an offset beyond every range

// Rows contiguous: the permutation of row k's 32-byte blocks
template <int R>
__device__ __forceinline__ int tp_swz(int k) {
    constexpr int MASK = R >= 128 ? 7 : R / 16 - 1;
    return ((k & 3) | (((k >> 3) & 1) << 2)) & MASK;
}

// Loader of one operand's R x 64 tile: offsets are set up once, the base advances.
template <int R, int NT, bool KC>
struct TpLoader {
    static constexpr int NL = R * 8 / NT;  // 16-byte loads per thread and tile
    static constexpr int STEP = KC ? NT / 8 : NT / (R / 8);  // rows (or k) between them
    static_assert(STEP % 16 == 0, "the permutation of a row's slots repeats every 16 rows");
    uint32_t voff;  // of the first load
    int kchunk;     // KC: the k of this lane's chunk within a tile
    __device__ __forceinline__ void init(int64_t ld) {
        const int t = threadIdx.x;
        if constexpr (KC) {
            const int r = t >> 3, slot = t & 7;
            const int c = slot ^ ((r >> 1) & 7);
            kchunk = c * 8;
            voff = (uint32_t)(r * ld + c * 8) * 2u;
        } else {
            constexpr int CR = R / 8;  // chunks per k row
            const int k = t / CR, slot = t % CR;
            const int c = slot ^ tp_swz<R>(k) * 2;
            kchunk = 0;
            voff = (uint32_t)(k * ld + c * 8) * 2u;
        }
    }
    __amdgpu_buffer_rsrc_t rs;
    int k_left;      // of this turn
    uint32_t ahead;  // bytes from one tile to the next one's
    // the tiles of a turn from k0 of a plane; live = false: zeros
    __device__ __forceinline__ void prepare(const uint16_t* p, int64_t ld, int rows, int K, int r0, int k0,
                                            bool live) {
        // a row of k ends at a whole chunk (what lies between is zero or meets zeros), and so
        // does a row of rows (the sums of what lies beyond are not stored)
        if (KC) K = (K + 7) & ~7;
        else rows = (rows + 7) & ~7;
        const int64_t first = KC ? (int64_t)r0 * ld + k0 : (int64_t)k0 * ld + r0;
        const int64_t total = KC ? (int64_t)(rows - 1) * ld + K : (int64_t)(K - 1) * ld + rows;
        int64_t bytes = (total - first) * 2;
        bytes = bytes < (int64_t)kTpMaxBytes ? bytes : (int64_t)kTpMaxBytes;
        rs = buf_rsrc(p + first, live && bytes > 0 ? (uint32_t)bytes : 0u);
        k_left = K - k0;
        ahead = (KC ? 1u : (uint32_t)ld) * 128u;
    }
    // fetch tile u of the turn into lds (offsets beyond the end stay there: the tiles of a turn span less
    // than 2 GiB)
    __device__ __forceinline__ void issue(int64_t ld, int u, uint16_t* lds) {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        asm volatile("" : "+v"(voff));  // the loads' offsets are formed here, not kept
        uint32_t v = voff + u * ahead;
        if (KC) v = u * 64 + kchunk < k_left ? v : kTpBeyond;
#pragma unroll
        for (int i = 0; i < NL; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (SC_LDS void*)(lds + i * NT * 8 + wave * 512), 16,
                                                     v + (uint32_t)(i * STEP * ld) * 2u, 0, 0, 0);
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
            off = (w0 + j) * 64 + ((g ^ (j >> 1)) << 3);
        } else {
            const int k = g * 8 + (j >> 2);
            off = k * R + (((w0 / 16) ^ tp_swz<R>(k)) << 4) + (j & 3) * 4;
        }
    }
    // The offsets are formed anew where this is called: kept in registers over the loop they
    // would not fit beside the sums.
    __device__ __forceinline__ void renew() { asm volatile("" : "+v"(off)); }
    // the 8 k values (32 kk + 8 * (lane / 16) ..) of row w0 + 16 b + lane % 16
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

// four consecutive elements at `at`, the first `left` of them inside the row
__device__ __forceinline__ void tp_store(void* base, int bf16, int64_t at, const float (&v)[4], int left) {
    if (bf16) {
        uint16_t* p = (uint16_t*)base + at;
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (r < left) gst(p + r, f32_to_bf16(v[r]));
    } else {
        float* p = (float*)base + at;
        if (left >= 4) {
            *(SC_GLOBAL v4f_any*)p = v4f_any{v[0], v[1], v[2], v[3]};
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (r < left) gst(p + r, v[r]);
        }
    }
}
// Pairs of 16-bit values of one row of NI blocks of 16 columns: in, lane group g = lane / 16 holds
// columns 4 g .. 4 g + 3 of every block; out, 4 NI consecutive columns, and the first of them.
// (Rows of 16 lanes change places between registers; the stores then write whole 16 bytes,
// and with NI = 4 a row's 128 bytes are four lanes'.)
template <int NI>
__device__ __forceinline__ int tp_gather_row(uint32_t (&d)[NI][2]) {
    static_assert(NI == 2 || NI == 4, "blocks of a wave");
    const int g = (threadIdx.x & 63) >> 4;
    auto swap16 = [](uint32_t& x, uint32_t& y) SC_INLINE {
        const auto r = __builtin_amdgcn_permlane16_swap(x, y, false, false);
        x = r[0];
        y = r[1];
    };
    auto swap32 = [](uint32_t& x, uint32_t& y) SC_INLINE {
        const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
        x = r[0];
        y = r[1];
    };
#pragma unroll
    for (int w = 0; w < 2; ++w) {
#pragma unroll
        for (int j = 0; j < NI; j += 2) swap16(d[j][w], d[j + 1][w]);
        if constexpr (NI == 4) {
            swap32(d[0][w], d[2][w]);
            swap32(d[1][w], d[3][w]);
        }
    }
    return NI == 4 ? 16 * g : 16 * (g & 1) + 4 * (g & 2);
}
template <int NI>
__device__ __forceinline__ void tp_store_row(uint16_t* p, const uint32_t (&d)[NI][2]) {
#pragma unroll
    for (int j = 0; j < NI; j += 2)
        *(SC_GLOBAL v4u_any*)(p + 4 * j) = v4u_any{d[j][0], d[j][1], d[j + 1][0], d[j + 1][1]};
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
// the row of C that holds row m of the product
__device__ __forceinline__ int64_t tp_row(const TpArgs& P, int m) { return P.rows ? gld(P.rows + m) : m; }
constexpr float kLog2e = 1.44269504088896340736f;
// The reference of a tile's exponentials.  TP_KEEP_EXP: the row maximum in powers of two,
// rounded up; otherwise the maximum itself.  A tile whose row is all -infinity takes 0, so
// that its exponentials are 0 and not NaN.
__device__ __forceinline__ float tp_reference(float mx, bool pow2) {
    if (mx == -__builtin_huge_valf()) return 0.0f;
    if (!pow2) return mx;
    float ref = ceilf(mx * kLog2e);
    // the product may have been rounded down to a whole number: no exponential is above 1
    if (fmaf(mx, kLog2e, -ref) > 0.0f) ref += fmaxf(1.0f, fabsf(ref) * 0x1p-23f);
    return ref;
}
// Two exponentials in [0, 1] as 16 bits each, the first one low: float32's bits without the sign
// and the upper bit of the exponent, which are 0 below 2, and without the last 14, rounded to
// nearest.  Nine bits of fraction are kept: half a step is 2^-10 of the value, where
// bfloat16's would be 2^-8.
__device__ __forceinline__ uint32_t tp_pack_unit(float a, float b) {
    return __builtin_amdgcn_perm((__float_as_uint(b) << 2) + 0x8000u, (__float_as_uint(a) << 2) + 0x8000u,
                                 0x07060302u);
}
__device__ __forceinline__ float tp_unit_lo(uint32_t w) { return __uint_as_float((w & 0xffffu) << 14); }
__device__ __forceinline__ float tp_unit_hi(uint32_t w) { return __uint_as_float(w >> 16 << 14); }

// Where the references of the rows are known beforehand (TpArgs::row_ref), a tile's exponentials are kept
// relative to its row's, and are the row's gradients but for a factor: as long as the tile's own reference is no
// more than 2^kByRow above it (a NaN is no such reference).  Bfloat16's exponents leave room for the
// products of such values and for the factors, their inverses.
constexpr float kByRow = 64.0f;
__device__ __forceinline__ bool tp_by_row(float ref, float row_ref) { return ref - row_ref <= kByRow; }

// What becomes of a tile's sums.
enum TpEpi {
    TP_STORE = 0,   // C = acc * alpha * gain[n], bfloat16 or float32
    TP_PART = 1,    // float32 sums of one split of k, [split][M][N]
    TP_STATS = 2,   // row maxima and exp sums of the tile; logits kept as P.keep says
    TP_GRAD = 3,    // (exp(acc - lse[m]) - [n is m's target]) * alpha, as bfloat16 planes
    TP_TAIL = 4,    // C = acc * coef[m] at row rows[m]; tiles that do not fill a round are cut along k
                    // (TpTail) and leave float32 sums, [split][tile][BM][BN]
    TP_STATS_TAIL = 5,  // TP_STATS, cut likewise
};
constexpr bool tp_stats(int epi) { return epi == TP_STATS || epi == TP_STATS_TAIL; }
constexpr bool tp_cuts(int epi) { return epi == TP_TAIL || epi == TP_STATS_TAIL; }

template <int BM_, int BN_, int WVM_, int WVN_, int NBUF_, int PER_CU_, bool ROTATE_ = false>
struct TpShape {
    static constexpr bool ROTATE = ROTATE_;
    static constexpr int BM = BM_, BN = BN_, WVM = WVM_, WVN = WVN_, NBUF = NBUF_, PER_CU = PER_CU_;
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

// LDS written before is read after, by every wave; loads into LDS may stay under way
__device__ __forceinline__ void tp_lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <class S, bool AKC, bool BKC, int EPI, bool HALF = false>
__global__ __launch_bounds__(S::NT, S::WAVES) void tile_product_kernel(const TpArgs P) {
    constexpr int BM = S::BM, BN = S::BN, NT = S::NT;
    constexpr int NBUF = S::NBUF;
    constexpr int WM = BM / S::WVM, WN = BN / S::WVN, MI = WM / 16, NI = WN / 16;
    using LA = TpLoader<BM, NT, AKC>;
    using LB = TpLoader<BN, NT, BKC>;
    constexpr int ASZ = BM * 64, BSZ = BN * 64;
    static_assert(NBUF >= 2 && NBUF <= 6, "buffers");
    __shared__ __align__(1024) uint16_t a0[ASZ], b0[BSZ], a1[ASZ], b1[BSZ];
    __shared__ __align__(1024) uint16_t a2[NBUF > 2 ? ASZ : 8], b2[NBUF > 2 ? BSZ : 8];
    __shared__ __align__(1024) uint16_t a3[NBUF > 3 ? ASZ : 8], b3[NBUF > 3 ? BSZ : 8];
    __shared__ __align__(1024) uint16_t a4[NBUF > 4 ? ASZ : 8], b4[NBUF > 4 ? BSZ : 8];
    __shared__ __align__(1024) uint16_t a5[NBUF > 5 ? ASZ : 8], b5[NBUF > 5 ? BSZ : 8];
    __shared__ float red[tp_stats(EPI) ? 2 * S::WVN * BM : 1];  // row maxima, then sums

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = (wave / S::WVN) * WM, wn = (wave % S::WVN) * WN;

    LA la;
    LB lb;
    la.init(P.lda);
    lb.init(P.ldb);
    TpReader<BM, MI, AKC> ra;
    TpReader<BN, NI, BKC> rb;
    ra.init(wm);
    rb.init(wn);

    v4f acc[MI][NI];

    // Tokens are the rows of A where it has k contiguous, else k; only the first of them may be live.
    int M = P.M, K = P.K, tiles_m = P.tiles_m;
    if (P.live) {
        const int live = __builtin_amdgcn_readfirstlane(gld(P.live));
        if constexpr (AKC) {
            M = min(M, live);
            tiles_m = (M + BM - 1) / BM;
            if (M == 0) return;
        } else {
            K = min(K, live);
        }
    }
    // k goes in turns of the buffers; what lies past its end multiplies zeros.
    const int kturns = max(1, (K + 64 * NBUF - 1) / (64 * NBUF)), total = kturns * P.nseg;
    const int tiles = tiles_m * P.tiles_n;
    TpTail tail = {0, tiles, P.splits};
    if constexpr (tp_cuts(EPI)) {
        tail.full = __builtin_amdgcn_readfirstlane(gld(&P.tail->full));
        tail.rest = __builtin_amdgcn_readfirstlane(gld(&P.tail->rest));
        tail.splits = __builtin_amdgcn_readfirstlane(gld(&P.tail->splits));
    }
    const int all = tail.full + tail.rest * tail.splits;
    // tile and part of k of a turn
    struct Item {
        int tile, split, from, to;
    };
    auto item = [&](int turn) SC_INLINE {
        Item i;
        if (tp_cuts(EPI) && turn < tail.full) {
            i.tile = xcd_remap(turn, tail.full);
            i.split = i.from = 0;
            i.to = total;
        } else {
            const int id = xcd_remap(turn - tail.full, all - tail.full);
            const int per = (total + tail.splits - 1) / tail.splits;
            i.split = id / tail.rest;
            i.tile = tail.full + id - i.split * tail.rest;
            i.from = i.split * per;
            i.to = min(total, i.from + per);
        }
        return i;
    };

    // the turn that is fetched next: its tile, segment and place in the segment
    struct Ahead {
        int m0, n0, seg, kt, left, rot;
    } ah;
    // Each tile's turns in an order of its own: where a row's bytes are a power of two, all tiles at the same k
    // would read from a few memory channels.
    constexpr bool ROTATE = S::ROTATE;
    auto begin_tile = [&](int turn) SC_INLINE {
        Item it = {0, 0, 0, 0};
        if (turn < all) it = item(turn);
        int tm, tn;
        tp_tile(it.tile, tiles_m, P.tiles_n, tm, tn);
        ah.m0 = tm * BM;
        ah.n0 = tn * BN;
        ah.left = it.to - it.from;
        ah.rot = ROTATE ? it.tile % kturns : 0;
        ah.seg = it.from / kturns;
        ah.kt = it.from - ah.seg * kturns;
    };
    auto prepare = [&]() SC_INLINE {
        const bool live = ah.left > 0;
        const uint32_t planes = live ? (uint32_t)(P.segs >> (4 * ah.seg)) : 0;
        int kt = ah.kt;
        if constexpr (ROTATE) kt = kt + ah.rot < kturns ? kt + ah.rot : kt + ah.rot - kturns;
        const int k0 = kt * 64 * NBUF;
        la.prepare(P.A + (planes & 3) * P.a_plane, P.lda, M, K, ah.m0, k0, live);
        lb.prepare(P.B + ((planes >> 2) & 3) * P.b_plane, P.ldb, P.N, K, ah.n0, k0, live);
        --ah.left;
        const bool wrap = ++ah.kt == kturns;
        ah.kt = wrap ? 0 : ah.kt;
        ah.seg += wrap;
    };
    auto issue = [&](int u, uint16_t* as, uint16_t* bs) SC_INLINE {
        la.issue(P.lda, u, as);
        lb.issue(P.ldb, u, bs);
    };
    // A step's products go in two phases, of MI / 2 row blocks each; a phase reads fragments of
    // the next step (half kk of a buffer) while it multiplies.
    constexpr int MG = MI / 2;
    v8bf fa[2][2][MG], fb[2][NI];  // [step's parity]
    // Products in place in the accumulation registers: left to itself the register allocator
    // moves sums about and spills fragments.
    auto product = [&](int cur, int grp, int p) SC_INLINE {
        const int i = p / NI, j = p % NI;  // transposed: a lane's four sums are consecutive n
        if constexpr (HALF)
            asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0"
                         : "+a"(acc[grp * MG + i][j])
                         : "v"(fb[cur][j]), "v"(fa[cur][grp][i]));
        else
            asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0"
                         : "+a"(acc[grp * MG + i][j])
                         : "v"(fb[cur][j]), "v"(fa[cur][grp][i]));
    };
    // The products of a group, and spread between them the next step's reads of A's group and,
    // with the first group, of B.
    auto phase = [&](auto parity, auto group, const uint16_t* as, const uint16_t* bs, int kk) SC_INLINE {
        constexpr int cur = decltype(parity)::value, nxt = cur ^ 1, grp = decltype(group)::value;
        constexpr int READS = MG + (grp == 0 ? NI : 0), PRODS = MG * NI;
        ra.renew();
        if constexpr (grp == 0) rb.renew();
#pragma unroll
        for (int p = 0; p < PRODS; ++p) {
#pragma unroll
            for (int r = (p * READS + PRODS - 1) / PRODS; r < ((p + 1) * READS + PRODS - 1) / PRODS; ++r) {
                if (grp == 0 && r < NI) fb[nxt][r] = rb.read(bs, kk, r);
                else fa[nxt][grp][r - (grp == 0 ? NI : 0)] = ra.read(as, kk, grp * MG + r - (grp == 0 ? NI : 0));
            }
            product(cur, grp, p);
            __builtin_amdgcn_sched_barrier(0x6);  // scalar and vector arithmetic may pass
        }
    };
    using P0 = std::integral_constant<int, 0>;
    using P1 = std::integral_constant<int, 1>;
    // every tile of a turn takes the same number of loads (the ones past the end fetch nothing)
    constexpr int PER = LA::NL + LB::NL;
    // Buffer u of a turn: its halves' fragments are read during the products of the step before
    // each.  Then it is free and filled with the tile NBUF further on.
    auto buffer = [&](int u, uint16_t* as, uint16_t* bs) SC_INLINE {
        phase(P1{}, P0{}, as, bs, 0);
        phase(P1{}, P1{}, as, bs, 0);
        phase(P0{}, P0{}, as, bs, 1);
        phase(P0{}, P1{}, as, bs, 1);
        // this wave's loads of the next buffer have landed and its reads of this one are done;
        // after the barrier that holds for every wave
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(PER * (NBUF - 2)) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        issue(u, as, bs);
        __builtin_amdgcn_sched_barrier(0x6);  // the loads go out before the products
    };
    begin_tile(blockIdx.x);
    prepare();
    issue(0, a0, b0);
    issue(1, a1, b1);
    if constexpr (NBUF > 2) issue(2, a2, b2);
    if constexpr (NBUF > 3) issue(3, a3, b3);
    if constexpr (NBUF > 4) issue(4, a4, b4);
    if constexpr (NBUF > 5) issue(5, a5, b5);
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(PER * (NBUF - 1)) : "memory");

    for (int turn = blockIdx.x; turn < all; turn += gridDim.x) {
        const Item it = item(turn);
        const int split = it.split;
        int tm, tn;
        tp_tile(it.tile, tiles_m, P.tiles_n, tm, tn);
        const int m0 = tm * BM, n0 = tn * BN;
        // (TP_STATS: a column past the last one starts at -infinity and, its operand being zero, stays)
#pragma unroll
        for (int j = 0; j < NI; ++j) {
            v4f start = {0.f, 0.f, 0.f, 0.f};
            if constexpr (tp_stats(EPI)) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int n = n0 + wn + 16 * j + 4 * ((threadIdx.x & 63) >> 4) + r;
                    start[r] = n < P.N ? 0.0f : -__builtin_huge_valf();
                }
            }
#pragma unroll
            for (int i = 0; i < MI; ++i) acc[i][j] = start;
        }
        // Every step reads the next one's fragments: the first reads come with products of zeros.
        const v8bf zeros = {};
#pragma unroll
        for (int j = 0; j < NI; ++j) fb[1][j] = zeros;
#pragma unroll
        for (int i = 0; i < MI; ++i) fa[1][i / MG][i % MG] = zeros;
        __builtin_amdgcn_s_barrier();  // the first buffer has landed for every wave
        asm volatile("s_nop 7" ::: "memory");  // and the zeros are written
        for (int turns = max(1, it.to - it.from); turns > 0; --turns) {
            if (turns == 1) begin_tile(turn + gridDim.x);  // the last turn fetches the next tile's first one
            prepare();
            buffer(0, a0, b0);
            buffer(1, a1, b1);
            if constexpr (NBUF > 2) buffer(2, a2, b2);
            if constexpr (NBUF > 3) buffer(3, a3, b3);
            if constexpr (NBUF > 4) buffer(4, a4, b4);
            if constexpr (NBUF > 5) buffer(5, a5, b5);
        }
#pragma unroll
        for (int grp = 0; grp < 2; ++grp)
#pragma unroll
            for (int p = 0; p < MG * NI; ++p) product(1, grp, p);  // the last step's
        // The next tile's buffers land before the stores go out: its first steps would else wait
        // for those too.
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

        // The last products are written before other instructions read them.  Row blocks leave the
        // accumulation registers one at a time.
        asm volatile("s_nop 15\n\ts_nop 3" ::: "memory");
        auto row_block = [&](int i) SC_INLINE {
#pragma unroll
            for (int j = 0; j < NI; ++j) asm volatile("" : "+a"(acc[i][j]));
        };

        // Lane l holds, of block (i, j): row m = wm + 16 i + l % 16, columns
        // n = wn + 16 j + 4 (l / 16) + 0..3.
        // (formed anew for every tile: the registers are the main loop's)
        int lane = threadIdx.x & 63;
        asm volatile("" : "+v"(lane));
        const int lm = m0 + wm + (lane & 15), ln = n0 + wn + 4 * (lane >> 4);
        const int N = P.N;
        const bool whole = n0 + BN <= N;  // all columns of the tile exist
        // a part of a cut tile
        const bool cut = tp_cuts(EPI) && turn >= tail.full && tail.splits > 1;
        float* part = P.part + ((int64_t)split * tail.rest + (it.tile - tail.full)) * (BM * BN);
        if constexpr (EPI == TP_STORE) {
            const float alpha = P.alpha ? gld(P.alpha) : 1.0f;
            float g[NI][4];
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) g[j][r] = alpha;
            if (P.gain) {
                auto scale = [&](auto* gain) SC_INLINE {
                    using G = std::remove_const_t<std::remove_pointer_t<decltype(gain)>>;
#pragma unroll
                    for (int j = 0; j < NI; ++j)
#pragma unroll
                        for (int r = 0; r < 4; ++r) g[j][r] *= Elem<G>::load(gain, min(ln + 16 * j + r, N - 1));
                };
                if (P.gain_bf16) scale((const uint16_t*)P.gain);
                else scale((const float*)P.gain);
            }
            if (P.c_bf16 && whole) {
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    row_block(i);
                    const int m = lm + 16 * i;
                    uint32_t d[NI][2];
#pragma unroll
                    for (int j = 0; j < NI; ++j)
#pragma unroll
                        for (int w = 0; w < 2; ++w)
                            d[j][w] = pack_bf16x2(acc[i][j][2 * w] * g[j][2 * w],
                                                  acc[i][j][2 * w + 1] * g[j][2 * w + 1]);
                    const int c = tp_gather_row<NI>(d);
                    if (m < M) tp_store_row<NI>((uint16_t*)P.C + (int64_t)m * P.ldc + n0 + wn + c, d);
                }
            } else {
                auto store = [&](auto bf16) SC_INLINE {
#pragma unroll
                    for (int i = 0; i < MI; ++i) {
                        row_block(i);
#pragma unroll
                        for (int j = 0; j < NI; ++j) {
                            const int m = lm + 16 * i, n = ln + 16 * j;
                            float v[4];
#pragma unroll
                            for (int r = 0; r < 4; ++r) v[r] = acc[i][j][r] * g[j][r];
                            if (m < M) tp_store(P.C, decltype(bf16)::value, (int64_t)m * P.ldc + n, v, N - n);
                        }
                    }
                };
                if (P.c_bf16) store(std::true_type{});
                else store(std::false_type{});
            }
        } else if constexpr (EPI == TP_PART) {
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                row_block(i);
#pragma unroll
                for (int j = 0; j < NI; ++j) {
                    const int m = lm + 16 * i, n = ln + 16 * j;
                    const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                    if (m < M) tp_store(P.part, 0, ((int64_t)split * M + m) * N + n, v, N - n);
                }
            }
        } else if constexpr (EPI == TP_TAIL) {
            // Each row block leaves the accumulation registers at one place, whatever becomes of it: where
            // the ways of storing it each read them, the register allocator moved sums ahead of the
            // waits above.
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                row_block(i);
                const int m = lm + 16 * i, in = min(m, M - 1);
                float f = 1.0f;  // (only the states' rows are tokens)
                if constexpr (AKC) f = P.coef && !cut ? gld(P.coef + in) : 1.0f;
                float v[NI][4];
#pragma unroll
                for (int j = 0; j < NI; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) v[j][r] = AKC ? acc[i][j][r] * f : acc[i][j][r];
                if (cut) {
#pragma unroll
                    for (int j = 0; j < NI; ++j)
                        gst4(part + (m - m0) * BN + ln - n0 + 16 * j, v4f{v[j][0], v[j][1], v[j][2], v[j][3]});
                    continue;
                }
                const int64_t at = (AKC ? tp_row(P, in) : in) * P.ldc + n0 + wn;
                if (P.c_bf16 && whole) {
                    uint32_t d[NI][2];
#pragma unroll
                    for (int j = 0; j < NI; ++j)
#pragma unroll
                        for (int w = 0; w < 2; ++w) d[j][w] = pack_bf16x2(v[j][2 * w], v[j][2 * w + 1]);
                    const int c = tp_gather_row<NI>(d);
                    if (m < M) tp_store_row<NI>((uint16_t*)P.C + at + c, d);
                } else if (m < M) {
#pragma unroll
                    for (int j = 0; j < NI; ++j)
                        tp_store(P.C, P.c_bf16, at + 4 * (lane >> 4) + 16 * j, v[j], N - (ln + 16 * j));
                }
            }
        } else if constexpr (tp_stats(EPI)) {
            // row maximum over the tile's columns: registers, the four lanes of a row, the
            // waves beside each other
            int hit[MI];  // the target's column in this wave's part, or -1
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                const int64_t t = gld(P.targets + min(lm + 16 * i, M - 1)) - P.n_first;
                const int64_t c = t - (n0 + wn);
                hit[i] = lm + 16 * i < M && t < N && c >= 0 && c < WN ? (int)c : -1;
            }
            const bool pow2 = !HALF && P.keep == TP_KEEP_EXP;  // (float32 logits are kept as such)
            float* sums = red + S::WVN * BM;
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                row_block(i);
                float v = -__builtin_huge_valf();
                v4f x[NI];  // (see TP_TAIL: one place)
                int ea = 0, eb_at = ln;
                if constexpr (HALF) {
                    ea = gld(P.a_exp + min(lm + 16 * i, M - 1));
                    asm volatile("" : "+v"(eb_at));  // read anew for each row block: kept, they would be spilled
                }
#pragma unroll
                for (int j = 0; j < NI; ++j) {
                    v4i eb;
                    if constexpr (HALF) eb = *(const SC_GLOBAL v4i*)(P.b_exp + eb_at + 16 * j);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        x[j][r] = acc[i][j][r];
                        if constexpr (HALF) x[j][r] = cut ? x[j][r] : ldexpf(x[j][r], ea + eb[r]);
                        v = fmaxf(v, x[j][r]);
                    }
                    if constexpr (HALF) acc[i][j] = x[j];
                }
                if (tp_cuts(EPI) && cut) {
#pragma unroll
                    for (int j = 0; j < NI; ++j) gst4(part + (lm + 16 * i - m0) * BN + ln - n0 + 16 * j, x[j]);
                    continue;
                }
                v = fmaxf(v, __shfl_xor(v, 16));
                v = fmaxf(v, __shfl_xor(v, 32));
                if (lane < 16) red[(wave % S::WVN) * BM + wm + 16 * i + lane] = v;
                if (__ballot(hit[i] >= 0)) {
#pragma unroll
                    for (int j = 0; j < NI; ++j)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (hit[i] == 16 * j + 4 * (lane >> 4) + r)
                                gst(P.target_logit + lm + 16 * i, x[j][r]);
                }
            }
            if (tp_cuts(EPI) && cut) continue;
            tp_lds_barrier();
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                row_block(i);
                const int m = lm + 16 * i;
                float mx = red[wm + 16 * i + (lane & 15)];
#pragma unroll
                for (int w = 1; w < S::WVN; ++w) mx = fmaxf(mx, red[w * BM + wm + 16 * i + (lane & 15)]);
                const float ref = tp_reference(mx, pow2);
                float z = 0.0f, unit = 1.0f;
                bool by_row = false;
                if constexpr (EPI == TP_STATS_TAIL && !HALF) {
                    if (P.row_ref) {
                        const float to = gld(P.row_ref + min(m, M - 1));
                        by_row = tp_by_row(ref, to);
                        unit = __builtin_amdgcn_exp2f(ref - to);
                    }
                }
                uint32_t d[NI][2];
                if (pow2) {
#pragma unroll
                    for (int j = 0; j < NI; ++j) {
                        float e[4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            e[r] = __builtin_amdgcn_exp2f(fmaf(acc[i][j][r], kLog2e, -ref));
                            z += e[r];
                        }
                        if (by_row) {
                            d[j][0] = pack_bf16x2(e[0] * unit, e[1] * unit);
                            d[j][1] = pack_bf16x2(e[2] * unit, e[3] * unit);
                        } else {
                            d[j][0] = tp_pack_unit(e[0], e[1]);
                            d[j][1] = tp_pack_unit(e[2], e[3]);
                        }
                    }
                    uint16_t* p = (uint16_t*)P.P + (int64_t)m * P.ldp;
                    const int c = tp_gather_row<NI>(d);
                    if (m < M) tp_store_row<NI>(p + n0 + wn + c, d);
                } else {
#pragma unroll
                    for (int j = 0; j < NI; ++j) {
#pragma unroll
                        for (int r = 0; r < 4; ++r) z += __builtin_amdgcn_exp2f((acc[i][j][r] - ref) * kLog2e);
                        if (P.keep == TP_KEEP_LOGIT && m < M)
                            gst4((float*)P.P + (int64_t)m * P.ldp + ln + 16 * j, acc[i][j]);
                    }
                }
                z += __shfl_xor(z, 16);
                z += __shfl_xor(z, 32);
                if (lane < 16) sums[(wave % S::WVN) * BM + wm + 16 * i + lane] = z;
                if (wave % S::WVN == 0 && lane < 16 && m < M)
                    gst(P.stat_max + (int64_t)(P.stat_first + tn) * P.M + m,
                        mx == -__builtin_huge_valf() ? mx : ref);
            }
            tp_lds_barrier();
            for (int r = threadIdx.x; r < BM; r += NT) {
                float z = sums[r];
#pragma unroll
                for (int w = 1; w < S::WVN; ++w) z += sums[w * BM + r];
                if (m0 + r < M) gst(P.stat_sum + (int64_t)(P.stat_first + tn) * P.M + m0 + r, z);
            }
        } else {
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                const int m = lm + 16 * i;
                row_block(i);
                if (m >= M) continue;
                float alpha = gld(P.coef ? P.coef + m : P.alpha);
                if (P.coef_zeros && alpha != 0.0f) alpha = 1.0f;
                // a row without weight is one of zeros, whatever its logits are
                const int64_t tgt = alpha != 0.0f ? tp_target(P.targets, P.vocab, m) : -1;
                const float lse = gld(P.lse + m);
                int ea = 0;
                if constexpr (HALF) ea = gld(P.a_exp + m);
                // (the rows' factors are made for the target's entry as the statistics' pass saw it)
                const float tl = P.coef_zeros ? gld(P.target_logit + m) : 0.0f;
                auto at_target = [&](int n, float x) SC_INLINE {
                    return P.coef_zeros && P.n_first + n == tgt ? tl : x;
                };
#pragma unroll
                for (int j = 0; j < NI; ++j) {
                    const int n = ln + 16 * j;
                    float v[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        float s = acc[i][j][r];
                        if constexpr (HALF) s = ldexpf(s, ea + gld(P.b_exp + min(n + r, N - 1)));
                        v[r] = tgt >= 0 && n + r < N ? (__builtin_amdgcn_exp2f((at_target(n + r, s) - lse) * kLog2e) -
                                                        (P.n_first + n + r == tgt ? 1.0f : 0.0f)) *
                                                           alpha
                                                     : 0.0f;
                    }
                    tp_store_planes((uint16_t*)P.P, P.p_planes, P.p_plane, (int64_t)m * P.ldp + n, v);
                }
            }
        }
    }
    // loads past the end may still be on their way into LDS
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
}

}  // namespace scopt
