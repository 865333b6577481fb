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
            const int c = slot ^ (r & 7) ^ ((r >> 3) & 1);
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
    // fetch the tile at k0 of a plane into lds; live = false fetches nothing (zeros)
    __device__ __forceinline__ void fetch(const uint16_t* p, int64_t ld, int rows, int K, int r0, int k0,
                                          bool live, uint16_t* lds) {
        asm volatile("" : "+v"(voff));  // the loads' offsets are formed here, not kept
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
            uint32_t v = voff + (uint32_t)(i * STEP * ld) * 2u;
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
            off = k * R + (((w0 / 16) ^ tp_swz<R>(k)) << 4) + (j & 3) * 4;
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
// Bfloat16 pairs of one row of NI blocks of 16 columns: in, lane group g = lane / 16 holds
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

// LDS written before is read after, by every wave; loads into LDS may stay under way
__device__ __forceinline__ void tp_lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
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
    __shared__ float red[EPI == TP_STATS ? 2 * S::WVN * BM : 1];  // row maxima, then sums

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

    const int ksteps = (P.K + 63) / 64, total = ksteps * P.nseg;
    const int per = (total + P.splits - 1) / P.splits;
    const int tiles = P.tiles_m * P.tiles_n, all = tiles * P.splits;

    // the step that is fetched next: its tile, segment and k
    struct Ahead {
        int m0, n0, seg, kst, left;
    } ah;
    auto begin_tile = [&](int turn) SC_INLINE {
        const int id = turn < all ? xcd_remap(turn, all) : 0;
        const int split = id / tiles;
        int tm, tn;
        tp_tile(id - split * tiles, P.tiles_m, P.tiles_n, tm, tn);
        ah.m0 = tm * BM;
        ah.n0 = tn * BN;
        const int step = split * per;
        ah.left = turn < all ? min(total, step + per) - step : 0;
        ah.seg = step / ksteps;
        ah.kst = step - ah.seg * ksteps;
    };
    auto fetch = [&](uint16_t* as, uint16_t* bs) SC_INLINE {
        const bool live = ah.left > 0;
        const uint32_t planes = live ? (uint32_t)(P.segs >> (4 * ah.seg)) : 0;
        la.fetch(P.A + (planes & 3) * P.a_plane, P.lda, P.M, P.K, ah.m0, ah.kst * 64, live, as);
        lb.fetch(P.B + ((planes >> 2) & 3) * P.b_plane, P.ldb, P.N, P.K, ah.n0, ah.kst * 64, live, bs);
        --ah.left;
        const bool wrap = ++ah.kst == ksteps;
        ah.kst = wrap ? 0 : ah.kst;
        ah.seg += wrap;
    };
    // A step's products go in four phases: each 32-deep half of k, in two groups of MI / 2 row
    // blocks.  A phase reads the fragments of the next one while it multiplies.
    constexpr int MG = MI / 2;
    v8bf fa[2][MG], fb[2][NI];
    auto read_a = [&](const uint16_t* as, int kk, int grp) SC_INLINE {
        ra.renew();
#pragma unroll
        for (int i = 0; i < MG; ++i) fa[grp][i] = ra.read(as, kk, grp * MG + i);
    };
    auto read_b = [&](const uint16_t* bs, int kk) SC_INLINE {
        rb.renew();
#pragma unroll
        for (int j = 0; j < NI; ++j) fb[kk][j] = rb.read(bs, kk, j);
    };
    auto multiply = [&](int kk, int grp) SC_INLINE {
#pragma unroll
        for (int i = 0; i < MG; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j)  // transposed: a lane's four sums are consecutive n
                acc[grp * MG + i][j] =
                    __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[kk][j], fa[grp][i], acc[grp * MG + i][j], 0, 0, 0);
    };
    // one phase's products with the reads spread between them
    auto spread = [&](auto reads) SC_INLINE {
        constexpr int READS = decltype(reads)::value, PRODS = MG * NI;
        constexpr int EVERY = PRODS / READS > 0 ? PRODS / READS : 1, AT_ONCE = (READS + PRODS - 1) / PRODS;
#pragma unroll
        for (int r = 0; r < READS / AT_ONCE; ++r) {
            __builtin_amdgcn_sched_group_barrier(0x100, AT_ONCE, 0);  // LDS reads
            __builtin_amdgcn_sched_group_barrier(0x008, EVERY, 0);    // products
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    using ReadsA = std::integral_constant<int, (AKC ? 1 : 2) * MG>;
    using ReadsAB = std::integral_constant<int, (AKC ? 1 : 2) * MG + (BKC ? 1 : 2) * NI>;
    // every step issues the same number of loads (the ones past the end fetch nothing)
    constexpr int PER = LA::NL + LB::NL;
    // On entry the fragments of this step's first phase are read or on their way.
    auto step = [&](uint16_t* as, uint16_t* bs, const uint16_t* an, const uint16_t* bn) SC_INLINE {
        read_a(as, 0, 1);
        multiply(0, 0);
        spread(ReadsA{});
        read_a(as, 1, 0);
        read_b(bs, 1);
        multiply(0, 1);
        spread(ReadsAB{});
        read_a(as, 1, 1);
        multiply(1, 0);
        spread(ReadsA{});
        // this wave's loads of the next step have landed and its reads of this step's buffer
        // are done; after the barrier that holds for every wave
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(PER * (NST - 2)) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        fetch(as, bs);
        __builtin_amdgcn_sched_barrier(0);  // the loads go out before the products
        read_a(an, 0, 0);
        read_b(bn, 0);
        multiply(1, 1);
        spread(ReadsAB{});
    };
    begin_tile(blockIdx.x);
    fetch(a0, b0);
    fetch(a1, b1);
    if constexpr (NST > 2) fetch(a2, b2);
    if constexpr (NST > 3) fetch(a3, b3);
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(PER * (NST - 1)) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");

    for (int turn = blockIdx.x; turn < all; turn += gridDim.x) {
    const int id = xcd_remap(turn, all), split = id / tiles;
    int tm, tn;
    tp_tile(id - split * tiles, P.tiles_m, P.tiles_n, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    // (the last step of the tile before has read these too, or they are the first)
    read_a(a0, 0, 0);
    read_b(b0, 0);
    // whole turns of the buffers, one at least: the steps past the end multiply zeros
    int left = max(1, min(total, split * per + per) - split * per);
    for (; left > 0; left -= NST) {
        if (left <= NST) begin_tile(turn + gridDim.x);  // the last turn fetches the next tile's first steps
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

    // Lane l holds, of block (i, j): row m = wm + 16 i + l % 16, columns
    // n = wn + 16 j + 4 (l / 16) + 0..3.
    // (formed anew for every tile: the registers are the main loop's)
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const int lm = m0 + wm + (lane & 15), ln = n0 + wn + 4 * (lane >> 4);
    const int M = P.M, N = P.N;
    const bool whole = n0 + BN <= N;  // all columns of the tile exist
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
                const int m = lm + 16 * i;
                uint32_t d[NI][2];
#pragma unroll
                for (int j = 0; j < NI; ++j)
#pragma unroll
                    for (int w = 0; w < 2; ++w)
                        d[j][w] = pack_bf16x2(acc[i][j][2 * w] * g[j][2 * w], acc[i][j][2 * w + 1] * g[j][2 * w + 1]);
                const int c = tp_gather_row<NI>(d);
                if (m < M) tp_store_row<NI>((uint16_t*)P.C + (int64_t)m * P.ldc + n0 + wn + c, d);
            }
        } else {
            auto store = [&](auto bf16) SC_INLINE {
#pragma unroll
                for (int i = 0; i < MI; ++i)
#pragma unroll
                    for (int j = 0; j < NI; ++j) {
                        const int m = lm + 16 * i, n = ln + 16 * j;
                        const float v[4] = {acc[i][j][0] * g[j][0], acc[i][j][1] * g[j][1], acc[i][j][2] * g[j][2],
                                            acc[i][j][3] * g[j][3]};
                        if (m < M) tp_store(P.C, decltype(bf16)::value, (int64_t)m * P.ldc + n, v, N - n);
                    }
            };
            if (P.c_bf16) store(std::true_type{});
            else store(std::false_type{});
        }
    } else if constexpr (EPI == TP_PART) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                const int m = lm + 16 * i, n = ln + 16 * j;
                const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                if (m < M) tp_store(P.part, 0, ((int64_t)split * M + m) * N + n, v, N - n);
            }
    } else if constexpr (EPI == TP_STATS) {
        // row maximum over the tile's columns: registers, the four lanes of a row, the
        // waves beside each other
        int hit[MI];  // the target's column in this wave's part, or -1
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int64_t t = gld(P.targets + min(lm + 16 * i, M - 1)) - P.n_first;
            const int64_t c = t - (n0 + wn);
            hit[i] = lm + 16 * i < M && t < N && c >= 0 && c < WN ? (int)c : -1;
        }
        if (!whole) {
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (ln + 16 * j + r >= N) acc[i][j][r] = -__builtin_huge_valf();
        }
        const bool pow2 = P.keep == TP_KEEP_EXP;
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            float v = acc[i][0][0];
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) v = fmaxf(v, acc[i][j][r]);
            v = fmaxf(v, __shfl_xor(v, 16));
            v = fmaxf(v, __shfl_xor(v, 32));
            if (lane < 16) red[(wave % S::WVN) * BM + wm + 16 * i + lane] = v;
            if (__ballot(hit[i] >= 0)) {
#pragma unroll
                for (int j = 0; j < NI; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (hit[i] == 16 * j + 4 * (lane >> 4) + r) gst(P.target_logit + lm + 16 * i, acc[i][j][r]);
            }
        }
        tp_lds_barrier();
        float* sums = red + S::WVN * BM;
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int m = lm + 16 * i;
            float mx = red[wm + 16 * i + (lane & 15)];
#pragma unroll
            for (int w = 1; w < S::WVN; ++w) mx = fmaxf(mx, red[w * BM + wm + 16 * i + (lane & 15)]);
            const float ref = tp_reference(mx, pow2);
            float z = 0.0f;
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
                    d[j][0] = pack_bf16x2(e[0], e[1]);
                    d[j][1] = pack_bf16x2(e[2], e[3]);
                }
                uint16_t* p = (uint16_t*)P.P + (int64_t)m * P.ldp;
                if (whole) {
                    const int c = tp_gather_row<NI>(d);
                    if (m < M) tp_store_row<NI>(p + n0 + wn + c, d);
                } else if (m < M) {
#pragma unroll
                    for (int j = 0; j < NI; ++j)
                        if (ln + 16 * j < P.ldp) *(SC_GLOBAL v2u*)(p + ln + 16 * j) = v2u{d[j][0], d[j][1]};
                }
            } else {
#pragma unroll
                for (int j = 0; j < NI; ++j) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) z += __builtin_amdgcn_exp2f((acc[i][j][r] - ref) * kLog2e);
                    if (P.keep == TP_KEEP_LOGIT && m < M && ln + 16 * j < P.ldp)
                        gst4((float*)P.P + (int64_t)m * P.ldp + ln + 16 * j, acc[i][j]);
                }
            }
            z += __shfl_xor(z, 16);
            z += __shfl_xor(z, 32);
            if (lane < 16) sums[(wave % S::WVN) * BM + wm + 16 * i + lane] = z;
            if (wave % S::WVN == 0 && lane < 16 && m < M)
                gst(P.stat_max + (int64_t)(P.stat_first + tn) * M + m,
                    mx == -__builtin_huge_valf() ? mx : ref);
        }
        tp_lds_barrier();
        for (int r = threadIdx.x; r < BM; r += NT) {
            float z = sums[r];
#pragma unroll
            for (int w = 1; w < S::WVN; ++w) z += sums[w * BM + r];
            if (m0 + r < M) gst(P.stat_sum + (int64_t)(P.stat_first + tn) * M + m0 + r, z);
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
                    v[r] = tgt >= 0 && n + r < N ? __builtin_amdgcn_exp2f((acc[i][j][r] - lse) * kLog2e) -
                                                       (P.n_first + n + r == tgt ? 1.0f : 0.0f)
                                                 : 0.0f;
                tp_store_planes((uint16_t*)P.P, P.p_planes, P.p_plane, (int64_t)m * P.ldp + n, v);
            }
        }
    }
    }
    // loads past the end may still be on their way into LDS
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
}

}  // namespace scopt
