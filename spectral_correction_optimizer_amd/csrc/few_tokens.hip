// The weights' gradient of few tokens (at most 128, bfloat16): dW[v][n] = sum over tokens of d[t][v] h[t][n].
// Such a product is a write of dW: the general kernel's tiles are mostly their own beginning and end (32000 x
// 2048 from 72 tokens 46 us, 2.9 TB/s).  Here a workgroup keeps its 256 columns of h, all tokens deep, in
// registers and goes down the rows of dW, 64 at a time: their d comes through LDS one step ahead, asked for before
// the step's stores, and those are waited for a step later only (the compiler's wait before the next step's reads of
// LDS, behind the loads after it).  The same product takes 30 us (4.4 TB/s).
#include "tile_product.hpp"

namespace scopt {

// KT: 64-token tiles
template <int KT>
__global__ __launch_bounds__(256, 4) void few_tokens_kernel(const uint16_t* __restrict__ d, int64_t ldd,
                                                         const uint16_t* __restrict__ h, int64_t ldh, int T,
                                                         const int* __restrict__ live, int V, int N, uint16_t* dW,
                                                         int64_t ldw, int panels, int blocks) {
    // two steps' d (KT tiles of 64 tokens x 64 rows); before them, 64 tokens of h: a half of the columns each
    __shared__ __align__(1024) uint16_t a0[64 * 128], a1[64 * 128];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int K = min(T, __builtin_amdgcn_readfirstlane(gld(live)));
    const int id = xcd_remap(blockIdx.x, gridDim.x);  // the panels of the same rows share an XCD
    const int n0 = id % panels * 256, wn = wave * 64;
    const int from = id / panels * blocks, to = min(from + blocks, (V + 63) / 64);

    v8bf b[2 * KT][4];
    {
        TpLoader<128, 256, false> load;
        load.init(ldh);
        TpReader<128, 4, false> read;
        read.init(wn & 64);
#pragma unroll
        for (int u = 0; u < KT; ++u) {
            __syncthreads();
            load.prepare(h, ldh, N, K, n0, 0, n0 < N);
            load.issue(ldh, u, a0);
            load.prepare(h, ldh, N, K, n0 + 128, 0, n0 + 128 < N);
            load.issue(ldh, u, a1);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __syncthreads();
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int j = 0; j < 4; ++j) b[2 * u + kk][j] = read.read(wave < 2 ? a0 : a1, kk, j);
        }
        __syncthreads();
    }

    TpLoader<64, 256, false> load;
    load.init(ldd);
    TpReader<64, 4, false> read;
    read.init(0);
    auto issue = [&](int blk, uint16_t* lds) SC_INLINE {
        load.prepare(d, ldd, V, K, blk * 64, 0, blk < to);
#pragma unroll
        for (int u = 0; u < KT; ++u) load.issue(ldd, u, lds + u * 64 * 64);
    };
    const bool whole = n0 + wn + 64 <= N;
    auto step = [&](int blk, uint16_t* lds, uint16_t* next) SC_INLINE {
        __builtin_amdgcn_s_barrier();  // every wave's part of this step's d is there, and the last step's was read
        asm volatile("" ::: "memory");
        issue(blk + 1, next);
        // the loads go out before this step's reads and stores: the wait at its end counts on that
        __builtin_amdgcn_sched_barrier(0x6);  // (scalar and vector arithmetic may pass)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v4f acc[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 2 * KT; ++k) {
                const v8bf a = read.read(lds + (k >> 1) * 64 * 64, k & 1, i);
#pragma unroll
                for (int j = 0; j < 4; ++j)  // transposed: a lane's four sums are consecutive columns
                    acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[k][j], a, acc[j], 0, 0, 0);
            }
            const int v = blk * 64 + 16 * i + (lane & 15);
            uint16_t* row = dW + (int64_t)v * ldw + n0 + wn;
            if (whole) {
                uint32_t w[4][2];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    w[j][0] = pack_bf16x2(acc[j][0], acc[j][1]);
                    w[j][1] = pack_bf16x2(acc[j][2], acc[j][3]);
                }
                const int c = tp_gather_row<4>(w);
                if (v < V) tp_store_row<4>(row + c, w);
            } else if (v < V) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int n = 16 * j + 4 * (lane >> 4);
                    const float x[4] = {acc[j][0], acc[j][1], acc[j][2], acc[j][3]};
                    tp_store(row, 1, n, x, N - (n0 + wn + n));
                }
            }
        }
        // The next step's d was asked for before this step's stores, 8 of them in a wave that has whole columns
        // (fewer where rows end: there is no next step).
        if (whole) asm volatile("s_waitcnt vmcnt(8) lgkmcnt(0)" ::: "memory");
        else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    };
    issue(from, a0);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    for (int blk = from; blk < to; blk += 2) {
        step(blk, a0, a1);
        if (blk + 1 < to) step(blk + 1, a1, a0);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // loads past the end may still be on their way into LDS
}

hipError_t launch_few_tokens(const uint16_t* d, int64_t ldd, const uint16_t* h, int64_t ldh, int T, const int* live,
                             int V, int N, uint16_t* dW, hipStream_t st) {
    constexpr int want = 1024;  // four workgroups a CU
    const int panels = (N + 255) / 256, rows = (V + 63) / 64;
    const int chunks = panels < want ? want / panels : 1;
    const int blocks = (rows + chunks - 1) / chunks;
    const dim3 grid((unsigned)((rows + blocks - 1) / blocks * panels));
    auto kernel = T <= 64 ? few_tokens_kernel<1> : few_tokens_kernel<2>;
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, d, ldd, h, ldh, T, live, V, N, dW, (int64_t)N, panels, blocks);
    return hipGetLastError();
}

}  // namespace scopt
