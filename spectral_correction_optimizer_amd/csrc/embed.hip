// Token embedding with scaling, and its gradient by sorted tokens.
//
//   out[t] = scale * table[ids[t]],   dW[v] = scale * sum over t with ids[t] = v of dy[t]
//
// An id outside [0, V) is no token: its output row is zero and it has no gradient.
//
// The gradient sums each table row's tokens in token order, in float32, without atomics on
// floating values, so it is the same on every run.  Token frequencies are far from even (the
// commonest token of a text owns several percent of the rows), so the work is split evenly
// over the sorted tokens and not over the table rows:
//   1. embed_bin_count, embed_bin_scatter: stable partition of the tokens into at most 512
//      bins of 2^shift neighbouring ids (one wavefront per block of tokens scatters, ranking
//      64 tokens at a time by ballots);
//   2. embed_bin_sort: each bin's tokens by id, and the table rows' starts;
//   3. embed_sum: stretches of kRun sorted tokens, whatever their ids.  A table row
//      whose tokens lie within one stretch is stored at once; a row that crosses stretches
//      leaves a float32 partial sum per stretch;
//   4. embed_finish: zeros where a row has no token, the sum of the partials of a row that
//      crossed.
// Bound by HBM: dy read once, dW written once (most rows of a large table are zeros).
#include "internal.hpp"
#include "rows.hpp"
#include "train.hpp"

namespace scopt {

namespace {
constexpr int kBins = 512;     // most bins; also the scatter's workgroup size
constexpr int kBlocks = 64;    // most token blocks
constexpr int kRun = 32;       // sorted tokens of a stretch
constexpr int kSlab = 512;     // columns of a wavefront

int64_t up(int64_t n, int64_t a) { return (n + a - 1) / a * a; }

// Among the 64 lanes with the same key (valid lanes): the mask of them.  `bits` key bits.
__device__ __forceinline__ uint64_t same_key(uint32_t key, bool valid, int bits) {
    uint64_t m = __ballot(valid);
    for (int b = 0; b < bits; ++b) {
        const uint64_t set = __ballot((key >> b) & 1);
        m &= (key >> b) & 1 ? set : ~set;
    }
    return m;
}
}  // namespace

template <typename E>
__global__ __launch_bounds__(256) void embed_kernel(const E* __restrict__ table, const int64_t* __restrict__ ids,
                                                    int64_t T, int64_t V, int H, float scale, E* out) {
    const int per_row = (H + 7) / 8;
    const int64_t n = T * per_row;
    for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < n; g += (int64_t)gridDim.x * 256) {
        const int64_t t = g / per_row;
        const int c = (int)(g - t * per_row) * 8;
        const int64_t id = gld(ids + t);
        float v[8];
        if (id >= 0 && id < V) {
            load8(table + id * H + c, H - c, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= scale;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.0f;
        }
        store8(out + t * H + c, H - c, v);
    }
}

// counts[block][bin] of the block's tokens
__global__ __launch_bounds__(256) void embed_bin_count_kernel(const int64_t* __restrict__ ids, int64_t T, int64_t V,
                                                              int64_t per_block, int shift, int bins,
                                                              int32_t* counts) {
    __shared__ int32_t cnt[kBins];
    for (int b = threadIdx.x; b < bins; b += 256) cnt[b] = 0;
    __syncthreads();
    const int64_t from = (int64_t)blockIdx.x * per_block, to = from + per_block < T ? from + per_block : T;
    for (int64_t t = from + threadIdx.x; t < to; t += 256) {
        const int64_t id = gld(ids + t);
        if (id >= 0 && id < V) atomicAdd(&cnt[id >> shift], 1);
    }
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += 256) gst(counts + (int64_t)blockIdx.x * bins + b, cnt[b]);
}

// Stable scatter of a block's tokens to their bins: (id within the bin, token).  Every
// workgroup sums the counts itself (at most kBlocks x kBins of them).
__global__ __launch_bounds__(kBins) void embed_bin_scatter_kernel(const int64_t* __restrict__ ids, int64_t T,
                                                                  int64_t V, int64_t per_block, int shift, int bins,
                                                                  int bin_bits, const int32_t* __restrict__ counts,
                                                                  int32_t* bin_start, int32_t* key, int32_t* pos) {
    __shared__ int32_t scan[kBins], at[kBins];
    const int b = threadIdx.x;
    int before = 0, total = 0;
    if (b < bins)
        for (unsigned k = 0; k < gridDim.x; ++k) {
            const int c = gld(counts + (int64_t)k * bins + b);
            total += c;
            if (k < blockIdx.x) before += c;
        }
    scan[b] = total;
    __syncthreads();
    for (int o = 1; o < kBins; o <<= 1) {
        const int x = b >= o ? scan[b - o] : 0;
        __syncthreads();
        scan[b] += x;
        __syncthreads();
    }
    const int start = scan[b] - total;
    at[b] = start + before;
    if (blockIdx.x == 0 && b < bins) {
        gst(bin_start + b, start);
        if (b == bins - 1) gst(bin_start + bins, start + total);
    }
    __syncthreads();
    if (threadIdx.x >= 64) return;
    // one wavefront from here on: its LDS accesses stay in order
    const int lane = threadIdx.x;
    const uint64_t below = (1ull << lane) - 1;
    const int64_t from = (int64_t)blockIdx.x * per_block, to = from + per_block < T ? from + per_block : T;
    int64_t next = from + lane < to ? gld(ids + from + lane) : -1;
    for (int64_t t0 = from; t0 < to; t0 += 64) {
        const int64_t t = t0 + lane, id = next;
        next = t + 64 < to ? gld(ids + t + 64) : -1;
        const bool valid = id >= 0 && id < V;
        const uint32_t bin = valid ? (uint32_t)(id >> shift) : 0;
        const uint64_t m = same_key(bin, valid, bin_bits);
        if (valid) {
            const int base = at[bin];
            const int o = base + __popcll(m & below);
            gst(key + o, (int32_t)(id - ((int64_t)bin << shift)));
            gst(pos + o, (int32_t)t);
        }
        __builtin_amdgcn_wave_barrier();
        if (valid && (m & below) == 0) at[bin] += __popcll(m);
        __builtin_amdgcn_wave_barrier();
    }
}

// One bin: its tokens in id order (token order within an id), and the starts of its rows.
__global__ __launch_bounds__(256) void embed_bin_sort_kernel(const int32_t* __restrict__ bin_start, int shift,
                                                             int64_t V, const int32_t* __restrict__ key,
                                                             const int32_t* __restrict__ pos, int32_t* row_start,
                                                             int32_t* sorted_id, int32_t* sorted_pos) {
    extern __shared__ int32_t at[];  // 2^shift counters, then starts
    __shared__ int32_t sums[256];
    const int rows = 1 << shift;
    const int from = gld(bin_start + blockIdx.x), to = gld(bin_start + blockIdx.x + 1);
    const int64_t first = (int64_t)blockIdx.x << shift;
    for (int r = threadIdx.x; r < rows; r += 256) at[r] = 0;
    __syncthreads();
    for (int i = from + threadIdx.x; i < to; i += 256) atomicAdd(&at[gld(key + i)], 1);
    __syncthreads();
    // exclusive scan: a thread's stretch of rows, then the threads' sums
    const int per = (rows + 255) / 256, r0 = min(rows, (int)threadIdx.x * per), r1 = min(rows, r0 + per);
    int mine = 0;
    for (int r = r0; r < r1; ++r) mine += at[r];
    sums[threadIdx.x] = mine;
    __syncthreads();
    for (int o = 1; o < 256; o <<= 1) {
        const int x = (int)threadIdx.x >= o ? sums[threadIdx.x - o] : 0;
        __syncthreads();
        sums[threadIdx.x] += x;
        __syncthreads();
    }
    int run = from + sums[threadIdx.x] - mine;
    for (int r = r0; r < r1; ++r) {
        const int c = at[r];
        at[r] = run;
        if (first + r < V) gst(row_start + first + r, run);
        run += c;
    }
    if (first + rows >= V && threadIdx.x == 0) gst(row_start + V, to);  // the last bin
    __syncthreads();
    if (threadIdx.x >= 64) return;
    const int lane = threadIdx.x;
    const uint64_t below = (1ull << lane) - 1;
    int nk = from + lane < to ? gld(key + from + lane) : 0, np = from + lane < to ? gld(pos + from + lane) : 0;
    for (int i0 = from; i0 < to; i0 += 64) {
        const int i = i0 + lane, k = nk, p = np;
        if (i + 64 < to) {
            nk = gld(key + i + 64);
            np = gld(pos + i + 64);
        }
        const bool valid = i < to;
        const uint64_t m = same_key((uint32_t)k, valid, shift);
        if (valid) {
            const int o = at[k] + __popcll(m & below);
            gst(sorted_id + o, (int32_t)(first + k));
            gst(sorted_pos + o, p);
        }
        __builtin_amdgcn_wave_barrier();
        if (valid && (m & below) == 0) at[k] += __popcll(m);
        __builtin_amdgcn_wave_barrier();
    }
}

// A wavefront sums one stretch's rows over kSlab columns.
template <typename E>
__global__ __launch_bounds__(256) void embed_sum_kernel(const E* __restrict__ dy, int H, int64_t V, float scale,
                                                        const int32_t* __restrict__ row_start,
                                                        const int32_t* __restrict__ sorted_id,
                                                        const int32_t* __restrict__ sorted_pos, int64_t tasks, int slabs,
                                                        E* dW, float* partial) {
    const int64_t task = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (task >= tasks) return;
    const int lane = threadIdx.x & 63;
    const int64_t run = task / slabs;
    const int c = (int)(task - run * slabs) * kSlab + lane * 8, left = H - c;
    const int total = gld(row_start + V);
    const int from = (int)run * kRun, to = min(total, from + kRun);
    if (from >= to) return;
    // one token a lane; ids and rows are broadcast from there
    const int mine = min(from + lane, to - 1);
    const int my_id = gld(sorted_id + mine), my_pos = gld(sorted_pos + mine);
    const int my_start = gld(row_start + my_id), my_end = gld(row_start + my_id + 1);
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
    constexpr int U = 8;  // rows in flight
    for (int k0 = 0; k0 < to - from; k0 += U) {
        float v[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) {  // past the end: the last token's row again, not summed
            const int64_t p = __builtin_amdgcn_readlane(my_pos, min(k0 + u, to - from - 1));
            load8(dy + p * H + c, left, v[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + u;
            if (k >= to - from) break;
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] += v[u][i];
            const int end = __builtin_amdgcn_readlane(my_end, k);
            if (from + k + 1 == end || from + k + 1 == to) {  // the row's last token here
                const int start = __builtin_amdgcn_readlane(my_start, k);
                if (left > 0) {
                    if (start >= from && end <= to) {
                        const int64_t id = __builtin_amdgcn_readlane(my_id, k);
#pragma unroll
                        for (int i = 0; i < 8; ++i) acc[i] *= scale;
                        store8(dW + id * H + c, left, acc);
                    } else {
                        store8(partial + (2 * run + (start < from ? 0 : 1)) * H + c, left, acc);
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
            }
        }
    }
}

// Eight table rows a wavefront, over kSlab columns.
template <typename E>
__global__ __launch_bounds__(256) void embed_finish_kernel(int H, int64_t V, float scale,
                                                           const int32_t* __restrict__ row_start,
                                                           const float* __restrict__ partial, int64_t tasks, int slabs,
                                                           E* dW) {
    const int64_t task = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (task >= tasks) return;
    const int lane = threadIdx.x & 63;
    const int64_t v0 = task / slabs * 8;
    const int c = (int)(task % slabs) * kSlab + lane * 8, left = H - c;
    const int64_t at = v0 + (lane & 15) < V ? v0 + (lane & 15) : V;
    const int my_start = gld(row_start + at);
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        if (v0 + r >= V) break;
        const int s = __builtin_amdgcn_readlane(my_start, r), e = __builtin_amdgcn_readlane(my_start, r + 1);
        float acc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
        if (s < e) {
            const int first = s / kRun, last = (e - 1) / kRun;
            if (first == last) continue;
            if (left > 0) {
                load8(partial + (2ll * first + 1) * H + c, left, acc);
                for (int k = first + 1; k <= last; ++k) {
                    float p[8];
                    load8(partial + 2ll * k * H + c, left, p);
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[i] += p[i];
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] *= scale;
        }
        if (left > 0) store8(dW + (v0 + r) * H + c, left, acc);
    }
}

hipError_t launch_embed(bool bf16, const void* table, const int64_t* ids, int64_t T, int64_t V, int H, float scale,
                        void* out, hipStream_t st) {
    if (T <= 0) return hipSuccess;
    const int64_t blocks = (T * ((H + 7) / 8) + 255) / 256;
    const dim3 grid((unsigned)(blocks < 65536 ? blocks : 65536));
    if (bf16)
        hipLaunchKernelGGL(embed_kernel<uint16_t>, grid, dim3(256), 0, st, (const uint16_t*)table, ids, T, V, H,
                           scale, (uint16_t*)out);
    else
        hipLaunchKernelGGL(embed_kernel<float>, grid, dim3(256), 0, st, (const float*)table, ids, T, V, H, scale,
                           (float*)out);
    return hipGetLastError();
}

EmbedGradPlan embed_grad_plan(int64_t T, int64_t V, int64_t H) {
    EmbedGradPlan p{};
    p.T = T;
    p.V = V;
    p.H = H;
    while (((V - 1) >> p.shift) >= kBins) ++p.shift;
    p.bins = (int)((V - 1) >> p.shift) + 1;
    p.per_block = up(T > 0 ? (T + kBlocks - 1) / kBlocks : 1, 1024);
    p.blocks = (T + p.per_block - 1) / p.per_block;
    if (p.blocks < 1) p.blocks = 1;
    p.runs = (T + kRun - 1) / kRun;
    int64_t o = 0;
    auto take = [&](int64_t bytes) {
        const int64_t at = o;
        o += up(bytes, 256);
        return at;
    };
    p.o_counts = take(4 * p.blocks * p.bins);
    p.o_bin = take(4 * (p.bins + 1));
    p.o_key = take(4 * T);
    p.o_pos = take(4 * T);
    p.o_id = take(4 * T);
    p.o_spos = take(4 * T);
    p.o_start = take(4 * (V + 1));
    p.o_part = take(4 * 2 * p.runs * H);
    p.bytes = o;
    return p;
}

hipError_t launch_embed_grad(const EmbedGradPlan& p, bool bf16, const void* dy, const int64_t* ids, float scale,
                             void* dW, void* workspace, hipStream_t st) {
    char* ws = (char*)workspace;
    int32_t *counts = (int32_t*)(ws + p.o_counts), *bin = (int32_t*)(ws + p.o_bin), *key = (int32_t*)(ws + p.o_key),
            *pos = (int32_t*)(ws + p.o_pos), *sid = (int32_t*)(ws + p.o_id), *spos = (int32_t*)(ws + p.o_spos),
            *start = (int32_t*)(ws + p.o_start);
    float* part = (float*)(ws + p.o_part);
    hipError_t e;
    int bin_bits = 0;
    while ((1 << bin_bits) < p.bins) ++bin_bits;
    hipLaunchKernelGGL(embed_bin_count_kernel, dim3((unsigned)p.blocks), dim3(256), 0, st, ids, p.T, p.V, p.per_block,
                       p.shift, p.bins, counts);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(embed_bin_scatter_kernel, dim3((unsigned)p.blocks), dim3(kBins), 0, st, ids, p.T, p.V,
                       p.per_block, p.shift, p.bins, bin_bits, counts, bin, key, pos);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(embed_bin_sort_kernel, dim3((unsigned)p.bins), dim3(256), sizeof(int32_t) << p.shift, st, bin,
                       p.shift, p.V, key, pos, start, sid, spos);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const int slabs = (int)((p.H + kSlab - 1) / kSlab);
    const int64_t sums = p.runs * slabs, rows = (p.V + 7) / 8 * slabs;
#define SC_EMBED(E_)                                                                                              \
    if (sums > 0)                                                                                                 \
        hipLaunchKernelGGL(embed_sum_kernel<E_>, dim3((unsigned)((sums + 3) / 4)), dim3(256), 0, st, (const E_*)dy, \
                           (int)p.H, p.V, scale, start, sid, spos, sums, slabs, (E_*)dW, part);                   \
    if ((e = hipGetLastError()) != hipSuccess) return e;                                                          \
    hipLaunchKernelGGL(embed_finish_kernel<E_>, dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, st, (int)p.H, p.V, \
                       scale, start, part, rows, slabs, (E_*)dW)
    if (bf16) {
        SC_EMBED(uint16_t);
    } else {
        SC_EMBED(float);
    }
#undef SC_EMBED
    return hipGetLastError();
}

}  // namespace scopt
