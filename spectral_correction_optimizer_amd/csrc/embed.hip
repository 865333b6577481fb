// Token embedding with scaling, and its gradient by sorted tokens.
//
//   out[t] = scale * table[ids[t]],   dW[v] = scale * sum over t with ids[t] = v of dy[t]
//
// An id outside [0, V) is no token: its output row is zero and it has no gradient.
//
// The gradient sums each table row's tokens in float32, in an order that the ids fix (token
// order within a stretch, then stretches), without atomics on floating values: it is the
// same on every run.  Token frequencies are far from even (the
// commonest token of a text owns several percent of the rows), so the work is split evenly
// over the sorted tokens and not over the table rows:
//   1. embed_bin_count, embed_bin_scatter: stable partition of the tokens into at most 512
//      bins of 2^shift neighbouring ids (each wavefront ranks its stretch of a block's
//      tokens, 64 at a time, by ballots);
//   2. embed_bin_sort: each bin's tokens by id in the same way, and the table rows' starts;
//   3. embed_sum: stretches of 8 to 32 sorted tokens, whatever their ids.  A table row
//      whose tokens lie within one stretch is stored at once; a row that crosses stretches
//      leaves a float32 partial sum per stretch.  Other workgroups of the same launch store
//      the zeros of the rows without a token;
//   4. embed_cross: the sum of the partials of each row that crossed.
// Bound by HBM: dy read once, dW written once (most rows of a large table are zeros).  65536
// tokens x 2048 in bfloat16, 131072 rows: 5 + 8 + 11 us for steps 1 and 2, 162 us for step 3
// (5.0 TB/s; zeros in a launch of their own: 114 + 119 us), 14 us for step 4.
#include "internal.hpp"
#include "rows.hpp"
#include "train.hpp"

namespace scopt {

namespace {
constexpr int kBins = 512;     // most bins; also the scatter's workgroup size
constexpr int kBlocks = 64;    // most token blocks
constexpr int kMaxRun = 32;    // most sorted tokens of a stretch
constexpr int kSlab = 512;     // columns of a wavefront
constexpr int64_t kMaxCross = 1 << 20;  // workgroups of embed_cross: a launch of 2^32 threads wraps, with no error

int64_t up(int64_t n, int64_t a) { return (n + a - 1) / a * a; }

// Exclusive sum of v over the nw wavefronts of a workgroup; sums: nw ints.
__device__ __forceinline__ int scan_exclusive(int v, int nw, int* sums) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int x = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(x, o);
        if (lane >= o) x += y;
    }
    if (lane == 63) sums[wave] = x;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < nw; ++w) before += w < wave ? sums[w] : 0;
    return before + x - v;
}

// LDS accesses of one wavefront stay in order; the compiler is told so
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

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

template <typename E, int ENDS>
__global__ __launch_bounds__(256) void embed_kernel(const E* __restrict__ table, const int64_t* __restrict__ ids,
                                                    int64_t T, int64_t V, int H, float scale, E* out) {
    const int per_row = (H + 7) / 8;
    const int64_t n = T * per_row;
    const bool small = n < (int64_t)1 << 31;
    for (int64_t g0 = (int64_t)blockIdx.x * 256 * kGroups + threadIdx.x; g0 < n;
         g0 += (int64_t)gridDim.x * 256 * kGroups) {
        Group8<E, ENDS> w[kGroups];
        int64_t t[kGroups], id[kGroups];
        int in[kGroups];
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            const int64_t g = g0 + k * 256;
            split_group(g < n ? g : n - 1, per_row, small, t[k], in[k]);
            id[k] = gld(ids + t[k]);
        }
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            const bool real = id[k] >= 0 && id[k] < V;
            w[k].load(table + (real ? id[k] : 0) * H, in[k] * 8, H);
        }
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            const int c = in[k] * 8;
            const bool real = id[k] >= 0 && id[k] < V;
            float v[8];
            value8(w[k], c, H, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = real ? v[i] * scale : 0.0f;
            if (g0 + k * 256 < n) store8(out + t[k] * H + c, H - c, v);
        }
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
// workgroup sums the counts itself (at most kBlocks x kBins of them); its 8 wavefronts take
// a stretch of the tokens each.
__global__ __launch_bounds__(kBins) void embed_bin_scatter_kernel(const int64_t* __restrict__ ids, int64_t T,
                                                                  int64_t V, int64_t per_block, int shift, int bins,
                                                                  int bin_bits, const int32_t* __restrict__ counts,
                                                                  int32_t* bin_start, int32_t* key, int32_t* pos) {
    constexpr int NW = kBins / 64;
    __shared__ int32_t at[NW][kBins];
    __shared__ int sums[NW];
    const int b = threadIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t from = (int64_t)blockIdx.x * per_block, to = from + per_block < T ? from + per_block : T;
    const int64_t part = per_block / NW;  // a multiple of 64
    const int64_t wfrom = from + wave * part, wto = wfrom + part < to ? wfrom + part : to;
    for (int w = 0; w < NW; ++w) at[w][b] = 0;
    __syncthreads();
    for (int64_t t = wfrom + lane; t < wto; t += 64) {
        const int64_t id = gld(ids + t);
        if (id >= 0 && id < V) atomicAdd(&at[wave][id >> shift], 1);
    }
    int before = 0, total = 0;
    if (b < bins) {
#pragma unroll 8
        for (unsigned k = 0; k < gridDim.x; ++k) {
            const int c = gld(counts + (int64_t)k * bins + b);
            total += c;
            before += k < blockIdx.x ? c : 0;
        }
    }
    const int start = scan_exclusive(total, NW, sums);  // its barrier also ends the counting
    if (blockIdx.x == 0 && b < bins) {
        gst(bin_start + b, start);
        if (b == bins - 1) gst(bin_start + bins, start + total);
    }
    int run = start + before;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const int c = at[w][b];
        at[w][b] = run;
        run += c;
    }
    __syncthreads();
    const uint64_t below = (1ull << lane) - 1;
    int64_t next = wfrom + lane < wto ? gld(ids + wfrom + lane) : -1;
    for (int64_t t0 = wfrom; t0 < wto; t0 += 64) {
        const int64_t t = t0 + lane, id = next;
        next = t + 64 < wto ? gld(ids + t + 64) : -1;
        const bool valid = id >= 0 && id < V;
        const uint32_t bin = valid ? (uint32_t)(id >> shift) : 0;
        const uint64_t m = same_key(bin, valid, bin_bits);
        if (valid) {
            const int o = at[wave][bin] + __popcll(m & below);
            gst(key + o, (int32_t)(id - ((int64_t)bin << shift)));
            gst(pos + o, (int32_t)t);
        }
        wave_fence();
        if (valid && (m & below) == 0) at[wave][bin] += __popcll(m);
        wave_fence();
    }
}

// One bin: its tokens in id order (token order within an id), and the starts of its rows.
// Each wavefront takes a stretch of the tokens; at: a counter per wavefront and row.
__global__ __launch_bounds__(1024) void embed_bin_sort_kernel(const int32_t* __restrict__ bin_start, int shift,
                                                              int64_t V, const int32_t* __restrict__ key,
                                                              const int32_t* __restrict__ pos, int32_t* row_start,
                                                              int32_t* sorted_id, int32_t* sorted_pos) {
    extern __shared__ int32_t at[];
    __shared__ int sums[16];
    const int rows = 1 << shift, nt = blockDim.x, nw = nt >> 6;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int from = gld(bin_start + blockIdx.x), to = gld(bin_start + blockIdx.x + 1);
    const int64_t first = (int64_t)blockIdx.x << shift;
    for (int i = threadIdx.x; i < nw * rows; i += nt) at[i] = 0;
    __syncthreads();
    const int part = (to - from + nt - 1) / nt * 64;
    const int wfrom = min(to, from + wave * part), wto = min(to, wfrom + part);
    int32_t* mine = at + wave * rows;
    for (int i = wfrom + lane; i < wto; i += 64) atomicAdd(&mine[gld(key + i)], 1);
    __syncthreads();
    // a thread's stretch of rows; its rows' counts over the wavefronts
    const int per = (rows + nt - 1) / nt, r0 = min(rows, (int)threadIdx.x * per), r1 = min(rows, r0 + per);
    int n = 0;
    for (int r = r0; r < r1; ++r)
        for (int w = 0; w < nw; ++w) n += at[w * rows + r];
    int run = from + scan_exclusive(n, nw, sums);
    for (int r = r0; r < r1; ++r) {
        if (first + r < V) gst(row_start + first + r, run);
        for (int w = 0; w < nw; ++w) {
            const int c = at[w * rows + r];
            at[w * rows + r] = run;
            run += c;
        }
    }
    if (first + rows >= V && threadIdx.x == 0) gst(row_start + V, to);  // the last bin
    __syncthreads();
    const uint64_t below = (1ull << lane) - 1;
    int nk = wfrom + lane < wto ? gld(key + wfrom + lane) : 0, np = wfrom + lane < wto ? gld(pos + wfrom + lane) : 0;
    for (int i0 = wfrom; i0 < wto; i0 += 64) {
        const int i = i0 + lane, k = nk, p = np;
        if (i + 64 < wto) {
            nk = gld(key + i + 64);
            np = gld(pos + i + 64);
        }
        const bool valid = i < wto;
        const uint64_t m = same_key((uint32_t)k, valid, shift);
        if (valid) {
            const int o = mine[k] + __popcll(m & below);
            gst(sorted_id + o, (int32_t)(first + k));
            gst(sorted_pos + o, p);
        }
        wave_fence();
        if (valid && (m & below) == 0) mine[k] += __popcll(m);
        wave_fence();
    }
}

// The first `sums` tasks: a wavefront sums one stretch's rows over kSlab columns.  The others:
// the zeros of eight table rows without a token, over kSlab columns.
template <typename E, int ENDS>
__global__ __launch_bounds__(256) void embed_sum_kernel(const E* __restrict__ dy, int H, int64_t V, float scale,
                                                        int len, const int32_t* __restrict__ row_start,
                                                        const int32_t* __restrict__ sorted_id,
                                                        const int32_t* __restrict__ sorted_pos, int64_t sums,
                                                        int64_t tasks, int slabs, E* dW, float* partial) {
    int64_t task = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (task >= tasks) return;
    const int lane = threadIdx.x & 63;
    const bool zeros = task >= sums;
    if (zeros) task -= sums;
    const int64_t run = task / slabs;
    const int c = (int)(task - run * slabs) * kSlab + lane * 8, left = H - c;
    if (zeros) {
        const int64_t v0 = run * 8;
        const int my_start = gld(row_start + (v0 + lane < V ? v0 + lane : V));
        const float none[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            if (v0 + r >= V) break;
            if (__builtin_amdgcn_readlane(my_start, r) == __builtin_amdgcn_readlane(my_start, r + 1) && left > 0)
                store8(dW + (v0 + r) * H + c, left, none);
        }
        return;
    }
    const int total = gld(row_start + V);
    const int from = (int)run * len, to = min(total, from + len);
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
        Group8<E, ENDS> w[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {  // past the end: the last token's row again, not summed
            const int64_t p = __builtin_amdgcn_readlane(my_pos, min(k0 + u, to - from - 1));
            w[u].load(dy + p * H, c, H);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + u;
            if (k >= to - from) break;
            float v[8];
            value8(w[u], c, H, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] += v[i];
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

// The row, if any, that crosses into stretch k + 1 from stretch k, where it begins: the sum of its
// partials, a quarter of them a wavefront.  Crossings and slabs beyond the grid's are taken in turn;
// which of them a workgroup skips is the same for all its threads.
template <typename E, int ENDS>
__global__ __launch_bounds__(256) void embed_cross_kernel(int H, int64_t V, float scale, int len,
                                                          const int32_t* __restrict__ row_start,
                                                          const int32_t* __restrict__ sorted_id,
                                                          const float* __restrict__ partial, int64_t items, int slabs,
                                                          E* dW) {
    __shared__ float red[3][kSlab];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int total = gld(row_start + V);
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int k = (int)(item / slabs) + 1;
        const int c = (int)(item % slabs) * kSlab + lane * 8, left = H - c;
        if (k * len >= total) break;
        const int64_t id = gld(sorted_id + k * len);
        const int s = gld(row_start + id), e = gld(row_start + id + 1);
        if (s >= k * len || s < (k - 1) * len) continue;
        const int last = (e - 1) / len, n = last - k + 2;  // partials: the first stretch's second one, then first ones
        const int per = (n + 3) / 4, p0 = min(n, wave * per), p1 = min(n, p0 + per);
        float acc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
#pragma unroll 4
        for (int p = p0; p < p1; ++p) {
            float v[8];
            load8<ENDS>(partial + (2ll * (k - 1 + p) + (p == 0 ? 1 : 0)) * H, c, H, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] += v[i];
        }
        if (wave > 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) red[wave - 1][i * 64 + lane] = acc[i];
        }
        __syncthreads();
        if (wave == 0 && left > 0) {
#pragma unroll
            for (int w = 0; w < 3; ++w)
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] += red[w][i * 64 + lane];
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] *= scale;
            store8(dW + id * H + c, left, acc);
        }
        __syncthreads();  // red is read
    }
}

hipError_t launch_embed(bool bf16, const void* table, const int64_t* ids, int64_t T, int64_t V, int H, float scale,
                        void* out, hipStream_t st) {
    if (T <= 0) return hipSuccess;
    const int64_t blocks = (T * ((H + 7) / 8) + 256 * kGroups - 1) / (256 * kGroups);
    const dim3 grid((unsigned)(blocks < 65536 ? blocks : 65536));
#define SC_EMBED(E_, ENDS_)                                                                              \
    hipLaunchKernelGGL((embed_kernel<E_, ENDS_>), grid, dim3(256), 0, st, (const E_*)table, ids, T, V, H, \
                       scale, (E_*)out);
    SC_BY_ENDS(bf16, H, SC_EMBED)
#undef SC_EMBED
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
    // the longest stretches that still give the chip 16 wavefronts a CU
    const int64_t slabs = (H + kSlab - 1) / kSlab;
    p.len = kMaxRun;
    while (p.len > 8 && T / p.len * slabs < 4096) p.len /= 2;
    p.runs = (T + p.len - 1) / p.len;
    p.slabs = slabs;
    p.tasks = (p.runs + (V + 7) / 8) * slabs;
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
    // a counter per wavefront and row of the bin in LDS: at most 32 KB
    const int waves = 8192 >> p.shift < 16 ? (8192 >> p.shift < 1 ? 1 : 8192 >> p.shift) : 16;
    hipLaunchKernelGGL(embed_bin_sort_kernel, dim3((unsigned)p.bins), dim3(64 * waves),
                       (waves * sizeof(int32_t)) << p.shift, st, bin, p.shift, p.V, key, pos, start, sid, spos);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const int H = (int)p.H, slabs = (int)p.slabs;
    const int64_t sums = p.runs * slabs, cross = (p.runs - 1) * slabs;
#define SC_EMBED(E_, ENDS_)                                                                                        \
    hipLaunchKernelGGL((embed_sum_kernel<E_, ENDS_>), dim3((unsigned)((p.tasks + 3) / 4)), dim3(256), 0, st,       \
                       (const E_*)dy, H, p.V, scale, p.len, start, sid, spos, sums, p.tasks, slabs, (E_*)dW, part); \
    if ((e = hipGetLastError()) != hipSuccess) return e;                                                           \
    if (cross > 0)                                                                                                 \
        hipLaunchKernelGGL((embed_cross_kernel<E_, ENDS_>), dim3((unsigned)(cross < kMaxCross ? cross : kMaxCross)), \
                           dim3(256), 0, st, H, p.V, scale, p.len, start, sid, part, cross, slabs, (E_*)dW);
    SC_BY_ENDS(bf16, p.H, SC_EMBED)
#undef SC_EMBED
    return hipGetLastError();
}

}  // namespace scopt
