// The global gradient norm over many tensors, and clipping by it:
//
//   sumsq = sum of g^2 over all elements,  norm = sqrt(sumsq),  scale = min(1, max_norm / (norm + 1e-6)),
//   out = g scale
//
// Two passes, each bound by HBM: 112 matrices, 3.9 GB in float32, are read in 0.69 ms (5.7 TB/s) and scaled into
// others in 1.43 ms (5.4).  A second read is not to be had from the 256 MB cache but for its end; gradients that fit
// there, 4 MB in 130 tensors, take 6.4 and 8 us, less than the host's 20.  The tensors' addresses come with the
// launch (kernel arguments, so the calls can be captured and hold nothing between them); a workgroup finds its tensor
// by the number of chunks before it.  Squares are summed in 64 bits: those of float32's largest and smallest gradients
// are out of its own range.
#include "common.hpp"
#include "internal.hpp"
#include "rows.hpp"
#include "train.hpp"

namespace scopt {

constexpr int kClipThreads = 256, kClipGroups = 4;
constexpr int64_t kClipChunk = (int64_t)kClipThreads * kClipGroups * 8;  // elements of a chunk
constexpr int kClipTensors = 140;  // a launch takes 4 KiB of arguments
constexpr int kSumsqGrid = 2048, kFewParts = 4 * kClipThreads;
// (112 matrices, a chunk each 2120 us, 8192 workgroups 2150, 32768 2112)
constexpr int kClipGrid = 32768;

struct ClipTable {
    const void* src[kClipTensors];
    void* dst[kClipTensors];
    int64_t size[kClipTensors];
    uint32_t first[kClipTensors + 1];  // chunks before each tensor
    int count, in_place;  // in_place: every dst is its src
};

static_assert(sizeof(ClipTable) <= 4000, "a launch's arguments");

// tensor of a chunk: the last one that begins at or before it
__device__ __forceinline__ int clip_find(const ClipTable& t, uint32_t chunk) {
    int lo = 0, hi = t.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (t.first[mid] <= chunk) lo = mid;
        else hi = mid;
    }
    return lo;
}

// eight elements at p, `left` of them inside the tensor
template <typename E> __device__ __forceinline__ void clip_load(const E* p, int64_t left, float (&v)[8]) {
    if (left >= 8) {
        Group8<E, ROW_WHOLE> g;
        g.load(p, 0, 8);
        g.raw(v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? Elem<E>::load(p, i) : 0.0f;
    }
}

template <typename E>
__global__ __launch_bounds__(kClipThreads) void sumsq_kernel(const ClipTable t, double* __restrict__ part) {
    __shared__ double red[kClipThreads / 64];
    double s = 0.0;
    const uint32_t chunks = t.first[t.count];
    for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int i = clip_find(t, c);
        const int64_t at = (int64_t)(c - t.first[i]) * kClipChunk;
        const E* p = (const E*)t.src[i] + at;
        const int64_t left = t.size[i] - at;
        float v[kClipGroups][8];
#pragma unroll
        for (int k = 0; k < kClipGroups; ++k) {
            const int o = (k * kClipThreads + (int)threadIdx.x) * 8;
            clip_load(p + o, left - o, v[k]);
        }
#pragma unroll
        for (int k = 0; k < kClipGroups; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) s = fma((double)v[k][j], (double)v[k][j], s);
    }
    s = block_sum_f64(s, red);
    if (threadIdx.x == 0) gst(part + blockIdx.x, s);
}

// (sumsq may be the first part)
__global__ __launch_bounds__(1024) void sumsq_join_kernel(const double* part, int parts, double* sumsq) {
    __shared__ double red[16];
    double s = 0.0;
    for (int i = threadIdx.x; i < parts; i += 1024) s += gld(part + i);
    s = block_sum_f64(s, red);
    if (threadIdx.x == 0) gst(sumsq, s);
}

// The sum of squares in at most kFewParts parts, which each workgroup adds up for itself: for few chunks that is less
// than another launch (130 small tensors: the call 24.5 us with it, 19.9 without).
template <typename E>
__global__ __launch_bounds__(kClipThreads) void clip_kernel(const ClipTable t, const double* __restrict__ sumsq, int parts,
                                                            float max_norm, float* norm, float* scale_out) {
    __shared__ double red[kClipThreads / 64];
    double all = parts == 1 ? gld(sumsq) : 0.0;
    if (parts != 1) {
#pragma unroll
        for (int i = 0; i < kFewParts; i += kClipThreads)
            all += i + (int)threadIdx.x < parts ? gld(sumsq + i + threadIdx.x) : 0.0;
        all = block_sum_f64(all, red);
    }
    const double n = sqrt(all);
    // (no limit: nothing is scaled, an infinite norm's gradients neither)
    const double want = n == n && max_norm == __builtin_huge_valf() ? 1.0 : (double)max_norm / (n + 1e-6);
    const float scale = want < 1.0 || want != want ? (float)want : 1.0f;
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) {
        gst(norm, (float)n);
        gst(scale_out, scale);
    }
    if (t.count == 0 || (t.in_place && scale == 1.0f)) return;
    // what was read last comes first: part of it is still in cache (112 matrices, 3.9 GB: 2115 us, 2129 in order)
    for (int64_t c = (int64_t)t.first[t.count] - 1 - blockIdx.x; c >= 0; c -= gridDim.x) {
        const int i = clip_find(t, (uint32_t)c);
        const int64_t at = (c - t.first[i]) * kClipChunk;
        const E* p = (const E*)t.src[i] + at;
        E* o = (E*)t.dst[i] + at;
        if (p == o && scale == 1.0f) continue;
        const int64_t left = t.size[i] - at;
        float v[kClipGroups][8];
#pragma unroll
        for (int k = 0; k < kClipGroups; ++k) {
            const int e = (k * kClipThreads + (int)threadIdx.x) * 8;
            clip_load(p + e, left - e, v[k]);
        }
#pragma unroll
        for (int k = 0; k < kClipGroups; ++k) {
            const int e = (k * kClipThreads + (int)threadIdx.x) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[k][j] *= scale;
            store8(o + e, left - e < 8 ? (int)(left - e < 0 ? 0 : left - e) : 8, v[k]);
        }
    }
}

namespace {
int64_t chunks_of(int64_t size) { return (size + kClipChunk - 1) / kClipChunk; }
// calls f(table) for tables of one type's tensors that are not empty; most: chunks of a table
template <typename F>
hipError_t each_table(const GradTensors& g, bool bf16, F f) {
    constexpr int64_t most = (int64_t)1 << 24;  // a launch holds fewer than 2^32 threads
    ClipTable t;
    t.count = 0;
    t.in_place = 1;
    t.first[0] = 0;
    auto flush = [&]() {
        const hipError_t e = t.count ? f(t) : hipSuccess;
        t.count = 0;
        t.in_place = 1;
        return e;
    };
    for (int i = 0; i < g.n; ++i) {
        if ((g.dtypes[i] == SC_BF16) != bf16) continue;
        const int64_t bytes = bf16 ? 2 : 4;
        for (int64_t at = 0; at < g.sizes[i];) {  // a tensor of more chunks than a table holds goes in parts
            int64_t size = g.sizes[i] - at;
            const int64_t room = (most - 1 - t.first[t.count]) * kClipChunk;
            if (room <= 0 || t.count == kClipTensors) {
                const hipError_t e = flush();
                if (e != hipSuccess) return e;
                continue;
            }
            if (size > room) size = room;
            t.src[t.count] = g.src ? (const char*)g.src[i] + at * bytes : nullptr;
            t.dst[t.count] = g.dst ? (char*)g.dst[i] + at * bytes : nullptr;
            t.size[t.count] = size;
            if (t.src[t.count] != t.dst[t.count]) t.in_place = 0;
            t.first[t.count + 1] = t.first[t.count] + (uint32_t)chunks_of(size);
            ++t.count;
            at += size;
        }
    }
    return flush();
}
int sumsq_grid(const ClipTable& t) {
    const uint32_t chunks = t.first[t.count];
    return (int)(chunks < (uint32_t)kSumsqGrid ? chunks : (uint32_t)kSumsqGrid);
}
}  // namespace

int64_t grad_sumsq_parts(const GradTensors& g) {
    int64_t parts = 0;
    for (int b = 0; b < 2; ++b)
        (void)each_table(g, b, [&](const ClipTable& t) {
            parts += sumsq_grid(t);
            return hipSuccess;
        });
    return parts;
}

// the partial sums, and how many
static hipError_t launch_parts(const GradTensors& g, double* part, int64_t& parts, hipStream_t st) {
    parts = 0;
    for (int b = 0; b < 2; ++b) {
        const hipError_t e = each_table(g, b, [&](const ClipTable& t) {
            const int grid = sumsq_grid(t);
            if (b) hipLaunchKernelGGL(sumsq_kernel<uint16_t>, dim3(grid), dim3(kClipThreads), 0, st, t, part + parts);
            else hipLaunchKernelGGL(sumsq_kernel<float>, dim3(grid), dim3(kClipThreads), 0, st, t, part + parts);
            parts += grid;
            return hipGetLastError();
        });
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_grad_sumsq(const GradTensors& g, double* sumsq, double* part, hipStream_t st) {
    int64_t parts;
    const hipError_t e = launch_parts(g, part, parts, st);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(sumsq_join_kernel, dim3(1), dim3(1024), 0, st, part, (int)parts, sumsq);
    return hipGetLastError();
}

hipError_t launch_clip_norm(const GradTensors& g, float max_norm, float* norm, float* scale, double* part,
                            hipStream_t st) {
    int64_t parts;
    hipError_t e = launch_parts(g, part, parts, st);
    if (e != hipSuccess) return e;
    if (parts > kFewParts) {
        hipLaunchKernelGGL(sumsq_join_kernel, dim3(1), dim3(1024), 0, st, part, (int)parts, part);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        parts = 1;
    }
    return launch_clip(g, part, (int)parts, max_norm, norm, scale, st);
}

hipError_t launch_clip(const GradTensors& g, const double* sumsq, int parts, float max_norm, float* norm, float* scale,
                       hipStream_t st) {
    bool told = false;
    for (int b = 0; b < 2; ++b) {
        const hipError_t e = each_table(g, b, [&](const ClipTable& t) {
            const uint32_t chunks = t.first[t.count];
            const dim3 grid(chunks < (uint32_t)kClipGrid ? chunks : (uint32_t)kClipGrid);
            float* to = told ? nullptr : norm;
            told = true;
            if (b) hipLaunchKernelGGL(clip_kernel<uint16_t>, grid, dim3(kClipThreads), 0, st, t, sumsq, parts, max_norm, to,
                                      scale);
            else hipLaunchKernelGGL(clip_kernel<float>, grid, dim3(kClipThreads), 0, st, t, sumsq, parts, max_norm, to,
                                    scale);
            return hipGetLastError();
        });
        if (e != hipSuccess) return e;
    }
    if (told) return hipSuccess;
    ClipTable none;  // no element at all: the norm is still told
    none.count = none.in_place = 0;
    none.first[0] = 0;
    hipLaunchKernelGGL(clip_kernel<float>, dim3(1), dim3(kClipThreads), 0, st, none, sumsq, parts, max_norm, norm,
                       scale);
    return hipGetLastError();
}

}  // namespace scopt
