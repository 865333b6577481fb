// Rows' log-sum-exps from their tiles' references and sums.
#pragma once

#include "common.hpp"
#include "train.hpp"

namespace scopt {

// A workgroup of 1024 threads and ROWS rows from `first`, one a lane (of ROWS), their tiles dealt to the 1024 / ROWS
// groups of lanes: lse of the rows before `end`, and tell(row, log-probability of the target).  A
// row of -infinity only has no finite log-sum-exp; like a row with NaN or +infinity it gives NaN.
template <int ROWS, typename Tell>
__device__ __forceinline__ void log_sums(const LogSums& a, int64_t end, int64_t first, float (*red)[ROWS], Tell tell) {
    constexpr int GROUPS = 1024 / ROWS;
    const int lane = threadIdx.x % ROWS, group = threadIdx.x / ROWS;
    const int64_t t = first + lane, at = t < end ? t : end - 1;
    const float none = -__builtin_huge_valf();
    // a difference of references as a factor; a tile of -infinity has sum 0 (or NaN)
    auto scaled = [&](float s, float r, float to) {
        return r == none ? s : s * (a.pow2 ? exp2f(r - to) : expf(r - to));
    };
    // some tiles' values in flight, joined to the running reference and sum
    float m = none, z = 0.0f;
    constexpr int U = ROWS == 64 ? 16 : 4;
    for (int i0 = group; i0 < a.tiles; i0 += GROUPS * U) {
        float r[U], s[U], top = m;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = i0 + GROUPS * u < a.tiles ? i0 + GROUPS * u : a.tiles - 1;
            r[u] = gld(a.smax + i * a.T + at);
            s[u] = gld(a.ssum + i * a.T + at);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) top = i0 + GROUPS * u < a.tiles ? fmaxf(top, r[u]) : top;
        z = scaled(z, m, top);
        m = top;
#pragma unroll
        for (int u = 0; u < U; ++u) z += i0 + GROUPS * u < a.tiles ? scaled(s[u], r[u], m) : 0.0f;
    }
    // the groups of a wavefront, then the wavefronts
    auto rescale = [&](float to) {
        z = scaled(z, m, to);
        m = to;
    };
    const int wave = threadIdx.x / 64;
    if constexpr (ROWS < 64) {
        float top = m;
#pragma unroll
        for (int o = ROWS; o < 64; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
        rescale(top);
#pragma unroll
        for (int o = ROWS; o < 64; o <<= 1) z += __shfl_xor(z, o);
    }
    if (threadIdx.x % 64 < ROWS) red[wave][lane] = m;
    __syncthreads();
    float top = none;
#pragma unroll
    for (int w = 0; w < 16; ++w) top = fmaxf(top, red[w][lane]);
    rescale(top);
    __syncthreads();
    if (threadIdx.x % 64 < ROWS) red[wave][lane] = z;
    __syncthreads();
    if (threadIdx.x >= ROWS || t >= end) return;
    z = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) z += red[w][lane];
    if constexpr (ROWS < 64) {
        // Losses add up log-probabilities of many tokens, and float32's logarithm is low by 3e-7 on the average at such
        // sums (300 to 1100), as much as a rounding of the result.
        const double base = a.pow2 ? m * 0.693147180559945309417 : (double)m;
        const double l = m == none ? __builtin_nan("") : base + log((double)z);
        gst(a.lse + t, (float)l);
        tell(t, (float)((double)gld(a.target_logit + t) - l));
        return;
    }
    // a power of two's logarithm in two parts: m * ln2 is off by less than 2^-40 of m
    const float base = a.pow2 ? m * 0.693145751953125f : m, rest = a.pow2 ? m * 1.42860682030941723e-6f : 0.0f;
    const float logz = m == none ? __builtin_nanf("") : logf(z) + rest;
    gst(a.lse + t, base + logz);
    tell(t, -((base - gld(a.target_logit + t)) + logz));
}

}  // namespace scopt
