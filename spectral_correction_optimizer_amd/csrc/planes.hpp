// Copies of operands' rows into bfloat16 planes.
#pragma once

#include "rows.hpp"

namespace scopt {

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

// 2^14 .. 2^15 of a row's largest finite magnitude: the exponent of the power of two that takes it there
__device__ __forceinline__ int half_exponent(float most) {
    const int e = (int)(__float_as_uint(most) >> 23) - 127;  // (a denormal number: -127, and the row stays small)
    return most > 0.0f ? min(14 - e, 126) : 0;
}
// x 2^e as two float16 values, h + l: off by at most 2^-22 of it or 2^-39 of the row's largest one.  An infinity is its
// own first value, beside 0.
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
__device__ __forceinline__ void split8_half(const float (&f)[8], int e, v8h& h, v8h& l) {
    const float unit = __uint_as_float((uint32_t)(e + 127) << 23);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = f[i] * unit;
        h[i] = (_Float16)x;
        l[i] = fabsf(x) == __builtin_huge_valf() ? (_Float16)0.0f : (_Float16)(x - (float)h[i]);
    }
}

// planes[p][at(r)][c]: kGroups groups of eight columns a thread (ld is a multiple of 8).  Where at(r) is negative the
// row of `cleared` (or NULL) is set to zeros instead; a row that is not live(r) is one of zeros.
template <typename E, int ENDS, typename At, typename Live>
__device__ __forceinline__ void planes_of_rows(const E* __restrict__ src, int64_t rows, int cols,
                                               uint16_t* __restrict__ dst, int64_t ld, int64_t plane,
                                               E* __restrict__ cleared, At at, Live is_live) {
    const int per_row = (int)(ld / 8);
    const int64_t n = rows * per_row;
    const bool small = n < (int64_t)1 << 31;
    for (int64_t g0 = (int64_t)blockIdx.x * 256 * kGroups + threadIdx.x; g0 < n;
         g0 += (int64_t)gridDim.x * 256 * kGroups) {
        Group8<E, ENDS> w[kGroups];
        int64_t r[kGroups], to[kGroups];
        int in[kGroups];
        bool live[kGroups];
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            const int64_t g = g0 + k * 256;
            split_group(g < n ? g : n - 1, per_row, small, r[k], in[k]);
            w[k].load(src + r[k] * cols, in[k] * 8, cols);
            live[k] = is_live(r[k]);
            to[k] = at(r[k]);
        }
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            if (g0 + k * 256 >= n) break;
            if (to[k] < 0) {
                const int c = in[k] * 8;
                const float none[8] = {};
                if (cleared && c < cols) store8(cleared + r[k] * cols + c, cols - c, none);
                continue;
            }
            uint16_t* o = dst + to[k] * ld + in[k] * 8;
            float f[8];
            value8(w[k], in[k] * 8, cols, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = live[k] ? f[i] : 0.0f;
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

}  // namespace scopt
