// Eight consecutive elements of a row of any alignment: rows of odd length start anywhere, and
// global loads and stores of gfx950 take any address, so a whole group is one access (two in
// float32) and only the group at a row's end goes by element.
#pragma once

#include "common.hpp"

namespace scopt {

typedef unsigned int v4u_any __attribute__((ext_vector_type(4), aligned(2)));
typedef float v4f_any __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned int v2u_any __attribute__((ext_vector_type(2), aligned(1)));

// `left` elements remain in the row; those beyond it read 0
__device__ __forceinline__ void load8(const uint16_t* p, int left, float (&v)[8]) {
    if (left >= 8) {
        const v4u_any w = *(const SC_GLOBAL v4u_any*)p;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(w[i]);
            v[2 * i + 1] = bf16_hi(w[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? bf16_to_f32(gld(p + i)) : 0.0f;
    }
}
__device__ __forceinline__ void load8(const float* p, int left, float (&v)[8]) {
    if (left >= 8) {
        const v4f_any a = *(const SC_GLOBAL v4f_any*)p, b = *(const SC_GLOBAL v4f_any*)(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? gld(p + i) : 0.0f;
    }
}
__device__ __forceinline__ void store8(uint16_t* p, int left, const float (&v)[8]) {
    if (left >= 8) {
        *(SC_GLOBAL v4u_any*)p = v4u_any{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                         pack_bf16x2(v[6], v[7])};
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) gst(p + i, f32_to_bf16(v[i]));
    }
}
__device__ __forceinline__ void store8(float* p, int left, const float (&v)[8]) {
    if (left >= 8) {
        *(SC_GLOBAL v4f_any*)p = v4f_any{v[0], v[1], v[2], v[3]};
        *(SC_GLOBAL v4f_any*)(p + 4) = v4f_any{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) gst(p + i, v[i]);
    }
}

// ---- 8-bit blocks: 32 elements of a row share the byte e = E + 127 ------------------------
constexpr int kActBlock = 32;
constexpr int kActMinExp = -120;
constexpr uint8_t kActNonFinite = 255;  // the block held a NaN or an infinity: it reads as NaN

// q and e of eight elements; the four lanes of a block share its largest magnitude
__device__ __forceinline__ void act_encode8(const float (&v)[8], int8_t (&q)[8], uint8_t& e) {
    uint32_t big = 0;  // magnitudes order like their bits
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t a = __float_as_uint(v[i]) & 0x7fffffffu;
        big = a > big ? a : big;
    }
    uint32_t o = __shfl_xor(big, 1);
    big = o > big ? o : big;
    o = __shfl_xor(big, 2);
    big = o > big ? o : big;
    int E = (int)(big >> 23) - 127;
    const bool finite = big < 0x7f800000u;
    E = E > kActMinExp ? E : kActMinExp;
    e = finite ? (uint8_t)(E + 127) : kActNonFinite;
    const float inv = __uint_as_float((uint32_t)(6 - E + 127) << 23);  // 2^(6 - E), E in [-120, 127]
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float r = rintf(v[i] * inv);  // the product is exact, ties to even
        q[i] = finite ? (int8_t)fminf(fmaxf(r, -127.0f), 127.0f) : (int8_t)0;
    }
}
__device__ __forceinline__ void store_q8(int8_t* p, int left, const int8_t (&q)[8]) {
    if (left >= 8) {
        v2u_any w;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = (uint32_t)(uint8_t)q[4 * i] | (uint32_t)(uint8_t)q[4 * i + 1] << 8 |
                   (uint32_t)(uint8_t)q[4 * i + 2] << 16 | (uint32_t)(uint8_t)q[4 * i + 3] << 24;
        *(SC_GLOBAL v2u_any*)p = w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) gst(p + i, q[i]);
    }
}
// the step 2^(e - 133) of a block; NaN for a block that was not finite
__device__ __forceinline__ float act_step(uint8_t e) {
    return e == kActNonFinite ? __builtin_nanf("") : ldexpf(1.0f, (int)e - 133);
}
__device__ __forceinline__ void load_q8(const int8_t* p, int left, float step, float (&v)[8]) {
    if (left >= 8) {
        const v2u_any w = *(const SC_GLOBAL v2u_any*)p;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)((int)(w[i / 4] << (24 - 8 * (i % 4))) >> 24) * step;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? (float)gld(p + i) * step : 0.0f;
    }
}

}  // namespace scopt
