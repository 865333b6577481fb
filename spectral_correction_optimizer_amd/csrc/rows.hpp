// Eight consecutive elements of a row of any alignment: rows of odd length start anywhere, and
// global loads and stores of gfx950 take any address, so a whole group is one access (two in
// float32).
//
// Loads have no branches: a branch around a load makes the wave wait for each one before the
// next is issued (the residual norm of 32 x 2048 took 7.2 us that way).  A group that would
// pass the row's end is fetched from the row's last eight elements and shifted into place,
// and a group beyond the row reads zeros; rows shorter than eight go by element.
#pragma once

#include "common.hpp"

namespace scopt {

typedef unsigned int v4u_any __attribute__((ext_vector_type(4), aligned(2)));
typedef float v4f_any __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned int v2u_any __attribute__((ext_vector_type(2), aligned(1)));

// How a row of H elements is cut into groups of eight.
enum RowEnds {
    ROW_WHOLE = 0,  // H % 8 = 0
    ROW_CUT = 1,    // H > 8, the last group is cut
    ROW_SHORT = 2,  // H < 8: one cut group
};
inline RowEnds row_ends(int64_t H) { return H % 8 == 0 ? ROW_WHOLE : H > 8 ? ROW_CUT : ROW_SHORT; }

// A group as it was fetched; value() is called where the values are needed, after other
// groups' loads have been issued.
template <typename E, int ENDS> struct Group8;
template <int ENDS> struct Group8<uint16_t, ENDS> {
    v4u w;
    __device__ __forceinline__ void load(const uint16_t* row, int c, int H) {
        if constexpr (ENDS == ROW_SHORT) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = (uint32_t)gld(row + min(2 * i, H - 1)) | (uint32_t)gld(row + min(2 * i + 1, H - 1)) << 16;
        } else {
            w = *(const SC_GLOBAL v4u_any*)(row + min(c, H - 8));
        }
    }
    __device__ __forceinline__ void arrived() { asm volatile("" : "+v"(w) : : "memory"); }  // waits for the load
    __device__ __forceinline__ void raw(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(w[i]);
            v[2 * i + 1] = bf16_hi(w[i]);
        }
    }
};
template <int ENDS> struct Group8<float, ENDS> {
    v4f a, b;
    __device__ __forceinline__ void load(const float* row, int c, int H) {
        if constexpr (ENDS == ROW_SHORT) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = gld(row + min(i, H - 1));
                b[i] = gld(row + min(4 + i, H - 1));
            }
        } else {
            const float* p = row + min(c, H - 8);
            a = *(const SC_GLOBAL v4f_any*)p;
            b = *(const SC_GLOBAL v4f_any*)(p + 4);
        }
    }
    __device__ __forceinline__ void arrived() { asm volatile("" : "+v"(a), "+v"(b) : : "memory"); }
    __device__ __forceinline__ void raw(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    }
};
// the values of the group at column c: zeros beyond the row
template <typename E, int ENDS>
__device__ __forceinline__ void value8(const Group8<E, ENDS>& g, int c, int H, float (&v)[8]) {
    g.raw(v);
    if constexpr (ENDS == ROW_WHOLE) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c < H ? v[i] : 0.0f;
    } else if constexpr (ENDS == ROW_CUT) {
        const int s = c - min(c, H - 8);  // fetched that many elements early
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = s & 4 ? (i < 4 ? v[i + 4] : 0.0f) : v[i];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = s & 2 ? (i < 6 ? v[i + 2] : 0.0f) : v[i];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = s & 1 ? (i < 7 ? v[i + 1] : 0.0f) : v[i];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = s < 8 ? v[i] : 0.0f;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c + i < H ? v[i] : 0.0f;
    }
}
template <int ENDS, typename E>
__device__ __forceinline__ void load8(const E* row, int c, int H, float (&v)[8]) {
    Group8<E, ENDS> g;
    g.load(row, c, H);
    value8(g, c, H, v);
}
// `left` elements remain in the row
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

// Elementwise kernels: groups of 8 of a thread, 256 groups apart; their loads are in flight
// together.
constexpr int kGroups = 4;
// row and group of a flat group index; 32-bit division where it serves
__device__ __forceinline__ void split_group(int64_t g, int per_row, bool small, int64_t& t, int& in) {
    if (small) {
        const uint32_t r = (uint32_t)g / (uint32_t)per_row;
        t = r;
        in = (int)((uint32_t)g - r * (uint32_t)per_row);
    } else {
        t = g / per_row;
        in = (int)(g - t * per_row);
    }
}

// calls X(E, ENDS) of the element type and the rows' ends
#define SC_BY_ENDS(bf16, H, X)                                                                  \
    switch (row_ends(H)) {                                                                      \
        case ROW_WHOLE: if (bf16) { X(uint16_t, ROW_WHOLE) } else { X(float, ROW_WHOLE) } break; \
        case ROW_CUT: if (bf16) { X(uint16_t, ROW_CUT) } else { X(float, ROW_CUT) } break;       \
        case ROW_SHORT: if (bf16) { X(uint16_t, ROW_SHORT) } else { X(float, ROW_SHORT) } break; \
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
// The same for values in 64 bits: the largest magnitude's exponent is that of its high words.
__device__ __forceinline__ void act_encode8(const double (&v)[8], int8_t (&q)[8], uint8_t& e) {
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t a = (uint32_t)(__double_as_longlong(v[i]) >> 32) & 0x7fffffffu;
        big = a > big ? a : big;
    }
    uint32_t o = __shfl_xor(big, 1);
    big = o > big ? o : big;
    o = __shfl_xor(big, 2);
    big = o > big ? o : big;
    int E = (int)(big >> 20) - 1023;
    const bool finite = E <= 127;
    E = E > kActMinExp ? E : kActMinExp;
    e = finite ? (uint8_t)(E + 127) : kActNonFinite;
    const double inv = __longlong_as_double((long long)(6 - E + 1023) << 52);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const double r = rint(v[i] * inv);
        q[i] = finite ? (int8_t)fminf(fmaxf((float)r, -127.0f), 127.0f) : (int8_t)0;
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
// the step 2^(e - 133) of a block, a denormal number below e = 7; NaN for a block that was not
// finite
__device__ __forceinline__ float act_step(uint32_t e) {
    const uint32_t bits = e >= 7 ? (e - 6) << 23 : 1u << (e + 16);
    return __uint_as_float(e == kActNonFinite ? 0x7fc00000u : bits);
}
// Eight 8-bit elements and their block's byte, as fetched.
template <int ENDS> struct GroupQ8 {
    v2u w;
    uint32_t e;
    __device__ __forceinline__ void load(const int8_t* row, const uint8_t* erow, int c, int H) {
        e = gld(erow + min(c, H - 1) / kActBlock);
        if constexpr (ENDS == ROW_SHORT) {
            w = v2u{0u, 0u};
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i / 4] |= (uint32_t)(uint8_t)gld(row + min(i, H - 1)) << (8 * (i % 4));
        } else {
            w = *(const SC_GLOBAL v2u_any*)(row + min(c, H - 8));
        }
    }
    __device__ __forceinline__ void value(int c, int H, float (&v)[8]) const {
        uint64_t x = (uint64_t)w[1] << 32 | w[0];
        if constexpr (ENDS == ROW_SHORT) {
            x = c < H ? x & ~0ull >> (64 - 8 * H) : 0;
        } else {
            const int s = c - min(c, H - 8);
            x = s < 8 ? x >> (8 * s) : 0;  // ROW_WHOLE: 0 or beyond the row
        }
        const float step = c < H ? act_step(e) : 0.0f;
        const uint32_t u[2] = {(uint32_t)x, (uint32_t)(x >> 32)};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float f = (float)((int)(u[i / 4] << (24 - 8 * (i % 4))) >> 24);
            v[i] = ENDS == ROW_WHOLE || c + i < H ? f * step : 0.0f;
        }
    }
};

}  // namespace scopt
