// Row formats of the banks, by 16-byte pieces: how a piece unpacks to float32 columns, and how a
// scale group of columns is quantised.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "sdm.h"
#include "sdm_device.cuh"

namespace sdm {

// A format has C columns in a 16-byte piece; unpack() gives their values without the scale, pack()
// rounds values that are already divided by the scale. Every scale group (32, 64 or 128 columns) is
// a whole number of pieces.

// Integer to float32 without the conversion unit (half rate): the byte, offset to be unsigned, goes
// into the mantissa of 2^23, and the offset is subtracted exactly.
struct Int8 {
    static constexpr int C = 16;
    static constexpr bool kQuantised = true;
    static constexpr float kLevels = 127.0f;
    static __device__ __forceinline__ void unpack(const uint4& v, float* x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t u = w[i] ^ 0x80808080u;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[4 * i + j] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440u + j)) - 8388736.0f;
        }
    }
    static __device__ __forceinline__ uint4 pack(const float* y) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // saturating pack of two integers above the two packed before
            const int a = __float2int_rn(y[4 * i]), b = __float2int_rn(y[4 * i + 1]), c = __float2int_rn(y[4 * i + 2]),
                      d = __float2int_rn(y[4 * i + 3]);
            uint32_t hi;
            asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, 0;" : "=r"(hi) : "r"(d), "r"(c));
            asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(w[i]) : "r"(b), "r"(a), "r"(hi));
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

struct Fp8 {
    static constexpr int C = 16;
    static constexpr bool kQuantised = true;
    static constexpr float kLevels = 448.0f;
    static __device__ __forceinline__ void unpack(const uint4& v, float* x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint16_t two = (uint16_t)(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu);
            uint32_t h;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
            asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %2; cvt.f32.f16 %0, lo; cvt.f32.f16 %1, hi; }"
                : "=f"(x[2 * i]), "=f"(x[2 * i + 1])
                : "r"(h));
        }
    }
    static __device__ __forceinline__ uint4 pack(const float* y) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint16_t lo, hi;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(y[4 * i + 1]), "f"(y[4 * i]));
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(y[4 * i + 3]), "f"(y[4 * i + 2]));
            w[i] = (uint32_t)lo | ((uint32_t)hi << 16);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

struct Int4 {
    static constexpr int C = 32;
    static constexpr bool kQuantised = true;
    static constexpr float kLevels = 7.0f;
    static __device__ __forceinline__ void unpack(const uint4& v, float* x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t u = w[i] ^ 0x88888888u;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[8 * i + j] = __uint_as_float(((u >> (4 * j)) & 15u) | 0x4B000000u) - 8388616.0f;
        }
    }
    static __device__ __forceinline__ uint4 pack(const float* y) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int q = max(-7, min(7, __float2int_rn(y[8 * i + j])));
                w[i] |= ((uint32_t)q & 15u) << (4 * j);
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

struct Bf16 {
    static constexpr int C = 8;
    static constexpr bool kQuantised = false;
    using E = uint16_t;
    static __device__ __forceinline__ void unpack(const uint4& v, float* x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};

struct F32 {
    static constexpr int C = 4;
    static constexpr bool kQuantised = false;
    using E = float;
    static __device__ __forceinline__ void unpack(const uint4& v, float* x) {
        x[0] = __uint_as_float(v.x);
        x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z);
        x[3] = __uint_as_float(v.w);
    }
};

// Bits of |x|: as unsigned integers they order like |x|, with infinity above every number and NaN
// above infinity, so that one maximum finds the largest magnitude and any non-finite value.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The scale of a group whose largest magnitude has the bits m, and the factor `inv` its values are
// multiplied with before rounding (0: codes of zero). Groups below 2^-100 become zeros, since the
// factor would overflow for subnormal magnitudes; a non-finite group gets the scale NaN.
template <typename F>
__device__ __forceinline__ float group_scale(uint32_t m, float* inv) {
    constexpr uint32_t kTiny = 0x0D800000u;  // 2^-100
    *inv = 0.0f;
    if (m >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
    if (m < kTiny) return 0.0f;
    const float top = __uint_as_float(m);
    *inv = __fdiv_rn(F::kLevels, top);
    return __fdiv_rn(top, F::kLevels);
}

// Quantise this lane's C columns of a row whose groups lie on `lanes` neighbouring lanes each (a
// power of two, aligned): the piece of codes, and the group's scale on every one of its lanes.
template <typename F>
__device__ __forceinline__ uint4 quantise_piece(const float* x, int lanes, float* scale) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < F::C; ++i) m = max(m, abs_bits(x[i]));
    for (int o = 1; o < lanes; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    float inv;
    *scale = group_scale<F>(m, &inv);
    float y[F::C];
#pragma unroll
    for (int i = 0; i < F::C; ++i) y[i] = inv > 0.0f ? x[i] * inv : 0.0f;
    return F::pack(y);
}

}  // namespace sdm
