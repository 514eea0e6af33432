// Row formats of the banks, by 16-byte pieces: how a piece unpacks to float32 columns, and how a
// scale group of columns is quantised.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "sdm.h"
#include "sdm_device.cuh"

namespace sdm {

// ---------------------------------------------------------------- loads and stores that may be left out
// A load of bank memory where `on`, zeros elsewhere, without a branch: loads in branches wait for one
// another where loads of a batch should be on their way together. Stores likewise.

__device__ __forceinline__ uint4 load16_if(const void* p, bool on) {
    uint4 r;
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@q ld.global.cg.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(r.x), "=&r"(r.y), "=&r"(r.z), "=&r"(r.w)
        : "l"(p), "r"((int)on)
        : "memory");
    return r;
}
__device__ __forceinline__ float load4_if(const float* p, bool on) {
    float r;
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\tmov.b32 %0, 0;\n\t@q ld.global.cg.b32 %0, [%1];\n\t}"
                 : "=&f"(r)
                 : "l"(p), "r"((int)on)
                 : "memory");
    return r;
}

__device__ __forceinline__ void store16_if(void* p, const uint4& v, bool on) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t@q st.global.v4.b32 [%4], {%0, %1, %2, %3};\n\t}" ::"r"(v.x), "r"(v.y),
                 "r"(v.z), "r"(v.w), "l"(p), "r"((int)on)
                 : "memory");
}
__device__ __forceinline__ void store4_if(float* p, float v, bool on) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t@q st.global.b32 [%1], %0;\n\t}" ::"f"(v), "l"(p), "r"((int)on)
                 : "memory");
}

// ---------------------------------------------------------------- pairs of float32
// Two columns in one 64-bit register for the packed float32 instructions, which round like their
// scalar forms at twice the rate.

using f32x2 = uint64_t;

__device__ __forceinline__ f32x2 pair(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void split(f32x2 p, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p)); }
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// ---------------------------------------------------------------- formats
// A format has C columns in a 16-byte piece; unpack2() gives their values without the scale, in
// pairs, and pack2() rounds values that are already divided by the scale. Every scale group (32, 64
// or 128 columns) is a whole number of pieces.
//
// Integers pass to and from float32 without the conversion unit (a quarter of the rate): a byte,
// offset to be unsigned, goes into the mantissa of 2^23, and the offset is subtracted exactly; the
// other way, adding 1.5 * 2^23 rounds to the nearest even integer and leaves it in the low bits.
__device__ __forceinline__ uint32_t round_bits(float y) {
    // the scalar sum: a packed sum behind a packed product is contracted with it, which rounds once
    // where the format's definition rounds twice
    return __float_as_uint(__fadd_rn(y, 12582912.0f));
}

template <typename F>
__device__ __forceinline__ void unpack(const uint4& v, float* x) {
    f32x2 p[F::C / 2];
    F::unpack2(v, p);
#pragma unroll
    for (int i = 0; i < F::C / 2; ++i) split(p[i], x[2 * i], x[2 * i + 1]);
}

struct Int8 {
    static constexpr int C = 16;
    static constexpr bool kQuantised = true;
    static constexpr float kLevels = 127.0f;
    static constexpr float kInvHigh = 0x1.020408p-7f, kInvLow = 0x1.020408p-35f;  // 1 / 127
    static __device__ __forceinline__ void unpack2(const uint4& v, f32x2* x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        const f32x2 off = pair(-8388736.0f, -8388736.0f);  // -(2^23 + 128)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t u = w[i] ^ 0x80808080u;
#pragma unroll
            for (int j = 0; j < 2; ++j)
                x[2 * i + j] = add2(pair(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440u + 2 * j)),
                                         __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7441u + 2 * j))),
                                    off);
        }
    }
    static __device__ __forceinline__ uint4 pack2(const f32x2* y) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b, c, d;
            split(y[2 * i], a, b);
            split(y[2 * i + 1], c, d);
            w[i] = __byte_perm(__byte_perm(round_bits(a), round_bits(b), 0x0040u), __byte_perm(round_bits(c), round_bits(d), 0x0040u),
                               0x5410u);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

struct Fp8 {
    static constexpr int C = 16;
    static constexpr bool kQuantised = true;
    static constexpr float kLevels = 448.0f;
    static constexpr float kInvHigh = 0x1.24924ap-9f, kInvLow = -0x1.b6db6ep-34f;  // 1 / 448
    static __device__ __forceinline__ void unpack2(const uint4& v, f32x2* x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint16_t two = (uint16_t)(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu);
            uint32_t h;
            float lo, hi;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
            asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h; }" : "=f"(lo), "=f"(hi) : "r"(h));
            x[i] = pair(lo, hi);
        }
    }
    static __device__ __forceinline__ uint4 pack2(const f32x2* y) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b, c, d;
            split(y[2 * i], a, b);
            split(y[2 * i + 1], c, d);
            uint16_t lo, hi;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
            w[i] = (uint32_t)lo | ((uint32_t)hi << 16);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

struct Int4 {
    static constexpr int C = 32;
    static constexpr bool kQuantised = true;
    static constexpr float kLevels = 7.0f;
    static constexpr float kInvHigh = 0x1.24924ap-3f, kInvLow = -0x1.b6db6ep-28f;  // 1 / 7
    static __device__ __forceinline__ void unpack_word(uint32_t w, f32x2* x) {  // 8 columns
        const f32x2 off = pair(-8388616.0f, -8388616.0f);  // -(2^23 + 8)
        const uint32_t u = w ^ 0x88888888u;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            x[j] = add2(pair(__uint_as_float(((u >> (8 * j)) & 15u) | 0x4B000000u),
                             __uint_as_float(((u >> (8 * j + 4)) & 15u) | 0x4B000000u)),
                        off);
    }
    static __device__ __forceinline__ uint32_t pack_word(const f32x2* y) {
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float a, b;
            split(y[j], a, b);
            w |= (round_bits(a) & 15u) << (8 * j) | (round_bits(b) & 15u) << (8 * j + 4);
        }
        return w;
    }
    static __device__ __forceinline__ void unpack2(const uint4& v, f32x2* x) {
        unpack_word(v.x, x);
        unpack_word(v.y, x + 4);
        unpack_word(v.z, x + 8);
        unpack_word(v.w, x + 12);
    }
};

struct Bf16 {
    static constexpr int C = 8;
    static constexpr bool kQuantised = false;
    using E = uint16_t;
    static __device__ __forceinline__ void unpack2(const uint4& v, f32x2* x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
};

struct F32 {
    static constexpr int C = 4;
    static constexpr bool kQuantised = false;
    using E = float;
    static __device__ __forceinline__ void unpack2(const uint4& v, f32x2* x) {
        x[0] = pair(__uint_as_float(v.x), __uint_as_float(v.y));
        x[1] = pair(__uint_as_float(v.z), __uint_as_float(v.w));
    }
};

// The largest of three magnitudes; NaN if there is one among them.
__device__ __forceinline__ float abs_max(float m, float a, float b) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a), "f"(b));
    return r;
}

// L / x, correctly rounded, for the normal x that a group's largest magnitude can be (2^-100 and up),
// without a branch: a division's rare path keeps the rows around it from overlapping. Markstein's
// method: the reciprocal, corrected by its own residual, then the quotient by its; both residuals are
// exact in a fused multiply-add. Large x are scaled so that the reciprocal stays normal.
__device__ __forceinline__ float levels_over(float levels, float x) {
    const float f = x > 0x1p64f ? 0x1p-64f : 1.0f;
    const float y = x * f;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
    r = fmaf(fmaf(-y, r, 1.0f), r, r);
    const float q = __fmul_rn(levels, r);
    return fmaf(fmaf(-y, q, levels), r, q) * f;
}

// The scale of a group whose largest magnitude is `top`, and the factor `inv` its values are
// multiplied with before rounding (0: codes of zero). Groups below 2^-100 become zeros, since the
// factor would overflow for subnormal magnitudes; a non-finite group gets the scale NaN.
template <typename F>
__device__ __forceinline__ float group_scale(float top, float* inv) {
    const bool finite = top <= 3.402823466e38f, some = top >= 7.888609052e-31f;  // 2^-100
    *inv = finite && some ? levels_over(F::kLevels, top) : 0.0f;
    // top / L correctly rounded in two operations, since L is known (Brisebarre, Muller: 1 / L as the
    // sum of two floats; the tests compare every significand, and every exponent, with a division)
    const float scale = fmaf(F::kInvHigh, top, __fmul_rn(F::kInvLow, top));
    return !finite ? __uint_as_float(0x7fc00000u) : some ? scale : 0.0f;
}

// The largest magnitude of this lane's C columns.
template <int C>
__device__ __forceinline__ float piece_top(const f32x2* x) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < C / 2; ++i) {
        float a, b;
        split(x[i], a, b);
        top = abs_max(top, a, b);
    }
    return top;
}

// From the largest magnitudes of N rows' pieces to the scales of their groups, which lie on `lanes`
// neighbouring lanes each (a power of two up to 8, aligned), and the factors to the codes.
template <typename F, int N>
__device__ __forceinline__ void group_scales(const float* top, int lanes, float* scale, float* inv) {
    uint32_t m[N];
#pragma unroll
    for (int n = 0; n < N; ++n) m[n] = __float_as_uint(top[n]) & 0x7fffffffu;  // they order like their bits, NaN above infinity
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const uint32_t other = __shfl_xor_sync(0xffffffffu, m[n], o);
            m[n] = o < lanes ? max(m[n], other) : m[n];
        }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) scale[n] = group_scale<F>(__uint_as_float(m[n]), &inv[n]);
}

// Codes of a piece with the factor of its group.
template <typename F>
__device__ __forceinline__ uint4 pack_piece(f32x2* x, float inv) {
    const f32x2 f = pair(inv, inv);
#pragma unroll
    for (int i = 0; i < F::C / 2; ++i) x[i] = mul2(x[i], f);
    const uint4 c = F::pack2(x);
    return inv > 0.0f ? c : make_uint4(0u, 0u, 0u, 0u);
}

}  // namespace sdm
