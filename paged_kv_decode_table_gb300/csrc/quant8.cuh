// quant8.cuh -- the 8-bit row format of the quantised KV cache.
//
// A cached K or V row (one token, one KV head, D values) is stored as D 8-bit
// values and one float32 scale:
//   scale = max(amax * (1 / Q), 2^-64),  value_i = rne(x_i * (1 / scale)),
//   x_i ~ value_i * scale,
// with Q the type's largest number: 448 for e4m3 (floating, 3 mantissa bits),
// 127 for int8.  Every operation above is a float32 operation rounded once, so
// the bytes are the same on every path that stores a row.  The scale is taken per
// row because a row is what a token writes and what attention reads as a whole:
// appending needs no other token's data, and in attention the K scale multiplies
// a score and the V scale a softmax weight, never a single element.  The floor
// 2^-64 keeps 1 / scale finite for rows that are all zero.  x_i * (1 / scale) can
// exceed Q by roundings of the scale and the product, which both conversions round
// back to Q.
// A row that holds a NaN or an infinity is stored as zeros with scale NaN.
#pragma once

#include "pkv_common.cuh"

namespace pkv {

constexpr float kMinScale = 5.421010862427522e-20f;  // 2^-64

// two floats <-> two halves, lo in bits 0-15
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t v) {
    float2 f;
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h;}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(v));
    return f;
}

// Two floats an instruction, each rounded.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long&>(r))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
    return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long&>(r))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<unsigned long long&>(r))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
          "l"(reinterpret_cast<unsigned long long&>(c)));
    return r;
}

struct FmtNone {  // rows kept in their own type
    static constexpr bool kQuant = false;
};

struct FmtE4M3 {
    static constexpr bool kQuant = true, kHasNaN = true;
    static constexpr float kInvQ = 1.0f / 448.0f;
    // two floats -> two bytes (lo in bits 0-7)
    static __device__ __forceinline__ uint32_t encode2(float lo, float hi) {
        uint16_t v;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(hi), "f"(lo));
        return v;
    }
    static __device__ __forceinline__ uint32_t encode4(const float* x) {
        return encode2(x[0], x[1]) | encode2(x[2], x[3]) << 16;
    }
    // bytes 0, 1 of v -> two halves (exact: every e4m3 number is a half)
    static __device__ __forceinline__ uint32_t decode2(uint16_t v) {
        uint32_t r;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
        return r;
    }
    // bytes (0, 1) and (2, 3) of v -> lo and hi
    static __device__ __forceinline__ void decode4(uint32_t v, uint32_t& lo, uint32_t& hi) {
        lo = decode2(static_cast<uint16_t>(v));
        hi = decode2(static_cast<uint16_t>(v >> 16));
    }
    // bytes (0, 2) and (1, 3) of v -> even and odd
    static __device__ __forceinline__ void decode4_pairs(uint32_t v, uint32_t& even, uint32_t& odd) {
        decode4(__byte_perm(v, 0u, 0x3120), even, odd);
    }
    static __device__ __forceinline__ float decode(uint8_t v) {
        const uint32_t h = decode2(v);
        float f;
        asm("{.reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.f32.f16 %0, lo;}" : "=f"(f) : "r"(h));
        return f;
    }
};

struct FmtI8 {
    static constexpr bool kQuant = true, kHasNaN = false;
    static constexpr float kInvQ = 1.0f / 127.0f;
    // |x| <= 127 (1 + 2^-22): adding 1.5 * 2^23 rounds to nearest even into the low byte
    static __device__ __forceinline__ uint32_t rounded(float x) { return __float_as_uint(__fadd_rn(x, 12582912.f)); }
    static __device__ __forceinline__ uint32_t encode2(float lo, float hi) {
        return __byte_perm(rounded(lo), rounded(hi), 0x0040) & 0xffffu;
    }
    static __device__ __forceinline__ uint32_t encode4(const float* x) {
        return __byte_perm(__byte_perm(rounded(x[0]), rounded(x[1]), 0x0040),
                           __byte_perm(rounded(x[2]), rounded(x[3]), 0x0040), 0x5410);
    }
    // x + 128 in the low byte of a half whose ulp is 1: 1024 + (x + 128), minus 1152
    static __device__ __forceinline__ uint32_t unbias(uint32_t h) {
        uint32_t r;
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(0x64806480u));
        return r;
    }
    static __device__ __forceinline__ void decode4(uint32_t v, uint32_t& lo, uint32_t& hi) {
        v ^= 0x80808080u;
        lo = unbias(__byte_perm(v, 0x64646464u, 0x4140));
        hi = unbias(__byte_perm(v, 0x64646464u, 0x4342));
    }
    static __device__ __forceinline__ void decode4_pairs(uint32_t v, uint32_t& even, uint32_t& odd) {
        v ^= 0x80808080u;
        even = unbias(__byte_perm(v, 0x64646464u, 0x4240));
        odd = unbias(__byte_perm(v, 0x64646464u, 0x4341));
    }
    static __device__ __forceinline__ float decode(uint8_t v) {
        return static_cast<float>(static_cast<int8_t>(v));
    }
};

__device__ __forceinline__ float row_scale(float amax, float inv_q) {
    return fmaxf(__fmul_rn(amax, inv_q), kMinScale);
}

}  // namespace pkv
