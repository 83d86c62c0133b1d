// Arithmetic shared by the block-128 kernels: the scale rule, code conversion
// of four values, gate activations, packed fp32 pairs.
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

#include "fp8gemm.h"
#include "quant_math.cuh"

namespace fp8g {

// Scale of a block from its largest magnitude (not NaN): amax / largest value of
// the format, at least 2^-126 so that its reciprocal is finite, 1 for zeros.  A
// block with an infinity has an infinite scale and NaN products.
template <int FMT>
__device__ __forceinline__ float b128_scale(float amax) {
    const float s = __fdiv_rn(amax, Fp8Fmt<FMT>::kMax);
    return s == 0.0f && amax == 0.0f ? 1.0f : fmaxf(s, 1.17549435e-38f);
}

// Packed pairs of fp32 (lo first).
__device__ __forceinline__ uint64_t b128_pair(float lo, float hi) {
    return (uint64_t)__float_as_uint(lo) | ((uint64_t)__float_as_uint(hi) << 32);
}
__device__ __forceinline__ uint64_t b128_pair(uint32_t lo, uint32_t hi) {
    return (uint64_t)lo | ((uint64_t)hi << 32);
}
__device__ __forceinline__ float b128_lo(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float b128_hi(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
// d += a b
__device__ __forceinline__ void b128_fma2(uint64_t &d, uint64_t a, uint64_t b) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}
__device__ __forceinline__ uint64_t b128_mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ uint64_t b128_add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t b128_madd2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// Codes of four values, first value lowest; NaN gives the code 0x7F.
template <int FMT>
__device__ __forceinline__ uint32_t b128_cvt4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    if constexpr (FMT == 0) {
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    } else {
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    }
    return (uint32_t)lo | ((uint32_t)hi << 16);
}
template <int FMT>
__device__ __forceinline__ uint32_t b128_codes(float a, float b, float c, float d, float r) {
    const uint64_t rr = b128_pair(r, r), x = b128_mul2(b128_pair(a, b), rr), y = b128_mul2(b128_pair(c, d), rr);
    return b128_cvt4<FMT>(b128_lo(x), b128_hi(x), b128_lo(y), b128_hi(y));
}
template <int FMT>
__device__ __forceinline__ uint32_t b128_codes4(const float (&v)[4], const float (&r)[4]) {
    const uint64_t x = b128_mul2(b128_pair(v[0], v[1]), b128_pair(r[0], r[1]));
    const uint64_t y = b128_mul2(b128_pair(v[2], v[3]), b128_pair(r[2], r[3]));
    return b128_cvt4<FMT>(b128_lo(x), b128_hi(x), b128_lo(y), b128_hi(y));
}

// Four codes -> fp32 (exact).
__device__ __forceinline__ void b128_decode(uint32_t q, int fmt, float (&v)[4]) {
    uint32_t lo, hi;
    if (fmt == FP8G_E4M3) {
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"((uint16_t)q));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"((uint16_t)(q >> 16)));
    } else {
        asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(lo) : "h"((uint16_t)q));
        asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(hi) : "h"((uint16_t)(q >> 16)));
    }
    const uint32_t w[2] = {lo, hi};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
            : "=f"(v[2 * i]), "=f"(v[2 * i + 1])
            : "r"(w[i]));
    }
}

// Larger of m (not NaN) and two magnitudes; NaN does not count.
__device__ __forceinline__ float b128_max3(float m, float a, float b) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(fabsf(a)), "f"(fabsf(b)));
    return r;
}
// Largest magnitude of four values; NaN counts as 0.
__device__ __forceinline__ float b128_amax4(float a, float b, float c, float d) {
    return b128_max3(b128_max3(0.0f, a, b), c, d);
}

// Largest of the warp's values (>= 0, not NaN: their bits are in order).
__device__ __forceinline__ float b128_warp_max(float v) {
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}

// Base-2 exponential and reciprocal of two values, the hardware's (relative errors 2^-22 and 2^-23;
// subnormal results are 0).
__device__ __forceinline__ uint64_t b128_exp2_2(uint64_t v) {
    float a, b;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(b128_lo(v)));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(b128_hi(v)));
    return b128_pair(a, b);
}
__device__ __forceinline__ uint64_t b128_rcp2(uint64_t v) {
    float a, b;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(b128_lo(v)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(b128_hi(v)));
    return b128_pair(a, b);
}
__device__ __forceinline__ uint64_t b128_two(float v) { return b128_pair(v, v); }

// 1 / (1 + e^-g) of two values (relative error about 2^-22 (1 + |g| / 4), beside the 2^-4 of the
// codes that it ends in; the exact division took the gated epilogue twice the instructions, and
// subnormal numbers, flushed here, change no sum with 1; a sigmoid below 2^-126 is 0).
__device__ __forceinline__ uint64_t b128_sigmoid2(uint64_t g) {
    return b128_rcp2(b128_add2(b128_exp2_2(b128_mul2(g, b128_two(-1.4426950408889634f))), b128_two(1.0f)));
}

// Phi(g) of two values, and e = e^(-g^2 / 2).  A block of values is coded relative to its own
// largest, so the tail has to keep its digits: 1 + erf(g / sqrt 2) has one left at g = -5 and none
// from -5.5 on.  Hastings's form, Phi(-x) = e^(-x^2 / 2) t P(t) with t = 1 / (1 + p x), keeps them all;
// p and P (degree 7) are a minimax fit of relative error 2^-23 over 0 <= x <= 13.4, beyond which e
// is 0.  With the roundings (19 + 1.5 g^2) 2^-24 of Phi at most.  Backward 4099 x 14336 127 us, gated
// 4099 x 14336 x 4096 with the checkpoint 427 (with erfcf in its place 192 and 505).
__device__ __forceinline__ uint64_t b128_phi2(uint64_t g, uint64_t &e) {
    const uint64_t one = b128_two(1.0f), x = g & 0x7FFFFFFF7FFFFFFFull;
    e = b128_exp2_2(b128_mul2(b128_mul2(g, g), b128_two(-0.72134752044448170f)));
    const uint64_t t = b128_rcp2(b128_madd2(x, b128_two(0.305f), one));
    constexpr float c[8] = {0.121639736f,   0.122466817f, 0.103420876f,  0.121021651f,
                            -0.037976779f, 0.185716838f, -0.152988285f, 0.036699187f};
    uint64_t v = b128_two(c[7]);
#pragma unroll
    for (int k = 6; k >= 0; --k) v = b128_madd2(v, t, b128_two(c[k]));
    const uint64_t q = b128_mul2(b128_mul2(v, t), e), rest = b128_madd2(q, b128_two(-1.0f), one);
    return b128_pair(b128_lo(g) < 0.0f ? b128_lo(q) : b128_lo(rest), b128_hi(g) < 0.0f ? b128_hi(q) : b128_hi(rest));
}

// The activation of two values; its value and derivative.
template <int GATE>
__device__ __forceinline__ uint64_t b128_gate2(uint64_t g) {
    if constexpr (GATE == FP8G_GATE_SILU) return b128_mul2(g, b128_sigmoid2(g));
    if constexpr (GATE == FP8G_GATE_GELU) {
        uint64_t e;
        return b128_mul2(g, b128_phi2(g, e));
    }
    const float a = b128_lo(g), b = b128_hi(g);
    return b128_pair(a < 0.0f ? 0.0f : a, b < 0.0f ? 0.0f : b);
}
template <int GATE>
__device__ __forceinline__ void b128_gate_grad2(uint64_t g, uint64_t &y, uint64_t &d) {
    if constexpr (GATE == FP8G_GATE_SILU) {
        const uint64_t one = b128_two(1.0f), s = b128_sigmoid2(g);
        y = b128_mul2(g, s);
        const uint64_t rest = b128_madd2(s, b128_two(-1.0f), one);  // 1 - s, rounded once
        d = b128_mul2(s, b128_madd2(g, rest, one));
    } else if constexpr (GATE == FP8G_GATE_GELU) {
        uint64_t e;
        const uint64_t c = b128_phi2(g, e);
        y = b128_mul2(g, c);
        d = b128_madd2(b128_mul2(g, e), b128_two(0.39894228040143268f), c);
    } else {
        y = b128_gate2<GATE>(g);
        const float a = b128_lo(g), b = b128_hi(g);
        d = b128_pair(a > 0.0f ? 1.0f : (isnan(a) ? a : 0.0f), b > 0.0f ? 1.0f : (isnan(b) ? b : 0.0f));
    }
}

}  // namespace fp8g
