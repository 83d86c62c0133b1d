// One value of the projection with adapters, by a warp from the operands in
// memory, for the kernels' epilogues.
//
// A low-rank step of the MMA takes an adapter's B against token columns (or rows)
// of which some are other adapters': V is zero there, and a zero times a finite
// value adds nothing.  A B that is infinite or NaN adds NaN.  So a NaN that an
// epilogue has stored is computed here again, as
//   sum_k (sx x)(sw w) + sum_j V_j B_j
// of its own row, adapter and feature, and stays NaN only where that is one.  A
// finite B costs the epilogues a comparison a value or less.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "stream.h"

namespace fp8g {

// The values of two codes of format fmt: of the low and of the next byte (E2M1:
// of the two nibbles of the low byte).
__device__ __forceinline__ float2 code_values(uint32_t c, int fmt) {
    uint32_t h;
    const uint16_t s = (uint16_t)c;
    if (fmt == FP8G_E4M3)
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(s));
    else if (fmt == FP8G_E5M2)
        asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"(s));
    else if (fmt == FP8G_E2M1)
        asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(h) : "r"(c));
    else if (fmt == FP8G_E2M3)
        asm("cvt.rn.f16x2.e2m3x2 %0, %1;" : "=r"(h) : "h"(s));
    else
        asm("cvt.rn.f16x2.e3m2x2 %0, %1;" : "=r"(h) : "h"(s));
    return __half22float2(*reinterpret_cast<__half2 *>(&h));
}

// The operands of a value.
struct LoraValue {
    const uint8_t *x, *w;        // codes of the row (E4M3) and of the feature (fmt)
    const uint8_t *sfx, *sfw;    // their bytes in the first chunk of packed scales
    int64_t sfx_step, sfw_step;  // bytes between chunks
    int32_t K, fmt, rank;        // rank 0: the row has no adapter
    int32_t pieces, per;         // V: LoraV, values of a block of rows, the row's first pieces
    int64_t block;
    const __nv_bfloat16 *v;
    const __nv_bfloat16 *b;      // the feature's row of B
};

// Byte of row r (of a 128-row tile) in a chunk of packed scales, block 0.
__device__ __forceinline__ int scale_byte(int64_t r) { return 16 * (int)(r & 31) + 4 * (int)(r >> 5 & 3); }

__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// By all lanes of a warp, o the same in each; the value in each.
static __device__ __noinline__ float lora_value(const LoraValue &o) {
    const int lane = threadIdx.x & 31;
    float low = 0.0f;
    for (int j = lane; j < o.rank; j += 32) {
        // (V was written by other SMs: not from L1)
        const unsigned short *v = reinterpret_cast<const unsigned short *>(o.v);
        float sum = 0.0f;  // of the pieces, exact
        for (int i = 0; i < o.pieces; ++i)
            sum += __uint_as_float((uint32_t)__ldcg(v + v_piece(i, o.per, o.block) + j) << 16);
        low = fmaf(sum, __bfloat162float(o.b[j]), low);
    }
    low = lane_sum(low);
    if (isnan(low)) return low;
    // eight codes a lane; bits of a code: 8, 6 or 4
    const bool fp8 = o.fmt == FP8G_E4M3 || o.fmt == FP8G_E5M2, fp4 = o.fmt == FP8G_E2M1;
    const int bits = fp8 ? 8 : fp4 ? 4 : 6;
    float sum = 0.0f;
    for (int u = lane; u < o.K / 8; u += 32) {
        const uint2 x = __ldcg(reinterpret_cast<const uint2 *>(o.x + (int64_t)u * 8));
        const uint8_t *wu = o.w + (int64_t)u * bits;
        uint64_t w;
        if (fp8) {
            w = *reinterpret_cast<const uint64_t *>(wu);
        } else if (fp4) {
            w = *reinterpret_cast<const uint32_t *>(wu);
        } else {
            const uint16_t *w3 = reinterpret_cast<const uint16_t *>(wu);
            w = w3[0] | (uint32_t)w3[1] << 16 | (uint64_t)w3[2] << 32;
        }
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t two = (uint32_t)(w >> (2 * bits * i));
            const float2 a = code_values((i < 2 ? x.x : x.y) >> (16 * (i & 1)), FP8G_E4M3);
            const float2 b = code_values(bits == 6 ? (two & 63u) | (two >> 6 & 63u) << 8 : two, o.fmt);
            dot = fmaf(a.y, b.y, fmaf(a.x, b.x, dot));
        }
        const int kb = u >> 2;  // 1x32 block
        const uint32_t ex = __ldcg(o.sfx + (kb >> 2) * o.sfx_step + (kb & 3));
        const uint32_t ew = o.sfw[(kb >> 2) * o.sfw_step + (kb & 3)];
        sum += ex == 255u || ew == 255u ? __int_as_float(0x7FC00000) : ldexpf(dot, (int)ex + (int)ew - 254);
    }
    return lane_sum(sum) + low;
}

}  // namespace fp8g
