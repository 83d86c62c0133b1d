// fp32 values as sums of bf16 pieces, as the tensor cores take them beside the
// adapters' bf16 A and B: three, cut after 8 bits each, are the value exactly (24
// significant bits; of values below 2^-110 the last bits go), two, rounded, the value
// to 2^-17.  V = alpha A x and an fp32 x are taken in three for an fp32 output, in two
// for a bf16 one.  Distance to the 64-bit result, one row at 4096 x 4096, rank 16: fp32
// output 4.2e-7 with three, 1.4e-6 with two; bf16 output 1.70e-3 either way, of its own
// rounding.  A third piece costs a low-rank step half as many MMAs again and a higher
// rank half as much of V: 128 rows of 32 adapters of rank 64 at 4096 x 14336 46.0 us,
// with two 41.9; 512 rows 124.5 and 113; 2048 rows of 8 at 4096 x 8192 88.9 and 86.9;
// 33 rows of rank 16 at 4096 x 4096 22.9 and 22.5 (in graphs).
#pragma once
#include <cuda_bf16.h>

#include "quant_math.cuh"
#include "stream.h"

namespace fp8g {

// The first of P pieces of v as fp32; v becomes the rest (of an infinity, or a value
// rounded to one: none).
template <int P>
__device__ __forceinline__ float next_piece(float &v) {
    const float top = P == 3 ? __uint_as_float(__float_as_uint(v) & 0xFFFF0000u)
                             : __bfloat162float(__float2bfloat16_rn(v));
    v = isinf(P == 3 ? v : top) ? 0.0f : v - top;
    return top;
}

// The same of two values, as a bf16 pair.
template <int P>
__device__ __forceinline__ uint32_t next_pieces(float &a, float &b) {
    const float x = next_piece<P>(a), y = next_piece<P>(b);
    return __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
}

// Eight consecutive values of x: as they are, or piece by piece.
template <bool BF16>
struct X8;
template <>
struct X8<true> {
    static constexpr int kMost = 1;  // pieces
    uint4 v;
    __device__ __forceinline__ void load(const void *x, int64_t off) {
        v = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(x) + off));
    }
    template <int P>
    __device__ __forceinline__ uint4 next() {
        return v;
    }
};
template <>
struct X8<false> {
    static constexpr int kMost = 3;
    float4 a, b;
    __device__ __forceinline__ void load(const void *x, int64_t off) { load8<false>(x, off, a, b); }
    template <int P>
    __device__ __forceinline__ uint4 next() {
        return make_uint4(next_pieces<P>(a.x, a.y), next_pieces<P>(a.z, a.w), next_pieces<P>(b.x, b.y),
                          next_pieces<P>(b.z, b.w));
    }
};

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A value of V to its pieces' places, hi the first one's, block: values of a block
// of rows.
template <int P>
__device__ __forceinline__ void store_v(__nv_bfloat16 *hi, float v, int per, int64_t block) {
#pragma unroll
    for (int i = 0; i < P; ++i) hi[v_piece(i, per, block)] = __float2bfloat16_rn(next_piece<P>(v));
}

// Zeros in 16 n values of V from hi on, in every piece.
template <int P>
__device__ __forceinline__ void zero_v(__nv_bfloat16 *hi, int n, int per, int64_t block) {
    for (int c = 0; c < 2 * n; ++c)
#pragma unroll
        for (int i = 0; i < P; ++i)
            reinterpret_cast<uint4 *>(hi + v_piece(i, per, block))[c] = make_uint4(0u, 0u, 0u, 0u);
}

}  // namespace fp8g
