// Declarations of the operators with scales for blocks of 128 (block128*.cu).
//
// Scales are fp32 and lie by block of the contraction first: one per 128
// consecutive values of a row at [block of the row][row], one per 128 values of
// a column at [block of the column][column].  So both operands' scales of one
// K block are contiguous over the rows (columns) of C, whichever way the
// operand lies.
#pragma once
#include "internal.h"

namespace fp8g {

constexpr int kBlk = 128;

// A product C[M, N] = sum over K blocks, or the gated projection pair.
struct B128Params {
    int64_t M, N, K;
    int32_t num_kb;         // ceil(K / 128)
    int32_t npm, npn;       // tiles of C
    int32_t first, T;       // tiles [first, T) of the npm npn
    // CTA pairs: pair c takes tiles first + c, first + c + pairs, ..; or with `share` > 0 the
    // tiles' K blocks c share .. one after the other
    int32_t pairs, share;
    float *part;            // [pairs][256 x 256] sums of a share that ends inside its tile
    int32_t *there;         // zeros at the start. [pairs][16] by warp: part is written; then
                            // the pairs that have begun
    const float *sa;        // [num_kb][M]
    const float *sb;        // vectors [num_kb][N]; tiles: block (n, k) at n sb_n + k sb_k
    int64_t sb_n, sb_k;
    int32_t n_blocks;       // tiles of 128 along N (gated: along F)
    uint32_t types;         // operand types and majors as instruction descriptor bits
    int32_t a_mn, b_mn;     // operand lies with M (N) contiguous
    void *C;
    // gated: columns of C are the F columns of h
    uint8_t *h, *gu;        // codes [M, F], [M, 2F] (gu may be null)
    float *sh, *sgu;        // [F / 128][M], [2 F / 128][M]
    unsigned int *status;
    uint64_t timeout_ns;
};

// What a product kernel ends in (kB128Gated + FP8G_GATE_*: h = act(g) u in 8 bits).
enum B128Out : int { kB128Bf16 = 0, kB128F32 = 1, kB128Add = 2, kB128Gated = 3 };

// block128_gemm.cu, block128_share.cu (p.share > 0; no gated outputs): CTA pairs over
// 256 x 256 tiles (gated: 256 rows, 128 columns of gate and of up).  vec_b: B's scales are
// vectors.
struct B128Maps {
    CUtensorMap A, B, C, gu;  // C (gated: h) and gu are written (host_store_map)
};
cudaError_t launch_b128_pair(const B128Maps &m, const B128Params &p, int out, bool vec_b, cudaStream_t stream);
cudaError_t launch_b128_share(const B128Maps &m, const B128Params &p, int out, bool vec_b, cudaStream_t stream);
constexpr int64_t kB128PartBytes = (int64_t)4 * kBlk * kBlk * 4;  // a pair's sums

// block128_few.cu: few rows of C.  The weights (B) are the MMA's 128-row operand,
// nt rows of A its columns; K split over clusters of `split` CTAs.
cudaError_t launch_b128_few(const CUtensorMap &A, const CUtensorMap &B, const B128Params &p,
                            int out, int nt, int split, cudaStream_t stream);
// Clusters of `split` CTAs with an SM each that run at once on device `dev`, the current one.
int b128_few_clusters(int split, int dev);

// block128_quant.cu.  src: FP8G_IN_F32 / FP8G_IN_BF16 values, rows ld apart, or
// codes of src_fmt with row scales (kB128Codes).  Outputs that are null are left out.
constexpr int kB128Codes = 2;
struct B128Quant {
    const void *x;
    int64_t ld, R, C;
    int32_t src, src_fmt;
    const float *s_src;
    uint8_t *q_row, *q_col, *q_tile;
    float *s_row, *s_col, *s_tile;
};
cudaError_t launch_b128_quant(const B128Quant &a, int fmt, cudaStream_t stream);

struct B128Backward {
    const void *dh;
    const uint8_t *gu;
    const float *sgu;
    int64_t M, F;
    uint8_t *row, *col, *h;      // [M, 2F], [M, 2F], [M, F]
    float *s_row, *s_col, *s_h;
    int32_t num_sms;
};
cudaError_t launch_b128_backward(const B128Backward &a, bool bf16, int gate, int fmt,
                                 cudaStream_t stream);

// Lets `kernel` have `bytes` of dynamic shared memory on the current device, once (`done`:
// the devices that it has it on; calls that race on it set it twice).
inline cudaError_t b128_allow_smem(const void *kernel, int bytes, unsigned long long &done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const unsigned long long bit = 1ull << (dev & 63);
    if (e != cudaSuccess || (done & bit) != 0ull) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done |= bit;
    return e;
}

}  // namespace fp8g
