// Quantiser for blocks of 128, and the gated backward pass that ends in it.
//
//   along rows     s[j][r] = amax of x[r][128 j .. + 127] / top
//   along columns  s[i][c] = amax of x[128 i .. + 127][c] / top
//   tiles          s[i][j] = amax of the 128 x 128 tile   / top
//   code = FP8(fl32(x fl32(1 / s))), nearest even, saturating
//
// (top 448 for E4M3, 57344 for E5M2; b128_scale's edge rules.)  Rows are the
// first operand of the forward product, columns both operands of a weight
// gradient, tiles the weights.  A gradient is needed along rows and along
// columns: both come from one reading.
//
// Backward of h = act(g) u from the 8-bit checkpoint of g and u:
//   dg = dh u act'(g),  du = dh act(g)   along rows and along columns
//   h  = act(g) u                         along columns (for the down weights)
//
// Bound by memory: a CTA takes a 128 x 128 tile, each warp 16 rows, each lane four
// columns, so that a row of a warp is a whole line of the source and of the codes.
// A row's largest magnitude is one warp reduction, a column's goes through 4 KB
// of shared memory.
#include "block128.h"
#include "block128_math.cuh"
#include "ptx.cuh"

namespace fp8g {

namespace {

constexpr int kTileThreads = 256;
constexpr int kTileWarps = kTileThreads / 32;
constexpr int kRowsPerWarp = kBlk / kTileWarps;

// Column maxima of the tile: this thread's of its warp's rows -> the tile's, in place.
// red: [kTileWarps][128] floats.
__device__ __forceinline__ void tile_col_max(float (&m)[4], float *red, int warp, int lane) {
    reinterpret_cast<float4 *>(red + warp * kBlk)[lane] = make_float4(m[0], m[1], m[2], m[3]);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kTileWarps; ++w) {
        const float4 v = reinterpret_cast<const float4 *>(red + w * kBlk)[lane];
        m[0] = fmaxf(m[0], v.x);
        m[1] = fmaxf(m[1], v.y);
        m[2] = fmaxf(m[2], v.z);
        m[3] = fmaxf(m[3], v.w);
    }
}

template <int SRC, int FMT, bool ROW, bool COL, bool TILE>
__global__ void __launch_bounds__(kTileThreads) b128_quant_kernel(const B128Quant a) {
    __shared__ float red[(COL || TILE) ? kTileWarps * kBlk : 1];
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r0 = (int64_t)blockIdx.y * kBlk, c = (int64_t)blockIdx.x * kBlk + 4 * lane;
    const int64_t row0 = r0 + warp * kRowsPerWarp;
    const bool in = c < a.C;  // (C is a multiple of 16: four columns are in or out together)
    float v[kRowsPerWarp][4];
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i) {
        const int64_t r = row0 + i;
        v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0.0f;
        if (in && r < a.R) {
            if constexpr (SRC == FP8G_IN_F32) {
                const float4 f = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(a.x) + r * a.ld + c));
                v[i][0] = f.x, v[i][1] = f.y, v[i][2] = f.z, v[i][3] = f.w;
            } else if constexpr (SRC == FP8G_IN_BF16) {
                const uint2 u = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.x) + r * a.ld + c));
                v[i][0] = __uint_as_float(u.x << 16), v[i][1] = __uint_as_float(u.x & 0xFFFF0000u);
                v[i][2] = __uint_as_float(u.y << 16), v[i][3] = __uint_as_float(u.y & 0xFFFF0000u);
            } else {
                const uint32_t q = __ldg(reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(a.x) + r * a.ld + c));
                const float s = __ldg(a.s_src + (int64_t)blockIdx.x * a.R + r);
                b128_decode(q, a.src_fmt, v[i]);
#pragma unroll
                for (int k = 0; k < 4; ++k) v[i][k] = __fmul_rn(v[i][k], s);
            }
        }
    }
    float cm[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    float own = 0.0f;  // lane i: the scale of row i of the warp
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i) {
        if constexpr (ROW) {
            const float s = b128_scale<FMT>(b128_warp_max(b128_amax4(v[i][0], v[i][1], v[i][2], v[i][3])));
            if (lane == i) own = s;
            const uint32_t q = b128_codes<FMT>(v[i][0], v[i][1], v[i][2], v[i][3], __frcp_rn(s));
            if (in && row0 + i < a.R) *reinterpret_cast<uint32_t *>(a.q_row + (row0 + i) * a.C + c) = q;
        }
        if constexpr (COL || TILE) {
#pragma unroll
            for (int k = 0; k < 4; ++k) cm[k] = fmaxf(cm[k], fabsf(v[i][k]));
        }
    }
    if constexpr (ROW) {
        if (lane < kRowsPerWarp && row0 + lane < a.R) a.s_row[(int64_t)blockIdx.x * a.R + row0 + lane] = own;
    }
    if constexpr (COL || TILE) {
        tile_col_max(cm, red, warp, lane);
        float s[4], r[4];
        if constexpr (TILE) {
            const float one = b128_scale<FMT>(b128_warp_max(fmaxf(fmaxf(cm[0], cm[1]), fmaxf(cm[2], cm[3]))));
#pragma unroll
            for (int k = 0; k < 4; ++k) s[k] = one;
            if (threadIdx.x == 0) a.s_tile[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = one;
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) s[k] = b128_scale<FMT>(cm[k]);
            if (warp == 0 && in)
                *reinterpret_cast<float4 *>(a.s_col + (int64_t)blockIdx.y * a.C + c) = make_float4(s[0], s[1], s[2], s[3]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) r[k] = __frcp_rn(s[k]);
        uint8_t *q = TILE ? a.q_tile : a.q_col;
#pragma unroll
        for (int i = 0; i < kRowsPerWarp; ++i)
            if (in && row0 + i < a.R)
                *reinterpret_cast<uint32_t *>(q + (row0 + i) * a.C + c) =
                    b128_codes4<FMT>(v[i], r);
    }
}

// The tile's sources lie in shared memory as they were read (64 KB for a bf16 dh,
// so that three CTAs share an SM and one's loads run beside another's arithmetic);
// dg, du and h are computed from them twice, for the rows and then for the columns,
// once the columns' maxima are known (kept in fp32 they would take 192 registers).
template <bool BF16>
struct BackTile {
    static constexpr int D = BF16 ? 2 : 4;  // bytes of a value of dh
    static constexpr int OFF_U = kBlk * kBlk, OFF_D = 2 * kBlk * kBlk;
    static constexpr int OFF_S = OFF_D + D * kBlk * kBlk;  // scales of g, u: [2][128]
    static constexpr int OFF_M = OFF_S + 2 * kBlk * 4;     // column maxima of dg, du, h: [3][128]
    static constexpr int BYTES = OFF_M + 3 * kBlk * 4;
};

template <bool BF16, int GATE, int FMT>
__global__ void __launch_bounds__(kTileThreads, BF16 ? 3 : 2) b128_backward_kernel(const B128Backward a) {
    using L = BackTile<BF16>;
    extern __shared__ __align__(16) uint8_t sm[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row0 = (int64_t)blockIdx.y * kBlk, c0 = (int64_t)blockIdx.x * kBlk;
    const int64_t F = a.F, F2 = 2 * F, fb = gridDim.x;
    const int rows = (int)min((int64_t)kBlk, a.M - row0);
    uint32_t *top = reinterpret_cast<uint32_t *>(sm + L::OFF_M);
    for (int i = threadIdx.x; i < 3 * kBlk; i += kTileThreads) top[i] = 0u;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    // (rows past the last are filled with zeros, and read nothing)
    const uint32_t base = ptx::smem_addr(sm);
#pragma unroll
    for (int k = 0; k < kBlk * 8 / kTileThreads; ++k) {
        const int j = threadIdx.x + k * kTileThreads, r = j >> 3, b = (j & 7) * 16;
        const int64_t at = (row0 + min(r, rows - 1)) * F2 + c0 + b;
        ptx::cp_async_16(base + j * 16, a.gu + at, r < rows ? 16 : 0);
        ptx::cp_async_16(base + L::OFF_U + j * 16, a.gu + at + F, r < rows ? 16 : 0);
    }
    constexpr int kPer = 8 * L::D;  // 16-byte pieces of a row of dh
#pragma unroll
    for (int k = 0; k < kBlk * kPer / kTileThreads; ++k) {
        const int j = threadIdx.x + k * kTileThreads, r = j / kPer, b = j % kPer * 16;
        const uint8_t *src = static_cast<const uint8_t *>(a.dh) + ((row0 + min(r, rows - 1)) * F + c0) * L::D + b;
        ptx::cp_async_16(base + L::OFF_D + j * 16, src, r < rows ? 16 : 0);
    }
    {
        const int r = threadIdx.x & (kBlk - 1), up = threadIdx.x / kBlk;
        const float *src = a.sgu + (up * fb + blockIdx.x) * a.M + row0 + min(r, rows - 1);
        ptx::cp_async_4(base + L::OFF_S + threadIdx.x * 4, src, r < rows ? 4 : 0);
    }
    ptx::cp_async_commit();
    ptx::cp_async_wait<0>();
    __syncthreads();
    const uint32_t *gq = reinterpret_cast<const uint32_t *>(sm), *uq = gq + L::OFF_U / 4;
    const float *sg = reinterpret_cast<const float *>(sm + L::OFF_S), *su = sg + kBlk;
    auto values = [&](int r, float (&dg)[4], float (&du)[4], float (&h)[4]) {
        float g[4], u[4], x[4];
        b128_decode(gq[r * 32 + lane], FP8G_E4M3, g);
        b128_decode(uq[r * 32 + lane], FP8G_E4M3, u);
        if constexpr (BF16) {
            const uint2 w = reinterpret_cast<const uint2 *>(sm + L::OFF_D)[r * 32 + lane];
            x[0] = __uint_as_float(w.x << 16), x[1] = __uint_as_float(w.x & 0xFFFF0000u);
            x[2] = __uint_as_float(w.y << 16), x[3] = __uint_as_float(w.y & 0xFFFF0000u);
        } else {
            const float4 w = reinterpret_cast<const float4 *>(sm + L::OFF_D)[r * 32 + lane];
            x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
        }
        const float s0 = sg[r], s1 = su[r];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float y, dy;
            const float uu = __fmul_rn(u[k], s1);
            b128_gate_grad(__fmul_rn(g[k], s0), GATE, y, dy);
            dg[k] = x[k] * uu * dy;
            du[k] = x[k] * y;
            h[k] = y * uu;
        }
    };
    const int first = warp * kRowsPerWarp, last = min(first + kRowsPerWarp, rows);
    float mg[4] = {}, mu[4] = {}, mh[4] = {};
    float own_g = 0.0f, own_u = 0.0f;
#pragma unroll 2
    for (int r = first; r < last; ++r) {
        float dg[4], du[4], h[4];
        values(r, dg, du, h);
        const float s0 = b128_scale<FMT>(b128_warp_max(b128_amax4(dg[0], dg[1], dg[2], dg[3])));
        const float s1 = b128_scale<FMT>(b128_warp_max(b128_amax4(du[0], du[1], du[2], du[3])));
        if (lane == r - first) own_g = s0, own_u = s1;
        uint8_t *q = a.row + (row0 + r) * F2 + c0 + 4 * lane;
        *reinterpret_cast<uint32_t *>(q) = b128_codes<FMT>(dg[0], dg[1], dg[2], dg[3], __frcp_rn(s0));
        *reinterpret_cast<uint32_t *>(q + F) = b128_codes<FMT>(du[0], du[1], du[2], du[3], __frcp_rn(s1));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            mg[k] = fmaxf(mg[k], fabsf(dg[k]));
            mu[k] = fmaxf(mu[k], fabsf(du[k]));
            mh[k] = fmaxf(mh[k], fabsf(h[k]));
        }
    }
    if (first + lane < last) {
        a.s_row[blockIdx.x * a.M + row0 + first + lane] = own_g;
        a.s_row[(fb + blockIdx.x) * a.M + row0 + first + lane] = own_u;
    }
    // (magnitudes that are not NaN: their bits are in order)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        atomicMax(top + 4 * lane + k, __float_as_uint(mg[k]));
        atomicMax(top + kBlk + 4 * lane + k, __float_as_uint(mu[k]));
        atomicMax(top + 2 * kBlk + 4 * lane + k, __float_as_uint(mh[k]));
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        mg[k] = b128_scale<FMT>(__uint_as_float(top[4 * lane + k]));
        mu[k] = b128_scale<FMT>(__uint_as_float(top[kBlk + 4 * lane + k]));
        mh[k] = b128_scale<FP8G_E4M3>(__uint_as_float(top[2 * kBlk + 4 * lane + k]));
    }
    if (warp == 0) {
        float *s = a.s_col + (int64_t)blockIdx.y * F2 + c0 + 4 * lane;
        *reinterpret_cast<float4 *>(s) = make_float4(mg[0], mg[1], mg[2], mg[3]);
        *reinterpret_cast<float4 *>(s + F) = make_float4(mu[0], mu[1], mu[2], mu[3]);
        *reinterpret_cast<float4 *>(a.s_h + (int64_t)blockIdx.y * F + c0 + 4 * lane) =
            make_float4(mh[0], mh[1], mh[2], mh[3]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) mg[k] = __frcp_rn(mg[k]), mu[k] = __frcp_rn(mu[k]), mh[k] = __frcp_rn(mh[k]);
#pragma unroll 2
    for (int r = first; r < last; ++r) {
        float dg[4], du[4], h[4];
        values(r, dg, du, h);
        uint8_t *q = a.col + (row0 + r) * F2 + c0 + 4 * lane;
        *reinterpret_cast<uint32_t *>(q) = b128_codes4<FMT>(dg, mg);
        *reinterpret_cast<uint32_t *>(q + F) = b128_codes4<FMT>(du, mu);
        *reinterpret_cast<uint32_t *>(a.h + (row0 + r) * F + c0 + 4 * lane) = b128_codes4<FP8G_E4M3>(h, mh);
    }
}

template <int SRC, int FMT>
cudaError_t quant_src(const B128Quant &a, cudaStream_t s) {
    const dim3 grid((unsigned)((a.C + kBlk - 1) / kBlk), (unsigned)((a.R + kBlk - 1) / kBlk));
    if (a.q_tile != nullptr)
        return launch_programmatic(b128_quant_kernel<SRC, FMT, false, false, true>, grid, dim3(kTileThreads), s, a);
    if (a.q_row != nullptr && a.q_col != nullptr)
        return launch_programmatic(b128_quant_kernel<SRC, FMT, true, true, false>, grid, dim3(kTileThreads), s, a);
    if (a.q_row != nullptr)
        return launch_programmatic(b128_quant_kernel<SRC, FMT, true, false, false>, grid, dim3(kTileThreads), s, a);
    return launch_programmatic(b128_quant_kernel<SRC, FMT, false, true, false>, grid, dim3(kTileThreads), s, a);
}

template <bool BF16, int GATE, int FMT>
cudaError_t backward_fmt(const B128Backward &a, cudaStream_t s) {
    const dim3 grid((unsigned)(a.F / kBlk), (unsigned)((a.M + kBlk - 1) / kBlk));
    auto kern = b128_backward_kernel<BF16, GATE, FMT>;
    constexpr int kBytes = BackTile<BF16>::BYTES;
    const cudaError_t e = b128_allow_smem(reinterpret_cast<const void *>(kern), kBytes);
    return e != cudaSuccess ? e : launch_programmatic_smem(kern, grid, dim3(kTileThreads), kBytes, s, a);
}

template <bool BF16, int GATE>
cudaError_t backward_gate(const B128Backward &a, int fmt, cudaStream_t s) {
    return fmt == FP8G_E4M3 ? backward_fmt<BF16, GATE, FP8G_E4M3>(a, s) : backward_fmt<BF16, GATE, FP8G_E5M2>(a, s);
}

}  // namespace

cudaError_t launch_b128_quant(const B128Quant &a, int fmt, cudaStream_t s) {
    if (a.src == kB128Codes) {  // codes are turned: along columns only
        const dim3 grid((unsigned)((a.C + kBlk - 1) / kBlk), (unsigned)((a.R + kBlk - 1) / kBlk));
        return fmt == FP8G_E4M3
                   ? launch_programmatic(b128_quant_kernel<kB128Codes, FP8G_E4M3, false, true, false>, grid,
                                         dim3(kTileThreads), s, a)
                   : launch_programmatic(b128_quant_kernel<kB128Codes, FP8G_E5M2, false, true, false>, grid,
                                         dim3(kTileThreads), s, a);
    }
    if (a.src == FP8G_IN_F32)
        return fmt == FP8G_E4M3 ? quant_src<FP8G_IN_F32, FP8G_E4M3>(a, s) : quant_src<FP8G_IN_F32, FP8G_E5M2>(a, s);
    return fmt == FP8G_E4M3 ? quant_src<FP8G_IN_BF16, FP8G_E4M3>(a, s) : quant_src<FP8G_IN_BF16, FP8G_E5M2>(a, s);
}

cudaError_t launch_b128_backward(const B128Backward &a, bool bf16, int gate, int fmt, cudaStream_t s) {
    if (gate == FP8G_GATE_SILU)
        return bf16 ? backward_gate<true, FP8G_GATE_SILU>(a, fmt, s) : backward_gate<false, FP8G_GATE_SILU>(a, fmt, s);
    if (gate == FP8G_GATE_GELU)
        return bf16 ? backward_gate<true, FP8G_GATE_GELU>(a, fmt, s) : backward_gate<false, FP8G_GATE_GELU>(a, fmt, s);
    return bf16 ? backward_gate<true, FP8G_GATE_RELU>(a, fmt, s) : backward_gate<false, FP8G_GATE_RELU>(a, fmt, s);
}

}  // namespace fp8g
