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
// Bound by memory.  Along columns (and in tiles) a CTA takes a 128 x 128 tile, copied
// to shared memory as it was read (cp.async; several CTAs share an SM, one's copies run
// beside another's arithmetic).  A first pass over it finds the rows' and the columns'
// largest magnitudes, a second writes all codes: each warp has 16 rows, each lane four
// columns, so that a row of a warp is a whole line of the codes.  A warp's 16 row
// scales are divided out side by side in 16 lanes (a division a row by every lane was a
// third of the instructions).  Along rows alone a lane takes 16 values of a row and
// eight lanes a block, with no second pass.  Measured: 4099 x 14336 bf16 both ways 39 us,
// 6.1 TB/s (in one pass from registers, two CTAs an SM, 104 us); 8192 x 4096 codes turned
// 13 us, 5.2 TB/s, the ALU pipe two thirds of the time (with decoded values kept in
// registers from the first pass, so fewer warps, 15.5).
#include "block128.h"
#include "block128_math.cuh"
#include "ptx.cuh"

namespace fp8g {

namespace {

constexpr int kTileThreads = 256;
constexpr int kTileWarps = kTileThreads / 32;
constexpr int kRowsPerWarp = kBlk / kTileWarps;

__device__ __forceinline__ void widen4(const uint2 u, float (&v)[4]) {
    v[0] = __uint_as_float(u.x << 16), v[1] = __uint_as_float(u.x & 0xFFFF0000u);
    v[2] = __uint_as_float(u.y << 16), v[3] = __uint_as_float(u.y & 0xFFFF0000u);
}

// rows x (16 * PIECES) bytes, `pitch` bytes apart in memory, to dst, packed; of a row
// the first `bytes` exist; rows past `rows` and bytes past `bytes` are filled with
// zeros and read nothing.
template <int PIECES, int THREADS = kTileThreads>
__device__ __forceinline__ void copy_tile(uint32_t dst, const void *src, int64_t pitch, int rows, int bytes) {
#pragma unroll
    for (int k = 0; k < kBlk * PIECES / THREADS; ++k) {
        const int j = threadIdx.x + k * THREADS, r = j / PIECES, b = j % PIECES * 16;
        const bool in = r < rows && b < bytes;
        ptx::cp_async_16(dst + j * 16, static_cast<const uint8_t *>(src) + (in ? r * pitch + b : 0), in ? 16 : 0);
    }
}

// ---------------------------------------------------------------- along rows

constexpr int kRowTile = 16;   // rows of a CTA, two a warp
constexpr int kColSpan = 512;  // columns of a CTA, 16 a lane

template <bool BF16, int FMT>
__global__ void __launch_bounds__(kTileThreads) b128_quant_rows_kernel(const B128Quant a) {
    __shared__ float scales[kColSpan / kBlk][kRowTile];
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t c = (int64_t)blockIdx.x * kColSpan + 16 * lane, row0 = (int64_t)blockIdx.y * kRowTile;
    float v[2][16];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t r = row0 + 2 * warp + i;
        const bool in = c < a.C && r < a.R;  // (C is a multiple of 16)
#pragma unroll
        for (int k = 0; k < 16; ++k) v[i][k] = 0.0f;
        if (in) {
            if constexpr (BF16) {
                const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.x) + r * a.ld + c);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint4 u = __ldg(x + k);
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[i][8 * k + 2 * j] = __uint_as_float(w[j] << 16);
                        v[i][8 * k + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
                    }
                }
            } else {
                const float4 *x = reinterpret_cast<const float4 *>(static_cast<const float *>(a.x) + r * a.ld + c);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float4 u = __ldg(x + k);
                    v[i][4 * k] = u.x, v[i][4 * k + 1] = u.y, v[i][4 * k + 2] = u.z, v[i][4 * k + 3] = u.w;
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float m[2] = {};
#pragma unroll
        for (int k = 0; k < 16; k += 2) m[(k >> 1) & 1] = b128_max3(m[(k >> 1) & 1], v[i][k], v[i][k + 1]);
        float top = fmaxf(m[0], m[1]);
#pragma unroll
        for (int o = 1; o < 8; o *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float s = b128_scale<FMT>(top), r = __frcp_rn(s);
        if ((lane & 7) == 0) scales[lane >> 3][2 * warp + i] = s;
        uint4 q;
        q.x = b128_codes<FMT>(v[i][0], v[i][1], v[i][2], v[i][3], r);
        q.y = b128_codes<FMT>(v[i][4], v[i][5], v[i][6], v[i][7], r);
        q.z = b128_codes<FMT>(v[i][8], v[i][9], v[i][10], v[i][11], r);
        q.w = b128_codes<FMT>(v[i][12], v[i][13], v[i][14], v[i][15], r);
        const int64_t row = row0 + 2 * warp + i;
        if (c < a.C && row < a.R) *reinterpret_cast<uint4 *>(a.q_row + row * a.C + c) = q;
    }
    __syncthreads();
    // the rows of a block side by side
    const int i = threadIdx.x % kRowTile, b = threadIdx.x / kRowTile;
    if (b < kColSpan / kBlk && row0 + i < a.R && (int64_t)blockIdx.x * kColSpan + b * kBlk < a.C)
        a.s_row[((int64_t)blockIdx.x * (kColSpan / kBlk) + b) * a.R + row0 + i] = scales[b][i];
}

// ------------------------------------------------------ along columns, in tiles

template <int SRC>
constexpr int kSrcBytes = SRC == FP8G_IN_F32 ? 4 : SRC == FP8G_IN_BF16 ? 2 : 1;

template <int SRC, int FMT, bool ROW, bool TILE>
__global__ void __launch_bounds__(kTileThreads, 4) b128_quant_tile_kernel(const B128Quant a) {
    constexpr int E = kSrcBytes<SRC>;
    extern __shared__ __align__(16) uint8_t sm[];
    uint32_t *top = reinterpret_cast<uint32_t *>(sm + kBlk * kBlk * E);  // column maxima [128]
    float *src_s = reinterpret_cast<float *>(top + kBlk);                // row scales of codes [128]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row0 = (int64_t)blockIdx.y * kBlk, c0 = (int64_t)blockIdx.x * kBlk, c = c0 + 4 * lane;
    const int rows = (int)min((int64_t)kBlk, a.R - row0);
    const bool in = c < a.C;  // (C is a multiple of 16: four columns are in or out together)
    if (threadIdx.x < kBlk) top[threadIdx.x] = 0u;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    copy_tile<8 * E>(ptx::smem_addr(sm), static_cast<const uint8_t *>(a.x) + (row0 * a.ld + c0) * E, a.ld * E, rows,
                     (int)min((int64_t)kBlk, a.C - c0) * E);
    if constexpr (SRC == kB128Codes) {
        if (threadIdx.x < kBlk)
            ptx::cp_async_4(ptx::smem_addr(src_s + threadIdx.x),
                            a.s_src + (int64_t)blockIdx.x * a.R + row0 + min((int)threadIdx.x, rows - 1), 4);
    }
    ptx::cp_async_commit();
    ptx::cp_async_wait<0>();
    __syncthreads();
    auto values = [&](int r, float s, float (&v)[4]) {
        if constexpr (SRC == FP8G_IN_F32) {
            const float4 f = reinterpret_cast<const float4 *>(sm)[r * 32 + lane];
            v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
        } else if constexpr (SRC == FP8G_IN_BF16) {
            widen4(reinterpret_cast<const uint2 *>(sm)[r * 32 + lane], v);
        } else {
            b128_decode(reinterpret_cast<const uint32_t *>(sm)[r * 32 + lane], a.src_fmt, v);
            const uint64_t ss = b128_pair(s, s);
            const uint64_t lo = b128_mul2(b128_pair(v[0], v[1]), ss), hi = b128_mul2(b128_pair(v[2], v[3]), ss);
            v[0] = b128_lo(lo), v[1] = b128_hi(lo), v[2] = b128_lo(hi), v[3] = b128_hi(hi);
        }
    };
    // (rows and columns past the matrix are zeros: they change no maximum)
    const int first = warp * kRowsPerWarp;
    float4 s4 = make_float4(0.0f, 0.0f, 0.0f, 0.0f);  // four rows' scales
    float cm[4] = {}, own = 0.0f;  // own: lane i has row first + i's
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; i += 2) {
        float v[4], w[4];
        if (SRC == kB128Codes && i % 4 == 0) s4 = *reinterpret_cast<const float4 *>(src_s + first + i);
        values(first + i, i % 4 == 0 ? s4.x : s4.z, v);
        values(first + i + 1, i % 4 == 0 ? s4.y : s4.w, w);
        if constexpr (ROW) {
            const float m0 = b128_warp_max(b128_amax4(v[0], v[1], v[2], v[3]));
            const float m1 = b128_warp_max(b128_amax4(w[0], w[1], w[2], w[3]));
            own = lane == i ? m0 : lane == i + 1 ? m1 : own;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) cm[k] = b128_max3(cm[k], v[k], w[k]);
    }
    // (magnitudes that are not NaN: their bits are in order)
#pragma unroll
    for (int k = 0; k < 4; ++k) atomicMax(top + 4 * lane + k, __float_as_uint(cm[k]));
    float rr = 0.0f;
    if constexpr (ROW) {
        const float s = b128_scale<FMT>(own);
        rr = __frcp_rn(s);
        if (lane < kRowsPerWarp && first + lane < rows) a.s_row[(int64_t)blockIdx.x * a.R + row0 + first + lane] = s;
    }
    __syncthreads();
    float s[4];  // 1 / scale of the lane's columns
    if constexpr (TILE) {
        const uint4 t = reinterpret_cast<const uint4 *>(top)[lane];
        const uint32_t most = max(max(t.x, t.y), max(t.z, t.w));
        const float one = b128_scale<FMT>(b128_warp_max(__uint_as_float(most)));
        if (threadIdx.x == 0) a.s_tile[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = one;
        s[0] = s[1] = s[2] = s[3] = __frcp_rn(one);
    } else {
        // (a column's divisions once, not by every warp: a tenth of the instructions)
        if (threadIdx.x < kBlk) {
            const float one = b128_scale<FMT>(__uint_as_float(top[threadIdx.x]));
            if (c0 + threadIdx.x < a.C) a.s_col[(int64_t)blockIdx.y * a.C + c0 + threadIdx.x] = one;
            top[threadIdx.x] = __float_as_uint(__frcp_rn(one));
        }
        __syncthreads();
        const float4 t = reinterpret_cast<const float4 *>(top)[lane];
        s[0] = t.x, s[1] = t.y, s[2] = t.z, s[3] = t.w;
    }
    const int64_t at = (row0 + first) * a.C + c;
    uint8_t *q = (TILE ? a.q_tile : a.q_col) + at, *q_row = ROW ? a.q_row + at : nullptr;
    const int live = in ? min(kRowsPerWarp, rows - first) : 0;
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i) {
        float v[4];
        if (SRC == kB128Codes && i % 4 == 0) s4 = *reinterpret_cast<const float4 *>(src_s + first + i);
        values(first + i, i % 4 == 0 ? s4.x : i % 4 == 1 ? s4.y : i % 4 == 2 ? s4.z : s4.w, v);
        const float r = ROW ? __shfl_sync(0xffffffffu, rr, i) : 0.0f;
        if (i < live) {
            if constexpr (ROW) *reinterpret_cast<uint32_t *>(q_row) = b128_codes<FMT>(v[0], v[1], v[2], v[3], r);
            *reinterpret_cast<uint32_t *>(q) = b128_codes4<FMT>(v, s);
        }
        q += a.C;
        q_row += a.C;
    }
}

// ------------------------------------------------------------ gated backward

// One CTA an SM takes tile after tile, the next one's copies running beside this one's
// arithmetic.  dg, du and h of a tile stay in registers (8 rows of four columns a
// thread, 96 values) between the maxima and the codes, and its arithmetic is packed where
// it can be: the instructions bound it (two thirds of the issue slots at 4099 x 14336, 107 us,
// 5.1 TB/s; with everything computed twice, for the maxima and for the codes, 162 us).
constexpr int kBackThreads = 512;
constexpr int kBackRows = kBlk / (kBackThreads / 32);

template <bool BF16>
struct BackTile {
    static constexpr int D = BF16 ? 2 : 4;  // bytes of a value of dh
    static constexpr int OFF_U = kBlk * kBlk, OFF_D = 2 * kBlk * kBlk;
    static constexpr int OFF_S = OFF_D + D * kBlk * kBlk;  // scales of g, u: [2][128]
    static constexpr int TILE = OFF_S + 2 * kBlk * 4;
    static constexpr int OFF_M = 2 * TILE;                 // column maxima of dg, du, h: [2][3][128]
    static constexpr int BYTES = OFF_M + 2 * 3 * kBlk * 4;
};

template <bool BF16, int GATE, int FMT>
__global__ void __launch_bounds__(kBackThreads, 1) b128_backward_kernel(const B128Backward a) {
    using L = BackTile<BF16>;
    extern __shared__ __align__(16) uint8_t sm[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t F = a.F, F2 = 2 * F;
    const int32_t fb = (int32_t)(F / kBlk), tiles = fb * (int32_t)((a.M + kBlk - 1) / kBlk);
    uint32_t *tops = reinterpret_cast<uint32_t *>(sm + L::OFF_M);
    for (int i = threadIdx.x; i < 2 * 3 * kBlk; i += kBackThreads) tops[i] = 0u;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    // Tile t to buffer i: a group of copies (rows past the last read nothing and become zeros)
    auto ask = [&](int32_t t, int i) {
        if (t < tiles) {
            const int64_t row0 = (int64_t)(t / fb) * kBlk, c0 = (int64_t)(t % fb) * kBlk;
            const int rows = (int)min((int64_t)kBlk, a.M - row0);
            const uint32_t base = ptx::smem_addr(sm) + i * L::TILE;
            copy_tile<8, kBackThreads>(base, a.gu + row0 * F2 + c0, F2, rows, kBlk);
            copy_tile<8, kBackThreads>(base + L::OFF_U, a.gu + row0 * F2 + F + c0, F2, rows, kBlk);
            copy_tile<8 * L::D, kBackThreads>(base + L::OFF_D, static_cast<const uint8_t *>(a.dh) + (row0 * F + c0) * L::D,
                                              F * L::D, rows, kBlk * L::D);
            if (threadIdx.x < 2 * kBlk) {
                const int r = threadIdx.x & (kBlk - 1), up = threadIdx.x / kBlk;
                ptx::cp_async_4(base + L::OFF_S + threadIdx.x * 4,
                                a.sgu + ((int64_t)up * fb + t % fb) * a.M + row0 + min(r, rows - 1), 4);
            }
        }
        ptx::cp_async_commit();
    };
    ask((int32_t)blockIdx.x, 0);
    const int first = warp * kBackRows;
    int i = 0;
    for (int32_t t = (int32_t)blockIdx.x; t < tiles; t += (int32_t)gridDim.x, i ^= 1) {
        ptx::cp_async_wait<0>();
        __syncthreads();  // this tile is there, and the other buffer read by all
        ask(t + (int32_t)gridDim.x, i ^ 1);
        const int64_t row0 = (int64_t)(t / fb) * kBlk, c0 = (int64_t)(t % fb) * kBlk;
        const int rows = (int)min((int64_t)kBlk, a.M - row0);
        const uint8_t *tile = sm + i * L::TILE;
        const uint32_t *gq = reinterpret_cast<const uint32_t *>(tile), *uq = gq + L::OFF_U / 4;
        const float *sg = reinterpret_cast<const float *>(tile + L::OFF_S), *su = sg + kBlk;
        uint32_t *top = tops + i * 3 * kBlk;
        float dg[kBackRows][4], du[kBackRows][4], h[kBackRows][4];
        float mg[4] = {}, mu[4] = {}, mh[4] = {};
        float own = 0.0f;  // lane j: dg's of row first + j, lane kBackRows + j: du's
#pragma unroll
        for (int j = 0; j < kBackRows; ++j) {
            const int r = first + j;
            float g[4], u[4], x[4];
            b128_decode(gq[r * 32 + lane], FP8G_E4M3, g);
            b128_decode(uq[r * 32 + lane], FP8G_E4M3, u);
            if constexpr (BF16) {
                widen4(reinterpret_cast<const uint2 *>(tile + L::OFF_D)[r * 32 + lane], x);
            } else {
                const float4 w = reinterpret_cast<const float4 *>(tile + L::OFF_D)[r * 32 + lane];
                x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
            }
            const uint64_t s0 = b128_pair(sg[r], sg[r]), s1 = b128_pair(su[r], su[r]);
#pragma unroll
            for (int k = 0; k < 4; k += 2) {  // (packed: the instructions bound this kernel)
                const uint64_t gg = b128_mul2(b128_pair(g[k], g[k + 1]), s0), uu = b128_mul2(b128_pair(u[k], u[k + 1]), s1);
                const uint64_t xx = b128_pair(x[k], x[k + 1]);
                uint64_t y, dy;
                b128_gate_grad2<GATE>(gg, y, dy);
                const uint64_t vg = b128_mul2(b128_mul2(xx, uu), dy), vu = b128_mul2(xx, y), vh = b128_mul2(y, uu);
                dg[j][k] = b128_lo(vg), dg[j][k + 1] = b128_hi(vg);
                du[j][k] = b128_lo(vu), du[j][k + 1] = b128_hi(vu);
                h[j][k] = b128_lo(vh), h[j][k + 1] = b128_hi(vh);
            }
            if (j & 1) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    mg[k] = b128_max3(mg[k], dg[j - 1][k], dg[j][k]);
                    mu[k] = b128_max3(mu[k], du[j - 1][k], du[j][k]);
                    mh[k] = b128_max3(mh[k], h[j - 1][k], h[j][k]);
                }
            }
            const float a0 = b128_warp_max(b128_amax4(dg[j][0], dg[j][1], dg[j][2], dg[j][3]));
            const float a1 = b128_warp_max(b128_amax4(du[j][0], du[j][1], du[j][2], du[j][3]));
            own = lane == j ? a0 : lane == kBackRows + j ? a1 : own;
        }
        // (magnitudes that are not NaN: their bits are in order)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            atomicMax(top + 4 * lane + k, __float_as_uint(mg[k]));
            atomicMax(top + kBlk + 4 * lane + k, __float_as_uint(mu[k]));
            atomicMax(top + 2 * kBlk + 4 * lane + k, __float_as_uint(mh[k]));
        }
        own = b128_scale<FMT>(own);
        const int own_row = first + (lane & (kBackRows - 1));
        if (lane < 2 * kBackRows && own_row < rows)
            a.s_row[((int64_t)(lane / kBackRows) * fb + t % fb) * a.M + row0 + own_row] = own;
        own = __frcp_rn(own);
        __syncthreads();
        // (a column's divisions once, not by every warp: an eighth of the instructions)
        if (threadIdx.x < 3 * kBlk) {
            const int col = threadIdx.x & (kBlk - 1), which = threadIdx.x / kBlk;
            const float m = __uint_as_float(top[threadIdx.x]);
            const float s = which == 2 ? b128_scale<FP8G_E4M3>(m) : b128_scale<FMT>(m);
            (which == 2 ? a.s_h + (int64_t)(t / fb) * F : a.s_col + (int64_t)(t / fb) * F2 + which * F)[c0 + col] = s;
            top[threadIdx.x] = __float_as_uint(__frcp_rn(s));
        }
        __syncthreads();
        auto columns = [&](int which, float(&r)[4]) {
            const float4 v = reinterpret_cast<const float4 *>(top + which * kBlk)[lane];
            r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
        };
        columns(0, mg), columns(1, mu), columns(2, mh);
        // the other buffer's maxima were read before this tile's first barrier: zeros for
        // the next tile
        for (int k = threadIdx.x; k < 3 * kBlk; k += kBackThreads) tops[(i ^ 1) * 3 * kBlk + k] = 0u;
        const int64_t at = (row0 + first) * F2 + c0 + 4 * lane;
        uint8_t *row = a.row + at, *col = a.col + at, *hq = a.h + (row0 + first) * F + c0 + 4 * lane;
#pragma unroll
        for (int j = 0; j < kBackRows; ++j) {
            const float r0 = __shfl_sync(0xffffffffu, own, j), r1 = __shfl_sync(0xffffffffu, own, kBackRows + j);
            if (first + j < rows) {
                *reinterpret_cast<uint32_t *>(row + j * F2) = b128_codes<FMT>(dg[j][0], dg[j][1], dg[j][2], dg[j][3], r0);
                *reinterpret_cast<uint32_t *>(row + j * F2 + F) = b128_codes<FMT>(du[j][0], du[j][1], du[j][2], du[j][3], r1);
                *reinterpret_cast<uint32_t *>(col + j * F2) = b128_codes4<FMT>(dg[j], mg);
                *reinterpret_cast<uint32_t *>(col + j * F2 + F) = b128_codes4<FMT>(du[j], mu);
                *reinterpret_cast<uint32_t *>(hq + j * F) = b128_codes4<FP8G_E4M3>(h[j], mh);
            }
        }
    }
}

template <int SRC, int FMT, bool ROW, bool TILE>
cudaError_t quant_tile(const B128Quant &a, cudaStream_t s) {
    auto kern = b128_quant_tile_kernel<SRC, FMT, ROW, TILE>;
    constexpr int kBytes = kBlk * kBlk * kSrcBytes<SRC> + 2 * kBlk * 4;
    if constexpr (kBytes > 48 * 1024) {
        static unsigned long long done = 0ull;
        const cudaError_t e = b128_allow_smem(reinterpret_cast<const void *>(kern), kBytes, done);
        if (e != cudaSuccess) return e;
    }
    const dim3 grid((unsigned)((a.C + kBlk - 1) / kBlk), (unsigned)((a.R + kBlk - 1) / kBlk));
    return launch_programmatic_smem(kern, grid, dim3(kTileThreads), kBytes, s, a);
}

template <int SRC, int FMT>
cudaError_t quant_src(const B128Quant &a, cudaStream_t s) {
    if (a.q_tile != nullptr) return quant_tile<SRC, FMT, false, true>(a, s);
    if (a.q_col != nullptr)
        return a.q_row != nullptr ? quant_tile<SRC, FMT, true, false>(a, s) : quant_tile<SRC, FMT, false, false>(a, s);
    const dim3 grid((unsigned)((a.C + kColSpan - 1) / kColSpan), (unsigned)((a.R + kRowTile - 1) / kRowTile));
    return launch_programmatic(b128_quant_rows_kernel<SRC == FP8G_IN_BF16, FMT>, grid, dim3(kTileThreads), s, a);
}

template <bool BF16, int GATE, int FMT>
cudaError_t backward_fmt(const B128Backward &a, cudaStream_t s) {
    auto kern = b128_backward_kernel<BF16, GATE, FMT>;
    constexpr int kBytes = BackTile<BF16>::BYTES;
    static unsigned long long done = 0ull;
    const cudaError_t e = b128_allow_smem(reinterpret_cast<const void *>(kern), kBytes, done);
    const int64_t tiles = (a.M + kBlk - 1) / kBlk * (a.F / kBlk);
    const dim3 grid((unsigned)min(tiles, (int64_t)a.num_sms));
    return e != cudaSuccess ? e : launch_programmatic_smem(kern, grid, dim3(kBackThreads), kBytes, s, a);
}

template <bool BF16, int GATE>
cudaError_t backward_gate(const B128Backward &a, int fmt, cudaStream_t s) {
    return fmt == FP8G_E4M3 ? backward_fmt<BF16, GATE, FP8G_E4M3>(a, s) : backward_fmt<BF16, GATE, FP8G_E5M2>(a, s);
}

}  // namespace

cudaError_t launch_b128_quant(const B128Quant &a, int fmt, cudaStream_t s) {
    if (a.src == kB128Codes)  // codes are turned: along columns only
        return fmt == FP8G_E4M3 ? quant_tile<kB128Codes, FP8G_E4M3, false, false>(a, s)
                                : quant_tile<kB128Codes, FP8G_E5M2, false, false>(a, s);
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
