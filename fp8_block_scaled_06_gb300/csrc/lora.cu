// A block-scaled projection with low-rank adapters of many requests.
//
//   C[i] = out( Q(x_i) W^T + bias + alpha_l B_l (A_l x_i) ),  l = adapter[i]
//
// Few rows: the streaming kernels (stream.cu).  Many: the rows quantised and
// V = alpha A x, then the CTA-pair product (gemm_pair.cu).  In both V
// is taken against the adapters' B rows as further K steps into the product's
// fp32 accumulator, so the sum is rounded once.
//
// V.  Rows are taken in tiles (a group of the streaming kernel, or the 256 rows
// of a pair).  The adapters among a tile's rows, in rising order,
// are its slots; a slot holds V of all the tile's rows, zero for those of
// other adapters, as two or three bf16 pieces (lora_pieces.cuh): the product
// then needs no gather, and an adapter costs rank / 128 of a K step's weights.
#include <cuda_bf16.h>

#include <type_traits>

#include "internal.h"
#include "kernel_common.cuh"
#include "lora_pieces.cuh"
#include "quant_math.cuh"
#include "stream.h"

namespace fp8g {

namespace {

constexpr int kLThreads = 512;
constexpr int kLWarps = kLThreads / 32;
constexpr int kMaxTile = 256;

struct LoraPrep {
    const void *x;
    int32_t M, K;
    uint8_t *xq;        // [M][K] codes
    uint8_t *xsf;       // packed scales [ks][n_rt][512]
    int32_t ks, n_rt;
    // low-rank part
    const __nv_bfloat16 *a;   // [L][r][K]
    const float *alpha;       // [L] or null
    const int32_t *adapter;   // [M]
    int32_t L, r, r64, per, blocks;  // LoraV
    int32_t tile, cap, tiles;  // tiles 0: no adapters
    __nv_bfloat16 *v;         // [tiles][cap][blocks][tile][r64]
    int32_t *slot_cnt, *slot_adapter;  // the pair kernel's tables
    int32_t items;            // blocks per tile and rank block of V
    int32_t row0;             // of the call: the first of these rows
    unsigned int *status;
};

// Row blockIdx.x of x: codes, scale bytes.  Behind lora_v_kernel, it starts beside
// it (that one began only when all before it was complete, and nothing of it is
// read here) and ends after it, so that the product can rely on both.
template <bool BF16>
__global__ void __launch_bounds__(256) lora_quant_kernel(const __grid_constant__ LoraPrep p) {
    if (p.tiles == 0) ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int tid = threadIdx.x, nt = blockDim.x, blk = blockIdx.x;
    const int rt = blk / 128, in_t = blk - rt * 128;
    const int groups = p.ks * 16;
    for (int c0 = 0; c0 < groups; c0 += nt) {
        const int c = c0 + tid;
        float4 v0 = make_float4(0.f, 0.f, 0.f, 0.f), v1 = v0;
        const bool in = c * 8 < p.K;
        if (in) load8<BF16>(p.x, (int64_t)blk * p.K + c * 8, v0, v1);
        float am = absmax8(v0, v1);
        am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
        am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
        const float s = pow2_scale<0>(am);
        if (in)
            *reinterpret_cast<uint2 *>(p.xq + (int64_t)blk * p.K + c * 8) = quant8_pow2<0>(v0, v1, s);
        if (c < groups && (c & 3) == 0)
            p.xsf[((int64_t)(c >> 4) * p.n_rt + rt) * 512 + 16 * (in_t & 31) + 4 * (in_t >> 5) + ((c >> 2) & 3)] =
                (uint8_t)(__float_as_uint(s) >> 23);
    }
    if (p.tiles != 0) ptx::grid_dep_wait();
}

// V.  A block takes an item of a tile and 16 ranks: items are the pairs (slot, 16
// of the slot's rows) in order; blocks past the last one leave.  The K range goes
// over the block's 16 warps, each a 16 x 16 product by mma.sync (ranks x rows),
// joined in shared memory in warp order.  A lane's 16-byte load covers 8
// consecutive K of a row; the same K permutation on both operands leaves the
// product unchanged.  Rows and ranks past the item's read others' values, into
// products that are not stored.
template <int P, bool BF16>
__global__ void __launch_bounds__(kLThreads, 2) lora_v_kernel(const __grid_constant__ LoraPrep p) {
    __shared__ int32_t ad[kMaxTile];
    __shared__ int32_t cnt[FP8G_MAX_ADAPTERS];
    __shared__ int32_t pick[3];  // adapter, slot, first of its rows
    __shared__ int32_t rows[16];
    __shared__ float acc[kLWarps][16][17];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int blk = blockIdx.x;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int rblocks = (p.r + 15) / 16;
    int w = blk;
    const int item = w % p.items;
    w /= p.items;
    const int rb = w % rblocks, tile = w / rblocks;
    const int row0 = tile * p.tile, n = min(p.tile, p.M - row0);
    for (int i = tid; i < p.L; i += kLThreads) cnt[i] = 0;
    __syncthreads();
    for (int i = tid; i < p.tile; i += kLThreads) {
        int l = i < n ? __ldg(p.adapter + row0 + i) : -1;
        if (l >= p.L) {
            if (item == 0 && rb == 0 && atomicCAS(&p.status[0], 0u, (unsigned)FP8G_ERR_INVALID_ARG) == 0u)
                atomicExch(&p.status[1], (unsigned)(p.row0 + row0 + i));
            l = -1;
        }
        ad[i] = l < 0 ? -1 : l;
        if (l >= 0) atomicAdd(&cnt[l], 1);
    }
    if (tid == 0) pick[0] = -1;
    if (tid < 16) rows[tid] = -1;
    __syncthreads();
    if (warp == 0) {
        int slots = 0, items = 0;  // of the adapters before this step's
        for (int l0 = 0; l0 < p.L; l0 += 32) {
            const int l = l0 + lane;
            const int c = l < p.L ? cnt[l] : 0, it = (c + 15) / 16, has = c > 0;
            int s_it = it, s_sl = has;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int vi = __shfl_up_sync(0xffffffffu, s_it, o), vs = __shfl_up_sync(0xffffffffu, s_sl, o);
                if (lane >= o) {
                    s_it += vi;
                    s_sl += vs;
                }
            }
            const int first = items + s_it - it, slot = slots + s_sl - has;
            if (has && item >= first && item < first + it) {
                pick[0] = l;
                pick[1] = slot;
                pick[2] = 16 * (item - first);
            }
            if (has && item == 0 && rb == 0) p.slot_adapter[tile * p.cap + slot] = l;
            items += __shfl_sync(0xffffffffu, s_it, 31);
            slots += __shfl_sync(0xffffffffu, s_sl, 31);
        }
        if (lane == 0 && item == 0 && rb == 0) p.slot_cnt[tile] = slots;
        __syncwarp();
        const int l = pick[0];
        if (l >= 0) {  // this item's rows: those of adapter l, from the pick[2]-th on
            int seen = 0;
            for (int i0 = 0; i0 < p.tile; i0 += 32) {
                const bool m = i0 + lane < p.tile && ad[i0 + lane] == l;
                const uint32_t b = __ballot_sync(0xffffffffu, m);
                const int at = seen + __popc(b & ((1u << lane) - 1u)) - pick[2];
                if (m && at >= 0 && at < 16) rows[at] = i0 + lane;
                seen += __popc(b);
            }
        }
    }
    __syncthreads();
    const int l = pick[0];
    if (l < 0) return;
    __nv_bfloat16 *hi =
        p.v + ((int64_t)(tile * p.cap + pick[1]) * p.blocks * p.tile) * p.r64 + rb * 16;
    const int64_t block = (int64_t)p.tile * p.r64;
    // zero rows of the other adapters (the slot's first item), and the columns
    // past the rank (its first rank block)
    if (pick[2] == 0)
        for (int i = tid; i < p.tile; i += kLThreads) {
            __nv_bfloat16 *d = hi + (int64_t)i * p.r64;
            if (ad[i] != l) zero_v<P>(d, 1, p.per, block);
            if (rb == 0) zero_v<P>(d + 16 * rblocks, (p.per == 1 ? p.r64 / 16 : p.per == 2 ? 2 : 1) - rblocks, p.per, block);
        }
    // this lane's x rows (g, g + 8) and adapter rows (ranks g, g + 8 of the block)
    const int g = lane >> 2, c8 = 8 * (lane & 3);
    const int i0 = rows[g] < 0 ? rows[0] : rows[g], i1 = rows[g + 8] < 0 ? rows[0] : rows[g + 8];
    const int64_t x0 = (int64_t)(row0 + i0) * p.K + c8, x1 = (int64_t)(row0 + i1) * p.K + c8;
    const int r0 = min(rb * 16 + g, p.r - 1), r1 = min(rb * 16 + g + 8, p.r - 1);
    const __nv_bfloat16 *a0 = p.a + ((int64_t)l * p.r + r0) * p.K + c8;
    const __nv_bfloat16 *a1 = p.a + ((int64_t)l * p.r + r1) * p.K + c8;
    float d0[4] = {}, d1[4] = {};  // rows 0-7, 8-15
    constexpr int kU = BF16 ? 2 : 1;
    auto go = [&](auto count, int s0) {
        constexpr int U = decltype(count)::value;
        uint4 wa[U], wb[U];
        X8<BF16> xa[U], xb[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (s0 + u) * 32;
            xa[u].load(p.x, x0 + k);
            xb[u].load(p.x, x1 + k);
            wa[u] = __ldg(reinterpret_cast<const uint4 *>(a0 + k));
            wb[u] = __ldg(reinterpret_cast<const uint4 *>(a1 + k));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t f0[4] = {wa[u].x, wb[u].x, wa[u].y, wb[u].y};
            const uint32_t f1[4] = {wa[u].z, wb[u].z, wa[u].w, wb[u].w};
#pragma unroll
            for (int i = 0; i < X8<BF16>::kMost; ++i) {
                if (i == P) break;
                const uint4 x = xa[u].template next<P>(), y = xb[u].template next<P>();
                mma_16816(d0, f0, x.x, x.y);
                mma_16816(d1, f0, y.x, y.y);
                mma_16816(d0, f1, x.z, x.w);
                mma_16816(d1, f1, y.z, y.w);
            }
        }
    };
    const int steps = p.K / 32;  // K is a multiple of 32
    int s0 = warp * kU;
#pragma unroll 1
    for (; s0 + kU <= steps; s0 += kLWarps * kU) go(std::integral_constant<int, kU>{}, s0);
    if (kU > 1 && s0 < steps) go(std::integral_constant<int, 1>{}, s0);
    const int c2 = 2 * (lane & 3);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        acc[warp][c2 + (e & 1)][g + 8 * (e >> 1)] = d0[e];
        acc[warp][8 + c2 + (e & 1)][g + 8 * (e >> 1)] = d1[e];
    }
    __syncthreads();
    if (tid < 256) {
        const int i = tid >> 4, c = tid & 15, row = rows[i];
        float v = 0.0f;
#pragma unroll
        for (int q = 0; q < kLWarps; ++q) v += acc[q][i][c];
        if (p.alpha != nullptr) v *= __ldg(p.alpha + l);
        if (row >= 0) {
            if (rb * 16 + c >= p.r) v = 0.0f;
            store_v<P>(hi + (int64_t)row * p.r64 + c, v, p.per, block);
        }
    }
}

bool is_aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool packed(int f) { return f == FP8G_E2M1 || f == FP8G_E2M3 || f == FP8G_E3M2; }
constexpr int64_t kMaxDim = (int64_t)1 << 31;
constexpr int64_t kMaxVBytes = (int64_t)1 << 30;

}  // namespace

}  // namespace fp8g

using namespace fp8g;

// Rows row0 .. row0 + M - 1 of a call whose arguments hold, x, adapter and C theirs.
static fp8g_status lora_rows(const HostDevice &d, int64_t row0, const void *x, int32_t x_dtype, const void *W,
                             const uint8_t *sfw, int32_t w_fmt, const void *lora_a, const void *lora_b,
                             const float *alpha, const int32_t *adapter, int32_t L, int32_t r, const float *bias,
                             void *C, int out, int64_t M, int64_t N, int64_t K, cudaStream_t stream) {
    const bool lora = L > 0;
    fp8g_status st = FP8G_OK;
    const LoraV lv(lora ? r : 1, out == FP8G_OUT_F32);
    const int32_t ks = (int32_t)((K + 127) / 128), n_rt = (int32_t)((N + 127) / 128);
    // CTA pairs from 513 rows on, and from 129 where the low-rank steps of a tile
    // are few beside its FP8 steps: they make all of a pair's 256 rows wait, where
    // the streaming kernel covers an adapter's columns.  256 rows at 4096 x 14336:
    // 8 adapters of rank 16 30.8 us (streamed 37.1), 32 of rank 64 63.9 (55.2); 128
    // rows: 30.3 (31.4) and 63.1 (43.0).
    const int most = lora ? (L < kMaxTile ? L : kMaxTile) * lv.kr * lv.blocks : 0;
    const bool pair = M > kStreamLoraRows || (M > kStreamMaxTokens && 2 * most <= ks);
    const int nb = pair ? 256 : stream_columns(M);
    const int tiles = (int)((M + nb - 1) / nb), cap = L < nb ? L : nb;
    const int32_t n_rtA = (int32_t)((M + 127) / 128);
    // rows of V and of the scales: 32-bit TMA coordinates
    if ((int64_t)tiles * cap * lv.blocks * nb >= kMaxDim || (int64_t)ks * n_rtA >= kMaxDim)
        return FP8G_ERR_UNSUPPORTED_SHAPE;
    StreamParams p{};
    StreamPhase &h = p.ph[0];
    if (!pair) {
        // one weight tile a ticket where pairs of them would be few: 33 rows at 4096 x
        // 14336 27.4 us by one, 29.6 by pairs; 4096 x 28672 41.7 and 35.5
        h.sub = tiles * ((N + 255) / 256) * 8 >= d.num_sms * 5 ? 2 : 1;
        h.mt = (int32_t)((N + 128 * h.sub - 1) / (128 * h.sub));
        stream_sizes(p, nb, h.sub, true, lv.blocks);
        h.ks = ks;
        h.rows = (int32_t)N;
        h.n_rt = n_rt;
        p.kr = lora ? lv.kr : 0;
        if ((int64_t)tiles * h.mt * (ks + (int64_t)cap * p.kr) >= INT32_MAX) return FP8G_ERR_UNSUPPORTED_SHAPE;
    }
    size_t at = 0;
    auto take = [&at](size_t bytes) {
        const size_t o = at;
        at += (bytes + 1023) / 1024 * 1024;
        return o;
    };
    const size_t o_xq = take((size_t)M * K), o_xsf = take((size_t)(pair ? n_rtA : tiles) * ks * 512);
    const size_t o_v = take((size_t)tiles * cap * lv.blocks * nb * lv.r64 * 2);
    const size_t o_part = take(pair ? (size_t)tiles * 4 : stream_part_bytes(p, d.num_sms));
    p.n_counters = 3 + kStreamSplitTiles;
    const size_t o_cnt = take(pair ? (size_t)tiles * cap * 4 : (size_t)p.n_counters * 4);
    cudaMemPool_t pool;
    if ((st = host_pool(d.dev, pool)) != FP8G_OK) return st;
    void *wsv = nullptr;
    if (cudaMallocFromPoolAsync(&wsv, at, pool, stream) != cudaSuccess) return FP8G_ERR_CUDA;
    uint8_t *ws = static_cast<uint8_t *>(wsv);
    CUtensorMap mb{}, mv{}, mv32{}, mv1{};
    if (lora) {
        const uint64_t db[3] = {(uint64_t)r, (uint64_t)N, (uint64_t)L};
        const uint32_t bb[3] = {64u, 128u, 1u};
        st = host_bf16_map(lora_b, 3, db, bb, d.dev, mb);
        if (pair) {
            const uint64_t dv[2] = {(uint64_t)lv.r64, (uint64_t)tiles * cap * lv.blocks * nb};
            const uint32_t bv[2] = {64u, 128u};
            if (st == FP8G_OK) st = host_bf16_map(ws + o_v, 2, dv, bv, d.dev, mv);
        } else {
            // boxes of 16 and 32 rows of all blocks, of 16 rows of one (LoraV), as far as used
            const uint64_t dv[3] = {(uint64_t)lv.r64, (uint64_t)nb, (uint64_t)tiles * cap * lv.blocks};
            const uint32_t b16[3] = {64u, 16u, (uint32_t)lv.blocks}, b32[3] = {64u, 32u, (uint32_t)lv.blocks};
            const uint32_t b1[3] = {64u, 16u, 1u};
            if (st == FP8G_OK) st = host_bf16_map(ws + o_v, 3, dv, b16, d.dev, mv);
            mv1 = mv;
            if (st == FP8G_OK && lv.blocks > 1) st = host_bf16_map(ws + o_v, 3, dv, b1, d.dev, mv1);
            if (st == FP8G_OK && lv.blocks > 1 && lv.pieces == 3)
                st = host_bf16_map(ws + o_v, 3, dv, b32, d.dev, mv32);
        }
    }
    const bool bf16 = x_dtype == FP8G_IN_BF16;
    cudaError_t e = cudaSuccess;
    if (st == FP8G_OK && !pair) {
        const uint64_t dw[3] = {(uint64_t)K, (uint64_t)N, 1u};
        const uint32_t bw[3] = {(uint32_t)kBK, 128u, 1u};
        const uint64_t dx[2] = {(uint64_t)K, (uint64_t)M};
        const uint32_t bx[2] = {(uint32_t)kBK, 16u};
        st = host_operand_map(W, w_fmt, 3, dw, bw, d.dev, h.W);
        const uint32_t by[2] = {(uint32_t)kBK, 64u};
        if (st == FP8G_OK) st = host_operand_map(ws + o_xq, FP8G_E4M3, 2, dx, bx, d.dev, h.X);
        if (st == FP8G_OK && nb % 64 == 0) st = host_operand_map(ws + o_xq, FP8G_E4M3, 2, dx, by, d.dev, h.X64);
        h.sfw = sfw;
        h.sfx = ws + o_xsf;
        p.w_fmt = host_mma_type(w_fmt) << 7;
        p.gap8 = host_gap8(w_fmt);
        p.x = x;
        p.x_bf16 = bf16;
        p.T = (int32_t)M;
        p.first_row = (int32_t)row0;
        p.K = (int32_t)K;
        p.idx = lora ? adapter : nullptr;
        p.n_idx = (int32_t)M;
        p.n_mat = L;
        p.xq = ws + o_xq;
        p.xsf = ws + o_xsf;
        p.counters = reinterpret_cast<int32_t *>(ws + o_cnt);
        h.part = reinterpret_cast<float *>(ws + o_part);
        h.part_cnt = p.counters + 3;
        p.out = C;
        p.out_f32 = out == FP8G_OUT_F32;
        p.status = d.status;
        p.timeout_ns = d.timeout_ns;
        p.B = mb;
        p.V = mv;
        p.V32 = mv32;
        p.V1 = mv1;
        p.w = static_cast<const uint8_t *>(W);
        p.b = lora_b;
        p.fmt = w_fmt;
        p.a = lora_a;
        p.alpha = alpha;
        p.bias = bias;
        p.v = ws + o_v;
        p.rank = lora ? r : 0;  // 0: the kernels read no idx
        p.r64 = lv.r64;
        p.pieces = lv.pieces;
        p.per = lv.per;
        p.blocks = lv.blocks;
        p.slot_cap = cap;
        if (st == FP8G_OK) e = launch_stream(true, p, d.num_sms, stream);
    } else if (st == FP8G_OK) {
        LoraPrep a{};
        a.x = x;
        a.M = (int32_t)M;
        a.K = (int32_t)K;
        a.xq = ws + o_xq;
        a.xsf = ws + o_xsf;
        a.ks = ks;
        a.n_rt = n_rtA;
        a.a = static_cast<const __nv_bfloat16 *>(lora_a);
        a.alpha = alpha;
        a.adapter = adapter;
        a.L = L;
        a.r = r;
        a.r64 = lv.r64;
        a.per = lv.per;
        a.blocks = lv.blocks;
        a.tile = nb;
        a.cap = cap;
        a.tiles = lora ? tiles : 0;
        a.v = reinterpret_cast<__nv_bfloat16 *>(ws + o_v);
        a.slot_cnt = reinterpret_cast<int32_t *>(ws + o_part);
        a.slot_adapter = reinterpret_cast<int32_t *>(ws + o_cnt);
        a.row0 = (int32_t)row0;
        a.items = nb / 16 + cap;  // at most one partly filled item per slot beside the whole ones
        a.status = d.status;
        if (lora) {
            const int64_t blocks = (int64_t)tiles * ((r + 15) / 16) * a.items;
            auto kern = lv.pieces == 3 ? (bf16 ? lora_v_kernel<3, true> : lora_v_kernel<3, false>)
                                       : (bf16 ? lora_v_kernel<2, true> : lora_v_kernel<2, false>);
            e = blocks >= INT32_MAX
                    ? cudaErrorInvalidValue
                    : launch_programmatic(kern, dim3((unsigned)blocks), dim3(kLThreads), stream, a);
        }
        if (e == cudaSuccess)
            e = bf16 ? launch_programmatic(lora_quant_kernel<true>, dim3((unsigned)M), dim3(256), stream, a)
                     : launch_programmatic(lora_quant_kernel<false>, dim3((unsigned)M), dim3(256), stream, a);
        PairLora pl{};
        if (lora) {
            pl.V = mv;
            pl.B = mb;
            pl.slots = a.slot_cnt;
            pl.adapters = a.slot_adapter;
            pl.cap = cap;
            pl.rank = r;
            pl.kr = lv.kr;
            pl.pieces = lv.pieces;
            pl.per = lv.per;
            pl.blocks = lv.blocks;
            pl.r64 = lv.r64;
            pl.L = L;
            pl.fmt = w_fmt;
            pl.row_adapter = adapter;
            pl.x = a.xq;
            pl.w = static_cast<const uint8_t *>(W);
            pl.v = a.v;
            pl.b = lora_b;
        }
        if (e == cudaSuccess)
            st = run_pair_packed(a.xq, a.xsf, W, sfw, w_fmt, bias, C, out, M, N, K, lora ? &pl : nullptr, stream);
    }
    const cudaError_t ef = cudaFreeAsync(wsv, stream);
    if (st != FP8G_OK) return st;
    return e == cudaSuccess && ef == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}

extern "C" fp8g_status fp8_gemm_lora(const void *x, int32_t x_dtype, const void *W, const uint8_t *sfw,
                                     int32_t w_fmt, const void *lora_a, const void *lora_b,
                                     const float *alpha, const int32_t *adapter, int32_t L, int32_t r,
                                     const float *bias, void *C, int out, int64_t M, int64_t N, int64_t K,
                                     cudaStream_t stream) {
    if (x_dtype != FP8G_IN_F32 && x_dtype != FP8G_IN_BF16) return FP8G_ERR_INVALID_ARG;
    if (out != FP8G_OUT_BF16 && out != FP8G_OUT_F32) return FP8G_ERR_INVALID_ARG;
    if (w_fmt < FP8G_E4M3 || w_fmt > FP8G_E3M2) return FP8G_ERR_INVALID_ARG;
    if (M < 0 || N < 1 || K < 1 || L < 0 || (L > 0 && r < 1)) return FP8G_ERR_INVALID_ARG;
    if (W == nullptr || sfw == nullptr) return FP8G_ERR_INVALID_ARG;
    if (M > 0 && (x == nullptr || C == nullptr)) return FP8G_ERR_INVALID_ARG;
    const bool lora = L > 0;
    if (lora && (lora_a == nullptr || lora_b == nullptr || (M > 0 && adapter == nullptr)))
        return FP8G_ERR_INVALID_ARG;
    if (K % (packed(w_fmt) ? 128 : 32) != 0 || (lora && r % 8 != 0)) return FP8G_ERR_UNSUPPORTED_SHAPE;
    if (L > FP8G_MAX_ADAPTERS || (lora && r > FP8G_MAX_LORA_RANK) || M >= (1 << 24) || N >= (1 << 24) ||
        K >= (1 << 24))
        return FP8G_ERR_UNSUPPORTED_SHAPE;
    if (!is_aligned(x, 16) || !is_aligned(C, 16) || !is_aligned(W, packed(w_fmt) ? 32 : 16) ||
        !is_aligned(sfw, 16) || !is_aligned(bias, 4) || (N * (out == FP8G_OUT_F32 ? 4 : 2)) % 16 != 0)
        return FP8G_ERR_ALIGNMENT;
    if (lora && (!is_aligned(lora_a, 16) || !is_aligned(lora_b, 16) || !is_aligned(alpha, 4) ||
                 !is_aligned(adapter, 4)))
        return FP8G_ERR_ALIGNMENT;
    HostDevice d;
    const fp8g_status st = host_device(d);
    if (st != FP8G_OK) return st;
    // V's temporary has a slot for every adapter in every 256 rows, as many as a tile
    // might use (8192 rows, rank 64, 256 adapters loaded: 537 MB): rows in even shares
    // of at most kMaxVBytes of it, so that it does not grow with them (262144 rows of
    // rank 256 would take 69 GB; from 2^22 on V's rows would pass 31 bits)
    int64_t step = M;
    if (lora && M > kStreamLoraRows) {
        const LoraV lv(r, out == FP8G_OUT_F32);
        const int64_t tile = (int64_t)(L < kMaxTile ? L : kMaxTile) * lv.blocks * kMaxTile * lv.r64 * 2;
        const int64_t tiles = (M + kMaxTile - 1) / kMaxTile, most = kMaxVBytes / tile;
        const int64_t shares = (tiles + most - 1) / most;
        step = (tiles + shares - 1) / shares * kMaxTile;
    }
    for (int64_t i = 0; i < M; i += step) {
        const fp8g_status si =
            lora_rows(d, i, static_cast<const uint8_t *>(x) + i * K * (x_dtype == FP8G_IN_BF16 ? 2 : 4), x_dtype,
                      W, sfw, w_fmt, lora_a, lora_b, alpha, lora ? adapter + i : nullptr, L, r, bias,
                      static_cast<uint8_t *>(C) + i * N * (out == FP8G_OUT_F32 ? 4 : 2), out,
                      M - i < step ? M - i : step, N, K, stream);
        if (si != FP8G_OK) return si;
    }
    return FP8G_OK;
}
