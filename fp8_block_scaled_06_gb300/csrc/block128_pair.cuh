// Products with fp32 scales for blocks of 128 on CTA pairs, sm_103a:
//
//   C[i, j] = sum_kb sa[kb][i] sb(kb, j) P_kb[i, j],  P_kb = sum_{k in kb} a_ik b_kj
//
// and the gated projection pair that ends in 8 bits,
//   g = x Wg^T, u = x Wu^T, h = act(g) u  ->  codes and scales of h (and of g, u).
//
// The tensor core takes no fp32 scales, so each K block's unscaled product P_kb
// goes to one of two 256-column tensor-memory buffers (kind::f8f6f4, the first of
// its four MMAs overwrites) and eight promotion warps per CTA add it, scaled, to
// fp32 registers while the MMAs of the next K block fill the other buffer.  The four
// MMAs of a pair's 256 x 256 tile take 725 cycles a K block; a buffer that is filled has to
// be read and released within that time, latencies included, or the MMAs wait.  So between
// a product's arrival and the release the promotion warps do nothing else, the release is
// a relaxed arrival (with release semantics it waited for copies in flight: 2500 cycles a
// K block), the MMA warp stays whole and one elected lane issues (one lane's own branch:
// 1020), and two other warps copy all scales (a ring of each promotion warp's own: 5% of
// 8192 cubed).  Measured 8192 x 8192 x 8192: 345 us, 3190 TFLOP/s, as the kernel whose
// scales the tensor core applies (gemm_pair.cu, powers of two for blocks of 32).
//
// A promotion warp has 32 rows and 128 columns.  Where one scale serves 128 columns (tiles
// of B), a lane has a row: 4 loads of 32 columns, 128 FMAs.  With a scale per column
// (weight gradients) it has two columns of four rows in each fragment of 8 x 16, so that it
// reads a quarter of the columns' scales (a row a lane, shared memory took 1024 cycles a K
// block to hand them out), in packed pairs; those loads take three times as long, and
// loads, arithmetic and scales come one after the other: 1200 cycles a K block, 1860
// TFLOP/s at 4096 x 14336 x 4096.
//
// Operands lie either way.  Contraction contiguous: 128 B rows of the 128-byte
// swizzle, an MMA's 32 values 32 B apart.  M (N) contiguous: the tile's 128 rows are
// the K values, an MMA's 32 of them 4 KB apart, and the instruction descriptor's
// major bit is set.  In both the eight-row swizzle atoms follow each other (1 KB),
// so the weights serve the forward product and the input gradient as they lie, and
// activations the forward product and the weight gradient.
//
// Roles (384 threads): warp 0 TMA producer (both CTAs, their own halves), warp 1 of
// the even CTA MMA issue, warps 2 and 3 scales (chunks of eight K blocks, two ahead), warps
// 4-11 promotion and epilogue: lane quarter warp & 3, 64 columns of either half of the
// tile.  These hold 128 accumulators a thread, so registers move to them (setmaxnreg: 256
// x 232 + 128 x 40 = 384 x 168).  Every wait is bounded.
#pragma once
#include <cuda_bf16.h>

#include "block128.h"
#include "block128_math.cuh"
#include "block128_wait.cuh"
#include "ptx.cuh"

namespace fp8g {

namespace {

constexpr int kThreads = 384;
constexpr int kProm0 = 4;              // first promotion warp
constexpr int kPromWarps = 8;
constexpr int kRegsLaunch = 168, kRegsProm = 232, kRegsRest = 40;
static_assert(32 * kPromWarps * kRegsProm + 128 * kRegsRest <= kThreads * kRegsLaunch,
              "setmaxnreg draws on the block's own registers");
constexpr int kTile = kBlk * kBlk;     // bytes of an operand tile of one CTA
constexpr int kBufs = 2;               // product buffers of 256 columns
constexpr int kUnit = 32 * 64;

template <bool VECB>
struct Lay {
    static constexpr int STAGES = 5;
    static constexpr int OFF_B = STAGES * kTile;
    // output on its way: two units of 32 rows of 64 bytes a promotion warp
    static constexpr int OFF_C = 2 * STAGES * kTile;
    // scales of CH K blocks: A's [CH][128 rows], then B's [CH][256 columns] or [CH][two
    // tiles]; two such chunks
    static constexpr int CH = 8;
    static constexpr int SCALES = CH * (kBlk + (VECB ? 2 * kBlk : 2));
    static constexpr int OFF_S = OFF_C + kPromWarps * 2 * kUnit;
    static constexpr int OFF_X = OFF_S + 2 * SCALES * 4;  // row maxima: [2][2][128] float4
    static constexpr int OFF_BAR = OFF_X + (VECB ? 0 : 2 * 2 * kBlk * 16);
    // full, empty [STAGES]; product full, product empty [kBufs]; row maxima [lane
    // quarter]; scales full, empty [2]; drain
    static constexpr int NUM_BARS = 2 * STAGES + 2 * kBufs + 4 + 4 + 1;
    static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
    static constexpr int BYTES = OFF_MISC + 16 + 1024;
    static_assert(BYTES <= 232448, "shared memory over the per-CTA limit");
};

// What pair c computes i-th: K blocks [k0, k1) of tile t.  A share of a tile's K blocks
// that does not reach its end comes first (`publish`: its sums go to memory), the one
// that does comes last and adds those of pairs [from, c) in their order: by then they are
// there, and a pair waits only for pairs before it, which run (they are numbered as they
// begin) and wait for nothing before they publish.
struct Item {
    int32_t t, k0, k1, from;
    bool publish;
};

template <bool SHARE>
__device__ __forceinline__ bool item(const B128Params &p, int32_t c, int32_t i, Item &o) {
    o.publish = false;
    o.from = c;
    o.k0 = 0;
    o.k1 = p.num_kb;
    if constexpr (!SHARE) {
        o.t = p.first + c + i * p.pairs;
        return o.t < p.T;
    }
    const int32_t kb = p.num_kb, all = (p.T - p.first) * kb;
    const int32_t u0 = min(c * p.share, all), u1 = min(u0 + p.share, all);
    if (u0 >= u1) return false;
    const int32_t r1 = (u1 - 1) / kb, end = u1 - r1 * kb;
    if (end < kb) {
        if (i == 0) {
            o.t = p.first + r1;
            o.k0 = max(u0 - r1 * kb, 0);
            o.k1 = end;
            o.publish = true;
            return true;
        }
        --i;
    }
    const int32_t r0 = u0 / kb;
    if (i > 0 || u1 < (r0 + 1) * kb) return false;
    o.t = p.first + r0;
    o.k0 = u0 - r0 * kb;
    if (o.k0 > 0) o.from = r0 * kb / p.share;
    return true;
}

__device__ __forceinline__ int32_t ld_acquire(const int32_t *a) {
    int32_t v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(a) : "memory");
    return v;
}
__device__ __forceinline__ void st_release(int32_t *a, int32_t v) {
    asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(a), "r"(v) : "memory");
}

// Until *flag is set (whole warp); bounded.
__device__ __forceinline__ bool wait_flag(const int32_t *flag, volatile int *abort_flag, const B128Params &p) {
    int ok = 1;
    if ((threadIdx.x & 31) == 0) {
        const uint64_t t0 = ptx::globaltimer();
        while (ld_acquire(flag) == 0) {
            if (*abort_flag) ok = 0;
            if (ok && ptx::globaltimer() - t0 > p.timeout_ns) {
                *abort_flag = 1;
                record_error(p, FP8G_ERR_TIMEOUT, 4 * 256);
                ok = 0;
            }
            if (!ok) break;
        }
    }
    ok = __shfl_sync(0xffffffffu, ok, 0);
    __syncwarp();
    return ok != 0;
}

// One K block's scales of the two warps that copy them: lane l of 64 has rows l and l + 64
// of the CTA's 128, and four columns of the tile's 256 (VECB) or, of the first 2 CH
// lanes, one of its two tiles of B in K block l / 2 of the chunk.
template <bool VECB, int OUT>
struct ScaleSource {
    const float *a0, *a1, *b;
    __device__ __forceinline__ void tile(const B128Params &p, int l, int64_t row0, int pn, int32_t k0) {
        a0 = p.sa + k0 * p.M + min(row0 + l, p.M - 1);
        a1 = p.sa + k0 * p.M + min(row0 + l + 64, p.M - 1);
        if constexpr (VECB) {  // (N is a multiple of 16)
            b = p.sb + k0 * p.N + min((int64_t)pn * 2 * kBlk + 4 * l, p.N - 4);
        } else {
            const int64_t n0 = OUT >= kB128Gated ? pn : 2 * pn;
            const int64_t n1 = OUT >= kB128Gated ? n0 + p.n_blocks : min(n0 + 1, (int64_t)p.n_blocks - 1);
            b = p.sb + ((l & 1) == 0 ? n0 : n1) * p.sb_n + (k0 + (l >> 1)) * p.sb_k;
        }
    }
};

// A promotion warp's output: units of 32 rows of 64 bytes, in the 64-byte swizzle, that TMA
// writes while the next one is made.  (Stored from registers, a row a lane, 32 lines an
// instruction: 3000 cycles a tile, and the MMAs waited.  Measured 4096 x 14336 x 4096: bf16 166 ->
// 160 us, fp32 188 -> 178, weight gradient added 285 -> 277; gated, with the checkpoint,
// 380 -> 367.  Five stages of operands make room for it and cost nothing.)
struct Output {
    uint32_t base;  // two units of shared memory
    int lane;
    uint32_t n;     // units of this tile so far
    // (made for each tile: nothing of it is kept in registers over the K blocks)
    __device__ __forceinline__ Output(uint32_t base_, int lane_) : base(base_), lane(lane_), n(0u) {
        if (lane == 0) ptx::bulk_wait_read<0>();
        __syncwarp();
    }
    __device__ __forceinline__ uint32_t begin() {
        if (n >= 2u) {
            if (lane == 0) ptx::bulk_wait_read<1>();
            __syncwarp();
        }
        return base + (n++ & 1u) * kUnit;
    }
    // where 16-byte piece `piece` of row r lies in the unit at `at`
    static __device__ __forceinline__ uint32_t piece(uint32_t at, int r, int piece) {
        return at + r * 64 + ((piece ^ ((r >> 1) & 3)) << 4);
    }
    // in: some of it lies in the matrix.  (The one lane asks; a branch of the warp around the
    // unit made the K blocks' loop slower, 8192 cubed 343 -> 363 us.)
    template <bool ADD>
    __device__ __forceinline__ void end(const CUtensorMap &map, uint32_t at, int64_t x, int64_t y, bool in) {
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            if (in) {
                if constexpr (ADD)
                    ptx::tma_add_2d(&map, at, (int32_t)x, (int32_t)y);
                else
                    ptx::tma_store_2d(&map, at, (int32_t)x, (int32_t)y);
            }
            ptx::bulk_commit();
        }
    }
    // one unit of which this lane has row `lane`
    template <bool ADD>
    __device__ __forceinline__ void row(const CUtensorMap &map, const uint32_t (&w)[16], int64_t x, int64_t y, bool in) {
        const uint32_t at = begin();
#pragma unroll
        for (int j = 0; j < 4; ++j) ptx::st_shared_v4(piece(at, lane, j), w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        end<ADD>(map, at, x, y, in);
    }
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t v;
    asm volatile("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(hi), "f"(lo));
    return v;
}

// 64 codes of one row from 64 values times r.
__device__ __forceinline__ void codes64(uint32_t (&o)[16], const float (&v)[64], float r) {
#pragma unroll
    for (int w = 0; w < 16; ++w)
        o[w] = b128_codes<FP8G_E4M3>(v[4 * w], v[4 * w + 1], v[4 * w + 2], v[4 * w + 3], r);
}

__device__ __forceinline__ float amax64(const float (&v)[64]) {
    float m[2] = {};
#pragma unroll
    for (int i = 0; i < 64; i += 2) m[(i >> 1) & 1] = b128_max3(m[(i >> 1) & 1], v[i], v[i + 1]);
    return fmaxf(m[0], m[1]);
}

template <bool VECB, int OUT, bool SHARE>
__global__ void __launch_bounds__(kThreads, 1)
    b128_pair_kernel(const __grid_constant__ B128Maps m, const B128Params p) {
    const CUtensorMap &tmA = m.A, &tmB = m.B;
    using L = Lay<VECB>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = ptx::smem_addr(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (raw_base & 1023u)) & 1023u);
    const uint32_t sbase = ptx::smem_addr(smem);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_rank();
    const bool leader = rank == 0;

    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::OFF_BAR);
    auto bar_full = [&](int s) { return ptx::smem_addr(&bars[s]); };
    auto bar_empty = [&](int s) { return ptx::smem_addr(&bars[L::STAGES + s]); };
    auto bar_pfull = [&](int b) { return ptx::smem_addr(&bars[2 * L::STAGES + b]); };
    auto bar_pempty = [&](int b) { return ptx::smem_addr(&bars[2 * L::STAGES + kBufs + b]); };
    auto bar_max = [&](int q) { return ptx::smem_addr(&bars[2 * L::STAGES + 2 * kBufs + q]); };
    auto bar_sfull = [&](int i) { return ptx::smem_addr(&bars[2 * L::STAGES + 2 * kBufs + 4 + i]); };
    auto bar_sempty = [&](int i) { return ptx::smem_addr(&bars[2 * L::STAGES + 2 * kBufs + 6 + i]); };
    const uint32_t bar_drain = ptx::smem_addr(&bars[L::NUM_BARS - 1]);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::OFF_MISC + 4);

    // ------------------------------------------------------------ setup
    if (threadIdx.x == 0) {
        for (int s = 0; s < L::STAGES; ++s) {
            ptx::mbar_init(bar_full(s), 1);
            ptx::mbar_init(bar_empty(s), 1);
        }
        for (int b = 0; b < kBufs; ++b) {
            ptx::mbar_init(bar_pfull(b), 1);
            ptx::mbar_init(bar_pempty(b), 2 * kPromWarps);
        }
        for (int i = 0; i < 4; ++i) ptx::mbar_init(bar_max(i), 2);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(bar_sfull(i), 64);
            ptx::mbar_init(bar_sempty(i), kPromWarps);
        }
        ptx::mbar_init(bar_drain, 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        ptx::prefetch_tmap(&tmA);
        ptx::prefetch_tmap(&tmB);
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(ptx::smem_addr(tmem_slot), 512);
        ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();  // both CTAs' barriers and tensor memory exist
    ptx::tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    if (tmem_base != 0u && threadIdx.x == 0) {  // all 512 columns: they begin at 0 in both CTAs
        record_error(p, FP8G_ERR_DEVICE, 0xA11Cu);
        *abort_flag = 1;
    }
    ptx::grid_dep_wait();  // global memory only after the previous kernel
    ptx::grid_dep_launch();
    __syncthreads();
    int32_t pair = (int32_t)ptx::cluster_id_x();
    if constexpr (SHARE) {
        // pairs count in the order in which they begin: one waits only for pairs that run
        int32_t *ticket = reinterpret_cast<int32_t *>(smem + L::OFF_MISC + 8);
        if (leader && threadIdx.x == 0) *ticket = atomicAdd(p.there + p.pairs * 16, 1);
        ptx::cluster_sync();
        pair = ptx::ld_cluster_s32(ptx::map_shared(ptx::smem_addr(ticket), 0));
    }
    const bool run = !*abort_flag;

    // (each in its own branch: the compiler allots a branch's registers by it)
    if (warp < kProm0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
        if (warp == 0) {
            // ===== TMA producer: both CTAs' copies complete on the even CTA's barrier =====
            if (lane == 0) {
                uint32_t stage = 0, phase = 0;
                Item it;
                for (int32_t i = 0; run && item<SHARE>(p, pair, i, it); ++i) {
                    int32_t pm, pn;
                    raster(it.t, p.npm, p.npn, kRasterG, pm, pn);
                    const int32_t m0 = (2 * pm + (int32_t)rank) * kBlk, n0 = (2 * pn + (int32_t)rank) * kBlk;
                    for (int kb = it.k0; kb < it.k1; ++kb) {
                        if (!wait_bar(bar_empty(stage), phase ^ 1u, abort_flag, p, 0 * 256 + stage)) goto roles_done;
                        const uint32_t fb = leader ? bar_full(stage) : ptx::map_shared(bar_full(stage), 0);
                        if (leader) ptx::mbar_arrive_expect_tx(fb, 4 * kTile);
                        const int32_t k0 = kb * kBlk;
                        ptx::tma_load_2d_pair(sbase + stage * kTile, &tmA, fb, p.a_mn ? m0 : k0, p.a_mn ? k0 : m0);
                        if constexpr (OUT >= kB128Gated)  // gate rows to the even CTA, up rows to the odd one
                            ptx::tma_load_3d_pair(sbase + L::OFF_B + stage * kTile, &tmB, fb, k0, pn * kBlk, (int32_t)rank);
                        else
                            ptx::tma_load_2d_pair(sbase + L::OFF_B + stage * kTile, &tmB, fb, p.b_mn ? n0 : k0,
                                                  p.b_mn ? k0 : n0);
                        if (++stage == L::STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                }
            }
        } else if (warp == 1 && leader) {
            // ===== MMA issue (even CTA): 256 x 256 x 32 per instruction =====
            // The whole warp runs the loop and one elected lane issues: from a branch of one
            // lane's own the four MMAs took 500 cycles to issue, in the chain from a buffer's
            // release to its next product.
            const uint32_t idesc = ptx::idesc_f8(2 * kBlk, 2 * kBlk) | p.types;
            const uint32_t a_step = (p.a_mn ? 32 * kBlk : 32) >> 4, b_step = (p.b_mn ? 32 * kBlk : 32) >> 4;
            const uint64_t a_desc = ptx::smem_desc(sbase, 1024, 1024, 2);
            const uint64_t b_desc = ptx::smem_desc(sbase + L::OFF_B, 1024, 1024, 2);
            uint32_t stage = 0, phase = 0, g = 0;
            Item it;
            for (int32_t i = 0; run && item<SHARE>(p, pair, i, it); ++i) {
                for (int kb = it.k0; kb < it.k1; ++kb, ++g) {
                    const uint32_t buf = g & 1u;
                    if (!b128_wait_all(bar_full(stage), phase, abort_flag, p, 1 * 256 + stage)) goto roles_done;
                    if (!b128_wait_all(bar_pempty(buf), ((g >> 1) & 1u) ^ 1u, abort_flag, p, 1 * 256 + 64 + buf))
                        goto roles_done;
                    ptx::tc_fence_after();
                    const uint64_t a0 = a_desc + stage * (kTile >> 4), b0 = b_desc + stage * (kTile >> 4);
                    if (ptx::elect_one()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            ptx::mma_f8_pair(buf * 2 * kBlk, a0 + k * a_step, b0 + k * b_step, idesc, k != 0 ? 1u : 0u);
                        ptx::tc_commit_pair_mc(bar_pfull(buf), 0x3);
                        ptx::tc_commit_pair_mc(bar_empty(stage), 0x3);
                    }
                    __syncwarp();
                    if (++stage == L::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
        } else if (warp >= 2) {
            // ===== scales: chunks of CH K blocks, two of them ahead, over all items =====
            const int l = (int)threadIdx.x - 64;
            uint32_t c = 0;
            Item it;
            for (int32_t i = 0; run && item<SHARE>(p, pair, i, it); ++i) {
                int32_t pm, pn;
                raster(it.t, p.npm, p.npn, kRasterG, pm, pn);
                ScaleSource<VECB, OUT> src;
                src.tile(p, l, (2 * (int64_t)pm + rank) * kBlk, pn, it.k0);
                const int32_t n = it.k1 - it.k0;
                for (int32_t kb = 0; kb < n; kb += L::CH, ++c) {
                    if (!b128_wait_all(bar_sempty(c & 1u), ((c >> 1) & 1u) ^ 1u, abort_flag, p, 2 * 256 + (c & 1u)))
                        goto roles_done;
                    const uint32_t at = sbase + L::OFF_S + (c & 1u) * L::SCALES * 4;
                    // (VECB: a fragment's four rows side by side)
                    const uint32_t to = at + (VECB ? l / 32 * 32 + l % 8 * 4 + l % 32 / 8 : l) * 4;
                    for (int j = 0; j < L::CH && kb + j < n; ++j) {
                        ptx::cp_async_4(to + j * kBlk * 4, src.a0, 4);
                        ptx::cp_async_4(to + j * kBlk * 4 + 256, src.a1, 4);
                        src.a0 += p.M;
                        src.a1 += p.M;
                        if constexpr (VECB) {
                            ptx::cp_async_16(at + (L::CH * kBlk + j * 2 * kBlk + 4 * l) * 4, src.b, 16);
                            src.b += p.N;
                        }
                    }
                    if constexpr (!VECB) {
                        if (l < 2 * L::CH && kb + (l >> 1) < n) ptx::cp_async_4(at + (L::CH * kBlk + l) * 4, src.b, 4);
                        src.b += L::CH * p.sb_k;
                    }
                    ptx::cp_async_arrive(bar_sfull(c & 1u));
                }
            }
        }
    } else {
        // ===== promotion and epilogue: this CTA's 128 rows =====
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsProm));
        const int q = warp & 3, half = (warp - kProm0) >> 2;
        // tensor-memory column of this warp's chunk c: 64 columns of the tile's first
        // block of B (gated: of gate) and the same 64 of its second (of up)
        const uint32_t lane_base = ((uint32_t)(q * 32) << 16) + half * 64;
        // scale vectors: the chunk is 16 rows of 64 columns, in fragments of 8 columns of which
        // a lane holds two of two rows, so that it reads a quarter of the columns' scales (a
        // whole row a lane, shared memory took 1024 cycles a K block to hand them out)
        auto chunk = [&](uint32_t i, int c) {
            const uint32_t at = lane_base + (i & 1u) * 2 * kBlk + (c >> 1) * kBlk;
            return VECB ? at + ((c & 1) << 20) : at + (c & 1) * 32;
        };
        auto load = [&](uint32_t i, int c, uint32_t(&r)[32]) {
            if constexpr (VECB)
                ptx::tmem_ld_16x256b(chunk(i, c), r);
            else
                ptx::tmem_ld_32x32b_x32(chunk(i, c), r);
        };
        const uint32_t free0 = ptx::map_shared(bar_pempty(0), 0), free1 = ptx::map_shared(bar_pempty(1), 0);
        const int row_in = (int)rank * kBlk + q * 32 + lane;
        uint32_t g = 0, lt = 0;
        uint32_t chunks = 0;  // of scales, over all items
        Item it;
        for (int32_t i = 0; run && item<SHARE>(p, pair, i, it); ++i) {
            // VECB: pairs of columns, in packed arithmetic (issue slots, not the pipe, ran short)
            float acc[VECB ? 1 : 4][32];
            uint64_t acc2[VECB ? 4 : 1][16];
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    if constexpr (VECB)
                        acc2[c][i / 2] = 0ull;
                    else
                        acc[c][i] = 0.0f;
                }
            uint32_t r0[32], r1[32];
            bool ok = true;
            const int32_t n = SHARE ? it.k1 - it.k0 : p.num_kb;
            for (int32_t kb = 0; kb < n; ++kb, ++g) {
                const uint32_t buf = g & 1u;
                const int32_t at_k = kb % L::CH;
                if (at_k == 0 && !b128_wait_all(bar_sfull(chunks & 1u), (chunks >> 1) & 1u, abort_flag, p, 3 * 256 + chunks % 2)) {
                    ok = false;
                    break;
                }
                const float *sc = reinterpret_cast<const float *>(smem + L::OFF_S) + (chunks & 1u) * L::SCALES;
                const float sa = VECB ? 0.0f : sc[at_k * kBlk + q * 32 + lane];
                float2 sb{};
                if constexpr (!VECB) sb = *reinterpret_cast<const float2 *>(sc + L::CH * kBlk + at_k * 2);
                // VECB: the lane's rows' and its columns' scales, the latter of one block of 64 at a
                // time, read while tensor memory is (before it, they lengthened the time that the buffer is
                // kept: 271 us at 4096 x 14336 x 4096 in place of 259)
                float2 ra[2];
                uint64_t cb[8];
                auto columns = [&](int block) {
                    const uint64_t *col = reinterpret_cast<const uint64_t *>(sc + L::CH * kBlk + at_k * 2 * kBlk + block * kBlk +
                                                                             half * 64);
#pragma unroll
                    for (int j = 0; j < 8; ++j) cb[j] = col[4 * j + (lane & 3)];
                };
                auto add = [&](int c, const uint32_t(&r)[32]) {
                    if constexpr (VECB) {
                        // (rows' scales first: the product with them does not wait for the columns'; 277 ->
                        // 271 us at 4096 x 14336 x 4096)
                        const uint64_t a0 = b128_pair(ra[c & 1].x, ra[c & 1].x), a1 = b128_pair(ra[c & 1].y, ra[c & 1].y);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            b128_fma2(acc2[c][2 * j], b128_mul2(b128_pair(r[4 * j], r[4 * j + 1]), a0), cb[j]);
                            b128_fma2(acc2[c][2 * j + 1], b128_mul2(b128_pair(r[4 * j + 2], r[4 * j + 3]), a1), cb[j]);
                        }
                    } else {
                        const float f = __fmul_rn(sa, c >= 2 ? sb.y : sb.x);
#pragma unroll
                        for (int i = 0; i < 32; ++i) acc[c][i] = __fmaf_rn(__uint_as_float(r[i]), f, acc[c][i]);
                    }
                };
                // From here to the arrival the buffer is kept from the MMAs of the K block after
                // next: two chunks are loaded at a time (64 registers), the next two as soon as
                // theirs are free, and everything else comes before or behind.
                if (!b128_wait_all(bar_pfull(buf), (g >> 1) & 1u, abort_flag, p, 3 * 256 + 64 + buf)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                load(g, 0, r0);
                load(g, 1, r1);
                if constexpr (VECB) {
                    const float4 r = reinterpret_cast<const float4 *>(sc + at_k * kBlk + q * 32)[lane >> 2];
                    ra[0] = make_float2(r.x, r.y);
                    ra[1] = make_float2(r.z, r.w);
                    columns(0);
                }
                ptx::tmem_ld_wait(r0);
                ptx::tmem_ld_wait(r1);
                add(0, r0);
                load(g, 2, r0);
                add(1, r1);
                load(g, 3, r1);
                if constexpr (VECB) columns(1);
                ptx::tmem_ld_wait(r0);
                ptx::tmem_ld_wait(r1);
                ptx::tc_fence_before();
                __syncwarp();
                ptx::mbar_arrive_cluster_relaxed(buf ? free1 : free0, lane == 0);
                add(2, r0);
                add(3, r1);
                if (at_k == L::CH - 1 || kb + 1 == n) {  // this chunk is read
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(bar_sempty(chunks & 1u));
                    ++chunks;
                }
            }
            if (!ok) break;
            int32_t pm, tn;
            raster(it.t, p.npm, p.npn, kRasterG, pm, tn);
            const int64_t row = (int64_t)pm * 2 * kBlk + row_in;
            if (SHARE && (it.publish || it.from < pair)) {
                // sums as the warp holds them, 16 bytes a lane
                auto at = [&](int32_t c) {
                    return p.part + c * (kB128PartBytes / 4) + ((int64_t)rank * kPromWarps + warp - kProm0) * 4096 + 4 * lane;
                };
                const int32_t flag = (int32_t)rank * kPromWarps + warp - kProm0;
                if (it.publish) {
                    float *dst = at(pair);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            float4 v;
                            if constexpr (VECB)
                                v = make_float4(b128_lo(acc2[c][2 * k]), b128_hi(acc2[c][2 * k]), b128_lo(acc2[c][2 * k + 1]),
                                                b128_hi(acc2[c][2 * k + 1]));
                            else
                                v = make_float4(acc[c][4 * k], acc[c][4 * k + 1], acc[c][4 * k + 2], acc[c][4 * k + 3]);
                            __stcg(reinterpret_cast<float4 *>(dst + (c * 8 + k) * 128), v);
                        }
                    __threadfence();
                    __syncwarp();
                    if (lane == 0) st_release(p.there + pair * 16 + flag, 1);
                    continue;
                }
                for (int32_t from = it.from; from < pair && ok; ++from) {
                    ok = wait_flag(p.there + from * 16 + flag, abort_flag, p);
                    if (!ok) break;
                    const float *src = at(from);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float4 v = __ldcg(reinterpret_cast<const float4 *>(src + (c * 8 + k) * 128));
                            if constexpr (VECB) {
                                acc2[c][2 * k] = b128_add2(acc2[c][2 * k], b128_pair(v.x, v.y));
                                acc2[c][2 * k + 1] = b128_add2(acc2[c][2 * k + 1], b128_pair(v.z, v.w));
                            } else {
                                acc[c][4 * k] += v.x;
                                acc[c][4 * k + 1] += v.y;
                                acc[c][4 * k + 2] += v.z;
                                acc[c][4 * k + 3] += v.w;
                            }
                        }
                }
                if (!ok) break;
            }

            // (lane and base read anew: what follows from them is not worked out before the K blocks
            // and kept; the gated kernel had 3% from it)
            uint32_t lane_again, base_again;
            asm volatile("mov.u32 %0, %%laneid;" : "=r"(lane_again));
            asm volatile("mov.u32 %0, %1;" : "=r"(base_again) : "r"(sbase));
            Output to(base_again + L::OFF_C + (warp - kProm0) * 2 * kUnit, (int)lane_again);
            const int64_t y = row - lane;  // the warp's first row (whole units past the matrix are left out)
            if constexpr (VECB) {
                // pairs of columns of 16 rows' halves: units of 64 bytes a row
                constexpr int COLS = OUT == kB128Bf16 ? 32 : 16, F = COLS / 8;  // columns, fragments of a unit
                const int64_t n0 = (int64_t)tn * 2 * kBlk + half * 64;
#pragma unroll
                for (int u = 0; u < 128 / COLS; ++u) {
                    const int block = u * COLS / 64, f0 = u * COLS % 64 / 8;
                    const int64_t x = n0 + block * kBlk + f0 * 8;
                    const uint32_t at = to.begin();
#pragma unroll
                    for (int i = 0; i < 4 * F; ++i) {
                        const int c = 2 * block + i / (2 * F), k = 2 * (f0 + i / 2 % F) + (i & 1);
                        const int r = (c & 1) * 16 + (i & 1) * 8 + (lane >> 2), f = i / 2 % F;
                        const float lo = b128_lo(acc2[c][k]), hi = b128_hi(acc2[c][k]);
                        if constexpr (OUT == kB128Bf16)
                            ptx::st_shared(Output::piece(at, r, f) + (lane & 3) * 4, pack_bf16(lo, hi));
                        else
                            ptx::st_shared_v2(Output::piece(at, r, 2 * f + ((lane >> 1) & 1)) + (lane & 1) * 8,
                                              __float_as_uint(lo), __float_as_uint(hi));
                    }
                    to.end<OUT == kB128Add>(m.C, at, x, y, y < p.M && x < p.N);
                }
            } else if constexpr (OUT < kB128Gated) {
                const int64_t n0 = (int64_t)tn * 2 * kBlk + half * 64;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int64_t x = n0 + (c >> 1) * kBlk + (c & 1) * 32;
                    uint32_t w[16];
                    if constexpr (OUT == kB128Bf16) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) w[i] = pack_bf16(acc[c][2 * i], acc[c][2 * i + 1]);
                        to.row<false>(m.C, w, x, y, y < p.M && x < p.N);
                    } else {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(acc[c][16 * h + i]);
                            to.row<OUT == kB128Add>(m.C, w, x + 16 * h, y, y < p.M && x + 16 * h < p.N);
                        }
                    }
                }
            } else {
                // h in the gate's place; a row's maxima from the two warps that share it
                float gv[64], uv[64], h[64];
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        gv[c * 32 + i] = acc[c][i];
                        uv[c * 32 + i] = acc[c + 2][i];
                    }
                const bool keep = p.gu != nullptr;
                float4 top = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int i = 0; i < 64; i += 2) {
                    const uint64_t y = b128_gate2<OUT - kB128Gated>(b128_pair(gv[i], gv[i + 1]));
                    const uint64_t v = b128_mul2(y, b128_pair(uv[i], uv[i + 1]));
                    h[i] = b128_lo(v), h[i + 1] = b128_hi(v);
                }
                top.x = amax64(h);
                top.y = amax64(gv);
                top.z = amax64(uv);
                // One barrier that both warps arrive on: its next phase ends with the slower warp's
                // next arrival, so neither gets a phase ahead of the other's wait. (With a barrier
                // of each warp's own, one that had at most two K blocks a tile, which both product
                // buffers hold, could pass two phases, and the other's parity never came.)
                // [tile parity][half][row]: a slot is written again two tiles later, after
                // its reader's next arrival
                const uint32_t par = lt++ & 1u;
                float4 *x = reinterpret_cast<float4 *>(smem + L::OFF_X) + par * 2 * kBlk;
                x[half * kBlk + q * 32 + lane] = top;
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar_max(q));
                if (!wait_bar_warp(bar_max(q), par, abort_flag, p, 3 * 256 + 96 + q)) break;
                const float4 o = x[(half ^ 1) * kBlk + q * 32 + lane];
                const int64_t F = p.N, f = (int64_t)tn * kBlk + half * 64;
                const bool in = row < p.M, any = y < p.M;
                uint32_t w[16];
                const float sh = b128_scale<FP8G_E4M3>(fmaxf(top.x, o.x));
                codes64(w, h, __frcp_rn(sh));
                to.row<false>(m.C, w, f, y, any);
                if (half == 0 && in) p.sh[tn * p.M + row] = sh;
                if (keep) {
                    const float sg = b128_scale<FP8G_E4M3>(fmaxf(top.y, o.y));
                    const float su = b128_scale<FP8G_E4M3>(fmaxf(top.z, o.z));
                    codes64(w, gv, __frcp_rn(sg));
                    to.row<false>(m.gu, w, f, y, any);
                    codes64(w, uv, __frcp_rn(su));
                    to.row<false>(m.gu, w, F + f, y, any);
                    if (half == 0 && in) {
                        p.sgu[tn * p.M + row] = sg;
                        p.sgu[(p.n_blocks + tn) * p.M + row] = su;
                    }
                }
            }
        }
        if (lane == 0) ptx::bulk_wait_all();
    }

roles_done:
    __syncwarp();
    __syncthreads();
    if (*abort_flag) {
        // drain the MMAs that are in flight, give copies a bounded time to land
        if (leader && warp == 1 && lane == 0) {
            ptx::tc_commit_pair(bar_drain);
            const uint64_t t0 = ptx::globaltimer();
            while (!ptx::mbar_try_wait(bar_drain, 0) && ptx::globaltimer() - t0 < p.timeout_ns) {
            }
        }
        const uint64_t t0 = ptx::globaltimer();
        while (ptx::globaltimer() - t0 < 200000ull) {
        }
        __syncthreads();
    }
    // neither CTA leaves while the other may still arrive on its barriers
    ptx::cluster_sync();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem_base, 512);
    }
}

template <bool VECB, int OUT, bool SHARE>
cudaError_t launch_pair(const B128Maps &m, const B128Params &p, int grid, cudaStream_t stream) {
    auto kern = b128_pair_kernel<VECB, OUT, SHARE>;
    static unsigned long long done = 0ull;
    if (done == 0ull) {
        // setmaxnreg.inc takes from what the block was launched with
        cudaFuncAttributes fa;
        const cudaError_t e = cudaFuncGetAttributes(&fa, kern);
        if (e != cudaSuccess) return e;
        if (fa.numRegs < kRegsLaunch) return cudaErrorInvalidConfiguration;
    }
    const cudaError_t e = b128_allow_smem(reinterpret_cast<const void *>(kern), Lay<VECB>::BYTES, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = Lay<VECB>::BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, m, p);
}

template <bool VECB, bool SHARE>
cudaError_t launch_product(const B128Maps &m, const B128Params &p, int out, int grid, cudaStream_t stream) {
    if (out == kB128Bf16) return launch_pair<VECB, kB128Bf16, SHARE>(m, p, grid, stream);
    if (out == kB128F32) return launch_pair<VECB, kB128F32, SHARE>(m, p, grid, stream);
    return launch_pair<VECB, kB128Add, SHARE>(m, p, grid, stream);
}

}  // namespace

}  // namespace fp8g
