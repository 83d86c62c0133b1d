// Streaming GEMM for few tokens: D[f, t] = sum_k (s W)[f, k] (s X)[t, k] with
// block-scaled weights W that are read once, tokens X in E4M3 with 1x32
// power-of-two scales.
//
// The weights are the MMA's 128-row operand and the tokens its columns
// (tcgen05.mma kind::mxf8f6f4, M = 128, N = the group's tokens rounded up to
// 16): with few tokens a tile costs what its weights cost to load, and no CUDA
// core touches them.  A work unit is one 128-wide K step of a pair of 128-row
// weight tiles (32 KB: the gate and the up rows of the same features, or two
// neighbouring tiles).  The units of all groups, tiles and K steps are one
// line that the CTAs share out evenly, one CTA per SM, so every SM streams
// the same number of bytes whatever the shape: a CTA's span may begin and end
// inside a tile.  A tile that several CTAs share is joined by the last of
// them to finish: each stores its fp32 partial tile and adds its units to the
// tile's counter, and whoever completes the count sums the partials in unit
// order (the result does not depend on who that is).  No CTA waits for another.
//
// Roles: warp 0 TMA producer (a ring of stages: two weight tiles, the tokens'
// K slice, the three packed scale chunks), warp 2 copies a stage's scales to
// tensor memory, warp 1 issues its MMAs, warps 4-11 epilogue.
//
// Low-rank steps (kStreamOut): after the FP8 steps a tile takes, per adapter
// among the group's tokens, 64-wide bf16 steps (kind::f16) of the adapter's B
// rows against V = alpha A x of those tokens (zero for the others), into the
// same fp32 accumulator.  V is held as two bf16 halves (V - bf16(V) rounded
// again: 16 significant bits), each an MMA of its own.
#include <cuda_bf16.h>

#include "kernel_common.cuh"
#include "quant_math.cuh"
#include "stream.h"

namespace fp8g {

namespace {

constexpr int kSThreads = 384;
constexpr int kSEpiWarp0 = 4;
constexpr int kSEpiWarps = 8;
constexpr int kWTile = 128 * 128;  // bytes of a weight tile in shared memory
constexpr int kMaxStages = 16;
constexpr int kJoin = 4;           // partial tiles read at a time
constexpr int kSfSlot = 16;        // tensor-memory columns of a stage's scales
constexpr int kSmemMax = 232448;

constexpr int kLoraGroups = kStreamMaxLoraRows / kStreamMaxTokens;

// Shared memory after the ring: barriers, table of groups.
struct StreamTail {
    uint64_t full[kMaxStages], empty[kMaxStages], sfr[kMaxStages], accf[2], acce[2], drain, drain_sf;
    uint32_t tmem;
    int abort_flag;
    int last;
    int units;
    StreamGroup g[kStreamMaxGroups + 1];
    union {
        int32_t cnt[FP8G_MAX_ROUTED_EXPERTS];  // rows per expert
        struct {
            uint32_t bits[kLoraGroups][kMaxAdapters / 32];      // adapters of a group's rows
            int32_t n[kLoraGroups];                             // slots: how many of them
            int16_t adapter[kLoraGroups][kStreamMaxTokens];     // in rising order
        } lora;
    };
};

static_assert(kSmemMax - 1024 - (int)sizeof(StreamTail) >= 6 * (2 * kWTile + 16 * 128 + 2048),
              "six stages with 16 token columns");

// A CTA's part of one tile.
struct StreamTile {
    int32_t g, mt, row0, n, n16;
    int32_t mat0, mat1, w0, w1;  // matrix and first row of the two weight tiles
    bool has1;                   // the second one exists
    int32_t k0, k1, upt;         // units [k0, k1) of the tile's upt
};

// Walks the tiles of units [u, end).
struct StreamWalk {
    int32_t g, u, end;
};

template <int EPI>
__device__ __forceinline__ bool stream_next(const StreamParams &p, const StreamTail &t, StreamWalk &w,
                                            StreamTile &o) {
    if (w.u >= w.end) return false;
    while (t.g[w.g + 1].unit0 <= w.u) ++w.g;
    const StreamGroup gr = t.g[w.g];
    o.g = w.g;
    o.upt = p.ks + (EPI == kStreamOut ? t.lora.n[w.g] * p.kr : 0);
    const int32_t rel = w.u - gr.unit0;
    o.mt = rel / o.upt;
    o.k0 = rel - o.mt * o.upt;
    o.k1 = min(o.upt, o.k0 + (w.end - w.u));
    o.row0 = gr.row0;
    o.n = gr.n;
    o.n16 = (gr.n + 15) & ~15;
    if constexpr (EPI == kStreamGated) {
        o.mat0 = 2 * gr.mat;
        o.mat1 = o.mat0 + 1;
        o.w0 = o.w1 = o.mt * 128;
        o.has1 = true;
    } else {
        o.mat0 = o.mat1 = gr.mat;
        o.w0 = o.mt * 128 * p.sub;
        o.w1 = o.w0 + 128;
        o.has1 = p.sub == 2 && o.w1 < p.rows;
    }
    w.u += o.k1 - o.k0;
    return true;
}

// First unit of CTA c of G sharing U units.
__device__ __forceinline__ int32_t span_begin(int64_t U, int G, int c) { return (int32_t)(U * c / G); }
// CTA that owns unit u: the largest c with U c / G <= u (rounded down).
__device__ __forceinline__ int span_owner(int64_t U, int G, int64_t u) {
    return (int)(((u + 1) * G - 1) / U);
}

// All epilogue warps: the AND of their flags (also a barrier among them; every
// one of them takes part in every call, so none is left waiting).
__device__ __forceinline__ bool epi_all(bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "barrier.cta.red.and.pred p, 1, %2, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(ok ? 1u : 0u), "n"(kSEpiWarps * 32)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ float gate_act(float g, int gate) {
    if (gate == FP8G_GATE_SILU) return g / (1.0f + expf(-g));
    if (gate == FP8G_GATE_GELU) return 0.5f * g * (1.0f + erff(g * 0.70710678118654752f));
    return g < 0.0f ? 0.0f : g;
}

// The groups and the number of units.  Call with all threads.
template <int EPI>
__device__ __forceinline__ void stream_tables(const StreamParams &p, StreamTail &t) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if constexpr (EPI == kStreamOut) {
        const int ng = (p.n_idx + p.nb - 1) / p.nb;
        for (int i = threadIdx.x; i < kLoraGroups * kMaxAdapters / 32; i += kSThreads)
            t.lora.bits[0][i] = 0;
        __syncthreads();
        if (p.kr > 0)
            for (int i = threadIdx.x; i < p.n_idx; i += kSThreads) {
                const int l = __ldcg(p.idx + i);
                if (l >= 0 && l < p.n_mat) atomicOr(&t.lora.bits[i / p.nb][l >> 5], 1u << (l & 31));
            }
        __syncthreads();
        if (warp < ng) {  // lane i: adapters 32 i .. 32 i + 31 (at most 12 groups)
            const uint32_t w = t.lora.bits[warp][lane];
            int at = __popc(w), sum = at;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += v;
            }
            at = sum - at;
            for (uint32_t m = w; m != 0; m &= m - 1)
                t.lora.adapter[warp][at++] = (int16_t)(32 * lane + __ffs((int)m) - 1);
            if (lane == 31) t.lora.n[warp] = sum;
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            int u = 0;
            for (int g = 0; g < ng; ++g) {
                t.g[g] = StreamGroup{0, g * p.nb, min(p.nb, p.n_idx - g * p.nb), u};
                u += p.mt * (p.ks + t.lora.n[g] * p.kr);
            }
            t.units = u;
            t.g[ng].unit0 = 0x7FFFFFFF;
        }
    } else {
        for (int e = threadIdx.x; e < p.n_mat; e += kSThreads) t.cnt[e] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < p.n_idx; i += kSThreads) {
            const int e = __ldcg(p.idx + i);
            if (e >= 0 && e < p.n_mat) atomicAdd(&t.cnt[e], 1);
        }
        __syncthreads();
        if (warp == 0) {
            const int per = p.mt * p.ks;
            int rr = 0, gg = 0;
            for (int e0 = 0; e0 < p.n_mat; e0 += 32) {
                const int e = e0 + lane;
                const int c = e < p.n_mat ? t.cnt[e] : 0, ng = (c + p.nb - 1) / p.nb;
                int s = c, sg = ng;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, s, o), vg = __shfl_up_sync(0xffffffffu, sg, o);
                    if (lane >= o) {
                        s += v;
                        sg += vg;
                    }
                }
                for (int i = 0; i < ng; ++i) {
                    const int g = gg + sg - ng + i;
                    t.g[g] = StreamGroup{e, rr + s - c + i * p.nb, min(p.nb, c - i * p.nb), g * per};
                }
                rr += __shfl_sync(0xffffffffu, s, 31);
                gg += __shfl_sync(0xffffffffu, sg, 31);
            }
            if (lane == 0) {
                t.units = gg * per;
                t.g[gg].unit0 = 0x7FFFFFFF;
            }
        }
    }
}

template <int EPI>
__global__ void __launch_bounds__(kSThreads, 1)
    stream_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                  const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmV,
                  const __grid_constant__ StreamParams p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = ptx::smem_addr(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (raw_base & 1023u)) & 1023u);
    const uint32_t sbase = ptx::smem_addr(smem);
    StreamTail &t = *reinterpret_cast<StreamTail *>(smem + p.stages * p.stage_bytes);
    volatile int *abort_flag = &t.abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t off_x = 2 * kWTile, off_sf = 2 * kWTile + p.x_bytes;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            ptx::mbar_init(ptx::smem_addr(&t.full[s]), 1);
            ptx::mbar_init(ptx::smem_addr(&t.empty[s]), 1);
            ptx::mbar_init(ptx::smem_addr(&t.sfr[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(ptx::smem_addr(&t.accf[a]), 1);
            ptx::mbar_init(ptx::smem_addr(&t.acce[a]), kSEpiWarps);
        }
        ptx::mbar_init(ptx::smem_addr(&t.drain), 1);
        ptx::mbar_init(ptx::smem_addr(&t.drain_sf), 1);
        t.abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        ptx::prefetch_tmap(&tmW);
        ptx::prefetch_tmap(&tmX);
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_addr(&t.tmem), 512);
        ptx::tmem_relinquish();
    }
    // Launched programmatically: the previous kernel, which writes the tokens'
    // codes, may still run.  What was complete before that kernel began (it
    // lets this one start only after its own wait), the weights and the
    // indices, is read right away: the first stages' weights are on their way
    // while the tokens are prepared.
    stream_tables<EPI>(p, t);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = t.tmem;
    const int64_t U = t.units;
    const int G = max(1, (int)min((int64_t)gridDim.x, U / kStreamMinUnits));
    const int cta = blockIdx.x;
    const int32_t u0 = cta < G ? span_begin(U, G, cta) : 0;
    const int32_t u1 = cta < G ? span_begin(U, G, cta + 1) : 0;
    StreamWalk walk{0, u0, u1};
    StreamTile ti;
    const int acc_cols = 2 * p.nb;
    const uint32_t sf_tmem0 = tmem + p.nacc * acc_cols;

    if (warp == 0) {
        // ===== TMA producer =====
        if (lane == 0) {
            const uint32_t w_tx = kWTile - kWTile / 8 * p.gap8;
            const bool two_v = p.v_rows > p.nb;
            // the two halves of a step's loads: weights and their scales (or an
            // adapter's rows), tokens and theirs (or V)
            auto weights = [&](const StreamTile &o, int k, int stage) {
                const uint32_t fb = ptx::smem_addr(&t.full[stage]);
                const uint32_t s0 = sbase + stage * p.stage_bytes;
                const uint32_t nw = o.has1 ? 2 : 1;
                if (EPI != kStreamOut || k < p.ks) {
                    ptx::mbar_arrive_expect_tx(fb, nw * (w_tx + 512u) + o.n16 * 128u + 512u);
                    const int64_t c0 = ((int64_t)o.mat0 * p.ks + k) * p.n_rt + o.w0 / 128;
                    ptx::tma_load_3d(s0, &tmW, fb, k * kBK, o.w0, o.mat0);
                    ptx::bulk_load(s0 + off_sf, p.sfw + c0 * 512, 512, fb);
                    if (o.has1) {
                        const int64_t c1 = ((int64_t)o.mat1 * p.ks + k) * p.n_rt + o.w1 / 128;
                        ptx::tma_load_3d(s0 + kWTile, &tmW, fb, k * kBK, o.w1, o.mat1);
                        ptx::bulk_load(s0 + off_sf + 512, p.sfw + c1 * 512, 512, fb);
                    }
                } else {
                    const int ls = k - p.ks, sl = ls / p.kr, c = (ls - sl * p.kr) * 64;
                    const int l = t.lora.adapter[o.g][sl];
                    ptx::mbar_arrive_expect_tx(fb, nw * kWTile + (two_v ? 2 : 1) * o.n16 * 128u);
                    ptx::tma_load_3d(s0, &tmB, fb, c, o.w0, l);
                    if (o.has1) ptx::tma_load_3d(s0 + kWTile, &tmB, fb, c, o.w1, l);
                }
            };
            auto tokens = [&](const StreamTile &o, int k, int stage) {
                const uint32_t fb = ptx::smem_addr(&t.full[stage]);
                const uint32_t s0 = sbase + stage * p.stage_bytes;
                if (EPI != kStreamOut || k < p.ks) {
                    ptx::bulk_load(s0 + off_sf + 1024, p.sfx + ((int64_t)o.g * p.ks + k) * 512, 512, fb);
                    for (int i = 0; i < o.n16; i += 16)
                        ptx::tma_load_2d(s0 + off_x + i * 128, &tmX, fb, k * kBK, o.row0 + i);
                } else {
                    const int ls = k - p.ks, sl = ls / p.kr, c = (ls - sl * p.kr) * 64;
                    const int v0 = (o.g * p.slot_cap + sl) * p.v_rows;
                    for (int i = 0; i < o.n16; i += 16) {
                        ptx::tma_load_2d(s0 + off_x + i * 128, &tmV, fb, c, v0 + i);
                        if (two_v)
                            ptx::tma_load_2d(s0 + off_x + (p.nb + i) * 128, &tmV, fb, c, v0 + p.nb + i);
                    }
                }
            };
            // the ring's first fill: weights before the wait, tokens after it
            int ahead = 0;
            {
                StreamWalk w2 = walk;
                while (ahead < p.stages && stream_next<EPI>(p, t, w2, ti))
                    for (int k = ti.k0; k < ti.k1 && ahead < p.stages; ++k) weights(ti, k, ahead++);
            }
            ptx::grid_dep_wait();
            ptx::grid_dep_launch();
            int stage = 0, done = 0;
            uint32_t phase = 0;
            while (stream_next<EPI>(p, t, walk, ti)) {
                for (int k = ti.k0; k < ti.k1; ++k, ++done) {
                    if (done >= ahead) {
                        if (!wait_bar(ptx::smem_addr(&t.empty[stage]), phase ^ 1u, abort_flag, p, stage))
                            goto roles_done;
                        weights(ti, k, stage);
                    }
                    tokens(ti, k, stage);
                    if (++stage == p.stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
        }
    } else if (warp == 1) {
        // ===== MMAs =====
        if (lane == 0) {
            int stage = 0, lt = 0;
            uint32_t phase = 0;
            for (; stream_next<EPI>(p, t, walk, ti); ++lt) {
                const int acc = p.nacc == 2 ? (lt & 1) : 0;
                const uint32_t par = (uint32_t)((p.nacc == 2 ? lt >> 1 : lt) & 1);
                if (!wait_bar(ptx::smem_addr(&t.acce[acc]), par ^ 1u, abort_flag, p, 256 + 64 + acc))
                    goto roles_done;
                ptx::tc_fence_after();
                const uint32_t d0 = tmem + acc * acc_cols, d1 = d0 + p.nb;
                const uint32_t id8 = ptx::idesc_mxf8(128, 0, 0) | ((uint32_t)(ti.n16 >> 3) << 17) | p.w_fmt;
                const uint32_t id16 = ptx::idesc_bf16(128, 0) | ((uint32_t)(ti.n16 >> 3) << 17);
                for (int k = ti.k0; k < ti.k1; ++k) {
                    if (!wait_bar(ptx::smem_addr(&t.sfr[stage]), phase, abort_flag, p, 256 + stage))
                        goto roles_done;
                    ptx::tc_fence_after();
                    const uint32_t s0 = sbase + stage * p.stage_bytes;
                    const uint32_t x0 = s0 + off_x;
                    if (EPI != kStreamOut || k < p.ks) {
                        const uint32_t sf = sf_tmem0 + stage * kSfSlot;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t id = id8 | ((uint32_t)j << 4) | ((uint32_t)j << 29);
                            const uint32_t on = (k != ti.k0 || j != 0) ? 1u : 0u;
                            const uint64_t dx = ptx::desc_kmajor_sw128(x0 + 32 * j);
                            ptx::mma_mxf8(d0, ptx::desc_kmajor_sw128(s0 + 32 * j), dx, id, sf, sf + 8, on);
                            if (ti.has1)
                                ptx::mma_mxf8(d1, ptx::desc_kmajor_sw128(s0 + kWTile + 32 * j), dx, id,
                                              sf + 4, sf + 8, on);
                        }
                    } else {
                        const int ls = k - p.ks, c = (ls - ls / p.kr * p.kr) * 64;
                        const int nk = (min(64, p.rank - c) + 15) / 16;
                        for (int j = 0; j < nk; ++j) {
                            const uint64_t dh = ptx::desc_kmajor_sw128(x0 + 32 * j);
                            // the lo half: rows of its own, or columns 32-63
                            const uint64_t dl = ptx::desc_kmajor_sw128(
                                x0 + (p.v_rows > p.nb ? p.nb * 128 : 64) + 32 * j);
                            const uint64_t w0 = ptx::desc_kmajor_sw128(s0 + 32 * j);
                            ptx::mma_bf16(d0, w0, dh, id16, (k != ti.k0 || j != 0) ? 1u : 0u);
                            ptx::mma_bf16(d0, w0, dl, id16, 1u);
                            if (ti.has1) {
                                const uint64_t w1 = ptx::desc_kmajor_sw128(s0 + kWTile + 32 * j);
                                ptx::mma_bf16(d1, w1, dh, id16, (k != ti.k0 || j != 0) ? 1u : 0u);
                                ptx::mma_bf16(d1, w1, dl, id16, 1u);
                            }
                        }
                    }
                    ptx::tc_commit(ptx::smem_addr(&t.empty[stage]));
                    if (++stage == p.stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                ptx::tc_commit(ptx::smem_addr(&t.accf[acc]));
            }
        }
    } else if (warp == 2) {
        // ===== scales to tensor memory =====
        // From a thread of their own: issued by the MMA thread each copy holds
        // up the MMAs behind it.  A stage's columns are rewritten only after
        // its next "full", when the MMAs that read them are complete.
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            while (stream_next<EPI>(p, t, walk, ti)) {
                for (int k = ti.k0; k < ti.k1; ++k) {
                    if (!wait_bar(ptx::smem_addr(&t.full[stage]), phase, abort_flag, p, 2 * 256 + stage))
                        goto roles_done;
                    ptx::tc_fence_after();
                    if (EPI != kStreamOut || k < p.ks) {
                        const uint32_t sf = sf_tmem0 + stage * kSfSlot;
                        const uint32_t cs = sbase + stage * p.stage_bytes + off_sf;
                        ptx::tc_cp_32x128b_warpx4(sf, ptx::desc_sf_chunk(cs));
                        if (ti.has1) ptx::tc_cp_32x128b_warpx4(sf + 4, ptx::desc_sf_chunk(cs + 512));
                        ptx::tc_cp_32x128b_warpx4(sf + 8, ptx::desc_sf_chunk(cs + 1024));
                    }
                    ptx::tc_commit(ptx::smem_addr(&t.sfr[stage]));
                    if (++stage == p.stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
        }
    } else if (warp >= kSEpiWarp0) {
        // ===== epilogue =====
        ptx::grid_dep_wait();  // counters, partials and outputs: after the previous kernel
        const int q = warp & 3, half = (warp - kSEpiWarp0) >> 2;
        const uint32_t tq = tmem + ((uint32_t)(q * 32) << 16);
        const int row_l = q * 32 + lane;  // weight row within a tile
        // two weight tiles: this warp takes tile `half`; gated, or one tile:
        // every other 16 columns (of both tiles, gated)
        constexpr int kSubs = EPI == kStreamGated ? 2 : 1;
        const bool by_cols = EPI == kStreamGated || p.sub == 1;
        const int c_first = by_cols ? half * 16 : 0, c_step = by_cols ? 32 : 16;
        const int my_sub = by_cols ? 0 : half;
        int lt = 0;
        for (; stream_next<EPI>(p, t, walk, ti); ++lt) {
            const int acc = p.nacc == 2 ? (lt & 1) : 0;
            const uint32_t par = (uint32_t)((p.nacc == 2 ? lt >> 1 : lt) & 1);
            const bool ok = wait_bar_warp(ptx::smem_addr(&t.accf[acc]), par, abort_flag, p, 3 * 256 + acc, 64);
            if (!epi_all(ok)) break;
            ptx::tc_fence_after();
            const bool whole = ti.k0 == 0 && ti.k1 == ti.upt;
            const bool live = my_sub == 0 || ti.has1;  // this warp has a weight tile
            const uint32_t ta = tq + acc * acc_cols;
            bool finish = whole;
            int c_lo = 0, c_hi = 0;  // CTAs that share the tile
            if (!whole) {
                const int64_t tu = (int64_t)t.g[ti.g].unit0 + (int64_t)ti.mt * ti.upt;
                c_lo = span_owner(U, G, tu);
                c_hi = span_owner(U, G, tu + ti.upt - 1);
                float *part = p.part + (int64_t)(2 * cta + (u0 > tu ? 0 : 1)) * 2 * p.nb * 128;
                if (live)
                    for (int c = c_first; c < ti.n; c += c_step) {
#pragma unroll
                        for (int s = 0; s < kSubs; ++s) {
                            const int sub = EPI == kStreamGated ? s : my_sub;
                            uint32_t r[16];
                            ptx::tmem_ld_32x32b_x16(ta + sub * p.nb + c, r);
                            ptx::tmem_ld_wait();
                            float *dst = part + ((int64_t)sub * p.nb + c) * 128 + row_l;
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (c + i < ti.n) __stcg(dst + i * 128, __uint_as_float(r[i]));
                        }
                    }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&t.acce[acc]));
                __threadfence();
                (void)epi_all(true);  // every partial of this CTA is stored
                if (threadIdx.x == kSEpiWarp0 * 32) {
                    const int mine = ti.k1 - ti.k0;
                    const int old = atomicAdd(p.tile_cnt + ti.g * p.mt + ti.mt, mine);
                    t.last = old + mine == ti.upt;
                    __threadfence();
                }
                (void)epi_all(true);
                finish = t.last != 0;
            }
            if (finish && live) {
                for (int c = c_first; c < ti.n; c += c_step) {
                    float v[kSubs][16];
#pragma unroll
                    for (int s = 0; s < kSubs; ++s) {
                        const int sub = EPI == kStreamGated ? s : my_sub;
                        if (whole) {
                            uint32_t r[16];
                            ptx::tmem_ld_32x32b_x16(ta + sub * p.nb + c, r);
                            ptx::tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 16; ++i) v[s][i] = __uint_as_float(r[i]);
                        } else {
                            const int64_t tu = (int64_t)t.g[ti.g].unit0 + (int64_t)ti.mt * ti.upt;
#pragma unroll
                            for (int i = 0; i < 16; ++i) v[s][i] = 0.0f;
                            // in unit order; several CTAs' loads in flight at a time
                            for (int o = c_lo; o <= c_hi; o += kJoin) {
                                float x[kJoin][16];
#pragma unroll
                                for (int j = 0; j < kJoin; ++j) {
                                    const int side = span_begin(U, G, o + j) > tu ? 0 : 1;
                                    const float *src = p.part + (int64_t)(2 * (o + j) + side) * 2 * p.nb * 128 +
                                                       ((int64_t)sub * p.nb + c) * 128 + row_l;
#pragma unroll
                                    for (int i = 0; i < 16; ++i)
                                        x[j][i] = o + j <= c_hi && c + i < ti.n ? __ldcg(src + i * 128) : 0.0f;
                                }
#pragma unroll
                                for (int j = 0; j < kJoin; ++j)
                                    if (o + j <= c_hi)
#pragma unroll
                                        for (int i = 0; i < 16; ++i) v[s][i] += x[j][i];
                            }
                        }
                    }
                    const int f = (my_sub ? ti.w1 : ti.w0) + row_l;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int col = c + i;
                        if (col < ti.n) {  // warp-uniform
                            if constexpr (EPI == kStreamGated) {
                                // this warp's 32 features are one 1x32 block (rows is a multiple of 32)
                                uint32_t code = 127u;  // blocks past the matrix: scale 1
                                if (f < p.rows) {
                                    const float h = __fmul_rn(gate_act(v[0][i], p.gate), v[kSubs - 1][i]);
                                    const uint32_t mag = isnan(h) ? 0u : __float_as_uint(fabsf(h));
                                    const float s = pow2_scale<0>(
                                        __uint_as_float(__reduce_max_sync(0xffffffffu, mag)));
                                    p.hq[(int64_t)(ti.row0 + col) * p.rows + f] =
                                        (uint8_t)fp8x2<0>(__fmul_rn(h, __frcp_rn(s)), 0.0f);
                                    code = __float_as_uint(s) >> 23;
                                }
                                if (lane == 0)
                                    p.hsf[((int64_t)ti.g * p.mt + ti.mt) * 512 + 16 * (col & 31) +
                                          4 * (col >> 5) + q] = (uint8_t)code;
                            } else if (f < p.rows) {
                                const int64_t at = (int64_t)(ti.row0 + col) * p.rows + f;
                                if constexpr (EPI == kStreamRows) {
                                    p.y[at] = v[0][i];
                                } else {
                                    const float o =
                                        p.bias != nullptr ? __fadd_rn(v[0][i], __ldg(p.bias + f)) : v[0][i];
                                    if (p.out_f32)
                                        static_cast<float *>(p.c)[at] = o;
                                    else
                                        static_cast<__nv_bfloat16 *>(p.c)[at] = __float2bfloat16_rn(o);
                                }
                            }
                        }
                    }
                }
            }
            if (whole) {
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&t.acce[acc]));
            }
        }
    }

roles_done:
    __syncwarp();
    __syncthreads();
    if (*abort_flag) {
        // wait (bounded) for this CTA's MMAs, then give copies in flight a
        // bounded time before shared memory is released
        if ((warp == 1 || warp == 2) && lane == 0) {
            const uint32_t db = ptx::smem_addr(warp == 1 ? &t.drain : &t.drain_sf);
            ptx::tc_commit(db);
            const uint64_t t0 = ptx::globaltimer();
            while (!ptx::mbar_try_wait(db, 0) &&
                   ptx::globaltimer() - t0 < p.timeout_ns) {
            }
        }
        const uint64_t t0 = ptx::globaltimer();
        while (ptx::globaltimer() - t0 < 200000ull) {
        }
        __syncthreads();
    }
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

template <int EPI>
cudaError_t launch_epi(const CUtensorMap &w, const CUtensorMap &x, const CUtensorMap &lb,
                       const CUtensorMap &v, const StreamParams &p, int grid, cudaStream_t s) {
    auto kern = stream_kernel<EPI>;
    static unsigned long long attr_done = 0ull;  // per device; races benignly
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if ((attr_done & bit) == 0ull) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
        if (e != cudaSuccess) return e;
        attr_done |= bit;
    }
    const size_t smem = (size_t)p.stages * p.stage_bytes + sizeof(StreamTail) + 1024;
    return launch_programmatic_smem(kern, dim3((unsigned)grid), dim3(kSThreads), smem, s, w, x, lb, v, p);
}

}  // namespace

void stream_sizes(StreamParams &p, int nb, int v_halves) {
    p.nb = nb;
    p.sub = 2;
    // two accumulators of two tiles each beside the scales, where they fit
    p.nacc = nb <= 64 ? 2 : 1;
    p.x_bytes = nb * 128 * v_halves;
    p.stage_bytes = 2 * kWTile + p.x_bytes + 2048;  // 1536 bytes of scales; 1024-byte multiples
    const int room = kSmemMax - 1024 - (int)sizeof(StreamTail);
    p.stages = room / p.stage_bytes;
    const int cols = (512 - p.nacc * 2 * nb) / kSfSlot;
    if (p.stages > cols) p.stages = cols;
    if (p.stages > kMaxStages) p.stages = kMaxStages;
}

size_t stream_part_bytes(const StreamParams &p, int grid) {
    return (size_t)grid * 2 * 2 * p.nb * 128 * sizeof(float);
}

cudaError_t launch_stream(int epi, const CUtensorMap &w, const CUtensorMap &x, const CUtensorMap &lb,
                          const CUtensorMap &v, const StreamParams &p, int grid, cudaStream_t s) {
    if (epi == kStreamGated) return launch_epi<kStreamGated>(w, x, lb, v, p, grid, s);
    if (epi == kStreamRows) return launch_epi<kStreamRows>(w, x, lb, v, p, grid, s);
    return launch_epi<kStreamOut>(w, x, lb, v, p, grid, s);
}

}  // namespace fp8g
