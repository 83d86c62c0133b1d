// Products and gated projections with scales for blocks of 128, for few rows of
// A: bound by the weights' bytes.
//
// The weights are the MMA's operand of 128 rows, NT rows of A its columns, so a
// tile of C is 128 weight rows by NT.  A CTA holds a ring of 16 KB weight tiles (32
// KB for gate and up), with two CTAs on an SM about 200 KB in flight.  The K blocks
// of a tile are split over a cluster of up to eight CTAs, so that a narrow C
// still uses every SM; each CTA's share of the sum stays in its shared memory,
// and the CTAs add each other's (distributed shared memory) in rank order, each for
// its own rows of A, so results do not vary.
//
// As in block128_pair.cuh each K block's product goes to a tensor-memory buffer of
// its own and is added, scaled, to registers, in fragments of which a lane holds two rows
// of A of four weight rows: it reads a quarter of the rows' scales (a weight row a lane,
// shared memory took 512 cycles a K block of 128 rows to hand them out).  Beyond 64 sums
// a thread (128 rows of A, or 64 of gate and up) four more warps take half of the rows,
// and a CTA has its SM alone.  Measured (58.7 MB of weights, back to back): 1 x 4096 x 14336
// 11.8 us, 64 x 14336 x 4096 15 us; gate and up, 1 row of F 14336, K 4096 21 us, 5.6 TB/s.
//
// Roles (256 or 384 threads): warp 0 TMA, warp 1 MMA issue, warps 4 and up promotion; all
// warps add and store.
#include <cuda_bf16.h>

#include <atomic>

#include "block128.h"
#include "block128_math.cuh"
#include "block128_wait.cuh"
#include "ptx.cuh"

namespace fp8g {

namespace {

constexpr int kTile = kBlk * kBlk;

template <int NT, bool GATED>
struct Few {
    static constexpr int G = GATED ? 2 : 1;              // weight tiles of a stage
    static constexpr int COLS = G * NT;                  // tensor-memory columns of a buffer
    // up to 64 sums a thread; more take a second set of promotion warps and an SM alone
    static constexpr int HALVES = COLS > 64 ? 2 : 1;
    static constexpr int WT = NT / HALVES;               // rows of A of a promotion warp
    static constexpr int PROM = 4 * HALVES;
    static constexpr int WARPS = 4 + PROM;
    static constexpr int PER_SM = HALVES == 1 ? 2 : 1;
    static constexpr int STAGE = G * kTile + NT * kBlk;
    static constexpr int STAGES = (PER_SM == 2 ? 110592 : 212992) / STAGE;
    static constexpr int BUFS = 4;
    static constexpr int TMEM = COLS * BUFS;
    static constexpr int RING = STAGES * STAGE;
    static constexpr int PITCH = kBlk + 4;               // of a column's sums: a warp's stores in 32 banks
    static constexpr int SUMS = COLS * PITCH * 4;        // this CTA's sums, in the ring's place
    static_assert(SUMS <= RING && (TMEM & (TMEM - 1)) == 0 && TMEM * PER_SM <= 512, "");
    // a promotion warp's scales of CH K blocks, A's [CH][WT] then B's [CH][G]; two such
    // chunks, one ahead
    static constexpr int CH = GATED ? 2 : 4;
    static constexpr int SCALES = CH * (WT + G) < 4 ? 4 : (CH * (WT + G) + 3) / 4 * 4;
    static constexpr int OFF_S = RING;
    static constexpr int OFF_BAR = OFF_S + PROM * 2 * SCALES * 4;
    static constexpr int NUM_BARS = 2 * STAGES + 2 * BUFS + 1;
    static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
    static constexpr int BYTES = OFF_MISC + 16 + 1024;
    static_assert(PER_SM * (BYTES + 1024) <= 233472, "CTAs to an SM");
};

template <int NT, int OUT>
__global__ void __launch_bounds__(32 * Few<NT, (OUT >= kB128Gated)>::WARPS, Few<NT, (OUT >= kB128Gated)>::PER_SM)
    b128_few_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const B128Params p) {
    constexpr bool GATED = (OUT >= kB128Gated);
    using L = Few<NT, GATED>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = ptx::smem_addr(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (raw_base & 1023u)) & 1023u);
    const uint32_t sbase = ptx::smem_addr(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = (int)gridDim.z, rank = (int)blockIdx.z;  // the cluster is (1, 1, split)
    const int pn = (int)blockIdx.x;
    const int64_t m0 = (int64_t)blockIdx.y * NT;
    const int kb0 = (int)((int64_t)p.num_kb * rank / split), kb1 = (int)((int64_t)p.num_kb * (rank + 1) / split);

    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::OFF_BAR);
    auto bar_full = [&](int s) { return ptx::smem_addr(&bars[s]); };
    auto bar_empty = [&](int s) { return ptx::smem_addr(&bars[L::STAGES + s]); };
    auto bar_pfull = [&](int b) { return ptx::smem_addr(&bars[2 * L::STAGES + b]); };
    auto bar_pempty = [&](int b) { return ptx::smem_addr(&bars[2 * L::STAGES + L::BUFS + b]); };
    const uint32_t bar_drain = ptx::smem_addr(&bars[L::NUM_BARS - 1]);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::OFF_MISC + 4);

    if (threadIdx.x == 0) {
        for (int s = 0; s < L::STAGES; ++s) {
            ptx::mbar_init(bar_full(s), 1);
            ptx::mbar_init(bar_empty(s), 1);
        }
        for (int b = 0; b < L::BUFS; ++b) {
            ptx::mbar_init(bar_pfull(b), 1);
            ptx::mbar_init(bar_pempty(b), L::PROM);
        }
        ptx::mbar_init(bar_drain, 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&tmA);
        ptx::prefetch_tmap(&tmB);
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_addr(tmem_slot), L::TMEM);
        ptx::tmem_relinquish();
    }
    // The first weights on their way to L2 while the kernel before this one ends (3% of 1 x
    // 4096 x 14336; twice as many were slower, and so was this where a CTA has its SM alone).
    // L2 is where that kernel's writes go too, so nothing old is kept.
    if (L::PER_SM == 2 && threadIdx.x == 0) {
        const int32_t n0 = pn * kBlk;
        for (int kb = kb0; kb < kb1 && kb < kb0 + L::STAGES; ++kb) {
            if constexpr (GATED) {
                ptx::tma_prefetch_3d(&tmB, kb * kBlk, n0, 0);
                ptx::tma_prefetch_3d(&tmB, kb * kBlk, n0, 1);
            } else {
                ptx::tma_prefetch_2d(&tmB, p.b_mn ? n0 : kb * kBlk, p.b_mn ? kb * kBlk : n0);
            }
        }
    }
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            uint32_t stage = 0, phase = 0;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!wait_bar(bar_empty(stage), phase ^ 1u, abort_flag, p, 0 * 256 + stage)) break;
                const uint32_t fb = bar_full(stage), st = sbase + stage * L::STAGE;
                const int32_t k0 = kb * kBlk, n0 = pn * kBlk;
                ptx::mbar_arrive_expect_tx(fb, L::STAGE);
                if constexpr (GATED) {
                    ptx::tma_load_3d(st, &tmB, fb, k0, n0, 0);
                    ptx::tma_load_3d(st + kTile, &tmB, fb, k0, n0, 1);
                } else {
                    ptx::tma_load_2d(st, &tmB, fb, p.b_mn ? n0 : k0, p.b_mn ? k0 : n0);
                }
                ptx::tma_load_2d(st + L::G * kTile, &tmA, fb, k0, (int32_t)m0);
                if (++stage == L::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
    } else if (warp == 1) {
        // (whole warp, one elected lane: block128_pair.cuh)
        const uint32_t idesc = ptx::idesc_f8(kBlk, NT) | p.types;
        const uint32_t w_step = (p.b_mn ? 32 * kBlk : 32) >> 4;
        const uint64_t w_desc = ptx::smem_desc(sbase, 1024, 1024, 2);
        uint32_t stage = 0, phase = 0, buf = 0, bphase = 0;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!b128_wait_all(bar_full(stage), phase, abort_flag, p, 1 * 256 + stage)) break;
            if (!b128_wait_all(bar_pempty(buf), bphase ^ 1u, abort_flag, p, 1 * 256 + 64 + buf)) break;
            ptx::tc_fence_after();
            const uint64_t w0 = w_desc + stage * (L::STAGE >> 4), x0 = w0 + (L::G * kTile >> 4);
            if (ptx::elect_one()) {
#pragma unroll
                for (int g = 0; g < L::G; ++g)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        ptx::mma_f8(tmem_base + buf * L::COLS + g * NT, w0 + (g * kTile >> 4) + k * w_step, x0 + k * 2,
                                    idesc, k != 0 ? 1u : 0u);
                ptx::tc_commit(bar_pfull(buf));
                ptx::tc_commit(bar_empty(stage));
            }
            __syncwarp();
            if (++stage == L::STAGES) {
                stage = 0;
                phase ^= 1u;
            }
            if (++buf == L::BUFS) {
                buf = 0;
                bphase ^= 1u;
            }
        }
    } else if (warp >= 4) {
        const int q = warp & 3, half = (warp - 4) >> 2;
        const uint32_t taddr = ((uint32_t)(q * 32) << 16) + tmem_base + half * L::WT;
        float *sc = reinterpret_cast<float *>(smem + L::OFF_S) + (warp - 4) * 2 * L::SCALES;
        const float *sb = p.sb + (pn + (int64_t)(lane & (L::G - 1)) * p.n_blocks) * p.sb_n;
        // Scales of K blocks kb .. to chunk i
        auto ask = [&](int kb, int i) {
            const uint32_t at = ptx::smem_addr(sc + (i & 1) * L::SCALES);
#pragma unroll
            for (int j = 0; j < L::CH; ++j)
                if (kb + j < kb1) {
#pragma unroll
                    for (int r = 0; r < L::WT; r += 32)
                        if (lane + r < L::WT)
                            ptx::cp_async_4(at + (j * L::WT + lane + r) * 4,
                                            p.sa + (kb + j) * p.M + min(m0 + half * L::WT + lane + r, p.M - 1), 4);
                    if (lane < L::G) ptx::cp_async_4(at + (L::CH * L::WT + j * L::G + lane) * 4, sb + (kb + j) * p.sb_k, 4);
                }
            ptx::cp_async_commit();
        };
        ask(kb0, 0);
        // pairs of rows of A: fragment j / 2's of weight row 16 h + lane / 4, + 8 for odd j
        uint64_t acc[L::G][2][L::WT / 4];
#pragma unroll
        for (int g = 0; g < L::G; ++g)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < L::WT / 4; ++j) acc[g][h][j] = 0ull;
        uint32_t buf = 0, bphase = 0;
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb) {
            const int at_k = (kb - kb0) % L::CH, chunk = (kb - kb0) / L::CH;
            if (at_k == 0) {
                ptx::cp_async_wait<0>();
                __syncwarp();  // the chunk is there for every lane, and the one before it read by all
                ask(kb + L::CH, chunk + 1);
            }
            const float *s = sc + (chunk & 1) * L::SCALES;
            uint64_t fb[L::G];
#pragma unroll
            for (int g = 0; g < L::G; ++g) {
                const float f = s[L::CH * L::WT + at_k * L::G + g];
                fb[g] = b128_pair(f, f);
            }
            s += at_k * L::WT;
            if (!b128_wait_all(bar_pfull(buf), bphase, abort_flag, p, 3 * 256 + 64 + buf)) {
                ok = false;
                break;
            }
            ptx::tc_fence_after();
#pragma unroll
            for (int g = 0; g < L::G; ++g) {
                // both halves at once where registers allow; the scales are read meanwhile
                constexpr bool BOTH = L::PER_SM == 1 || L::WT < 64;
                uint32_t r[BOTH ? 2 : 1][L::WT / 2];
                auto load = [&](int h) {
                    ptx::tmem_ld_16x256b(taddr + buf * L::COLS + g * NT + ((uint32_t)h << 20), r[BOTH ? h : 0]);
                };
                load(0);
                if (BOTH) load(1);
                uint64_t f[L::WT / 8];
#pragma unroll
                for (int j = 0; j < L::WT / 8; ++j)
                    f[j] = b128_mul2(reinterpret_cast<const uint64_t *>(s)[4 * j + (lane & 3)], fb[g]);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (!BOTH && h == 1) load(1);
                    auto &v = r[BOTH ? h : 0];
                    ptx::tmem_ld_wait(v);
#pragma unroll
                    for (int j = 0; j < L::WT / 8; ++j) {
                        b128_fma2(acc[g][h][2 * j], b128_pair(v[4 * j], v[4 * j + 1]), f[j]);
                        b128_fma2(acc[g][h][2 * j + 1], b128_pair(v[4 * j + 2], v[4 * j + 3]), f[j]);
                    }
                }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar_pempty(buf));
            if (++buf == L::BUFS) {
                buf = 0;
                bphase ^= 1u;
            }
        }
        // every MMA and every copy of this CTA is done: its sums take the ring's place,
        // [column][weight row]
        if (ok) {
            float *sums = reinterpret_cast<float *>(smem) + q * 32 + (lane >> 2);
#pragma unroll
            for (int g = 0; g < L::G; ++g)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < L::WT / 4; ++j) {
                        float *at = sums + (g * NT + half * L::WT + 8 * (j >> 1) + 2 * (lane & 3)) * L::PITCH + 16 * h + 8 * (j & 1);
                        at[0] = b128_lo(acc[g][h][j]);
                        at[L::PITCH] = b128_hi(acc[g][h][j]);
                    }
        }
    }
    __syncwarp();
    __syncthreads();
    if (*abort_flag) {
        if (warp == 1 && lane == 0) {
            ptx::tc_commit(bar_drain);
            const uint64_t t0 = ptx::globaltimer();
            while (!ptx::mbar_try_wait(bar_drain, 0) && ptx::globaltimer() - t0 < p.timeout_ns) {
            }
        }
        const uint64_t t0 = ptx::globaltimer();
        while (ptx::globaltimer() - t0 < 200000ull) {
        }
        __syncthreads();
    }
    ptx::cluster_sync();  // the cluster's sums are in place
    // Row i of the tile's rows of A is added and stored by CTA i % split; a warp takes
    // a row at a time, four weight rows a lane.
    auto total = [&](int col) {
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const uint32_t at = sbase + (col * L::PITCH + 4 * lane) * 4;
        for (int j = 0; j < split; ++j) {
            const float4 o = ptx::ld_cluster_f4(ptx::map_shared(at, j));
            v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
        }
        return v;
    };
    for (int i = rank + split * warp; i < NT && m0 + i < p.M; i += split * L::WARPS) {
        const int64_t m = m0 + i, n = (int64_t)pn * kBlk + 4 * lane;
        if constexpr (!GATED) {
            float4 v = total(i);
            if (n < p.N) {
                if constexpr (OUT == kB128Bf16) {
                    __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
                    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.C) + m * p.N + n) =
                        make_uint2(*reinterpret_cast<uint32_t *>(&lo), *reinterpret_cast<uint32_t *>(&hi));
                } else {
                    float4 *c = reinterpret_cast<float4 *>(static_cast<float *>(p.C) + m * p.N + n);
                    if constexpr (OUT == kB128Add) {
                        const float4 o = *c;
                        v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
                    }
                    *c = v;
                }
            }
        } else {
            const float4 g = total(i), u = total(NT + i);
            constexpr int GATE = GATED ? OUT - kB128Gated : 0;
            const uint64_t h0 = b128_mul2(b128_gate2<GATE>(b128_pair(g.x, g.y)), b128_pair(u.x, u.y));
            const uint64_t h1 = b128_mul2(b128_gate2<GATE>(b128_pair(g.z, g.w)), b128_pair(u.z, u.w));
            const float4 h = make_float4(b128_lo(h0), b128_hi(h0), b128_lo(h1), b128_hi(h1));
            auto code = [&](const float4 v, uint8_t *q, float *s) {
                const float sv = b128_scale<FP8G_E4M3>(b128_warp_max(b128_amax4(v.x, v.y, v.z, v.w)));
                *reinterpret_cast<uint32_t *>(q) = b128_codes<FP8G_E4M3>(v.x, v.y, v.z, v.w, __frcp_rn(sv));
                if (lane == 0) *s = sv;
            };
            code(h, p.h + m * p.N + n, p.sh + pn * p.M + m);
            if (p.gu != nullptr) {
                code(g, p.gu + m * 2 * p.N + n, p.sgu + pn * p.M + m);
                code(u, p.gu + m * 2 * p.N + p.N + n, p.sgu + ((int64_t)p.n_blocks + pn) * p.M + m);
            }
        }
    }
    ptx::cluster_sync();  // no CTA leaves while another reads its sums
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem_base, L::TMEM);
    }
}

// The launch of n_blocks x rows clusters of `split`; to(kernel, configuration) uses it.
template <int NT, int OUT, typename F>
cudaError_t few_config(int64_t n_blocks, int64_t rows, int split, cudaStream_t stream, F to) {
    using L = Few<NT, (OUT >= kB128Gated)>;
    auto kern = b128_few_kernel<NT, OUT>;
    static unsigned long long done = 0ull;
    const cudaError_t e = b128_allow_smem(reinterpret_cast<const void *>(kern), L::BYTES, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)n_blocks, (unsigned)rows, (unsigned)split);
    cfg.blockDim = dim3(32 * L::WARPS, 1, 1);
    cfg.dynamicSmemBytes = L::BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = (unsigned)split;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return to(kern, cfg);
}

template <int NT, int OUT>
cudaError_t launch_few(const CUtensorMap &A, const CUtensorMap &B, const B128Params &p, int split,
                       cudaStream_t stream) {
    return few_config<NT, OUT>(p.n_blocks, (p.M + NT - 1) / NT, split, stream, [&](auto kern, cudaLaunchConfig_t &cfg) {
        return cudaLaunchKernelEx(&cfg, kern, A, B, p);
    });
}

template <int NT>
cudaError_t few_out(const CUtensorMap &A, const CUtensorMap &B, const B128Params &p, int out, int split,
                    cudaStream_t stream) {
    if (out == kB128Bf16) return launch_few<NT, kB128Bf16>(A, B, p, split, stream);
    if (out == kB128F32) return launch_few<NT, kB128F32>(A, B, p, split, stream);
    return launch_few<NT, kB128Add>(A, B, p, split, stream);
}

template <int OUT>
cudaError_t few_gated(const CUtensorMap &A, const CUtensorMap &B, const B128Params &p, int nt, int split,
                      cudaStream_t stream) {
    return nt == 16   ? launch_few<16, OUT>(A, B, p, split, stream)
           : nt == 32 ? launch_few<32, OUT>(A, B, p, split, stream)
                      : launch_few<64, OUT>(A, B, p, split, stream);
}

}  // namespace

int b128_few_clusters(int split, int dev) {
    static std::atomic<int> cache[64][9];
    std::atomic<int> &c = cache[dev & 63][split];
    int n = c.load(std::memory_order_relaxed);
    if (n > 0) return n;
    const cudaError_t e =
        few_config<128, kB128Bf16>(64, 1, split, nullptr, [&](auto kern, cudaLaunchConfig_t &cfg) {
            return cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
        });
    if (e != cudaSuccess || n < 1) {
        cudaGetLastError();  // clear
        return 0;
    }
    c.store(n, std::memory_order_relaxed);
    return n;
}

cudaError_t launch_b128_few(const CUtensorMap &A, const CUtensorMap &B, const B128Params &p, int out,
                            int nt, int split, cudaStream_t stream) {
    if (out == kB128Gated + FP8G_GATE_SILU) return few_gated<kB128Gated + FP8G_GATE_SILU>(A, B, p, nt, split, stream);
    if (out == kB128Gated + FP8G_GATE_GELU) return few_gated<kB128Gated + FP8G_GATE_GELU>(A, B, p, nt, split, stream);
    if (out == kB128Gated + FP8G_GATE_RELU) return few_gated<kB128Gated + FP8G_GATE_RELU>(A, B, p, nt, split, stream);
    return nt == 16    ? few_out<16>(A, B, p, out, split, stream)
           : nt == 32  ? few_out<32>(A, B, p, out, split, stream)
           : nt == 64  ? few_out<64>(A, B, p, out, split, stream)
                       : few_out<128>(A, B, p, out, split, stream);
}

}  // namespace fp8g
