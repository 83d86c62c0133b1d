// Few tokens against block-scaled weights that are read once, in one launch:
// the MoE layer (quantise, gate/up product, gated activation, down product,
// weighted sum) and the projection with low-rank adapters (quantise, A x,
// product with the adapters' B as further K steps).
//
//   D[f, t] = sum_k (s W)[f, k] (s X)[t, k]
//
// The weights are the MMA's 128-row operand and the tokens its columns
// (tcgen05.mma kind::mxf8f6f4, M = 128, N = the group's tokens rounded up to
// 16): with few tokens a tile costs what its weights cost to load, and no CUDA
// core touches them.  A work unit is one 128-wide K step of a pair of 128-row
// weight tiles (32 KB: the gate and the up rows of the same features, or two
// neighbouring tiles).  The units of all groups, tiles and K steps of a product
// are one line that the CTAs, one per SM, share out evenly, so every SM streams
// the same number of bytes whatever the shape.
//
// Split tiles.  A CTA's span may begin and end inside a tile.  The tile belongs
// to the CTA that has its first unit, which comes to it last; the others begin
// with it, store their fp32 partial and raise a flag long before the owner asks.
// The owner adds them to its own accumulator in unit order, so the result does
// not depend on timing.
//
// Phases.  The CTAs meet at flag barriers (each raises its own flag, a warp of
// each watches all of them): tokens quantised, h quantised, y complete.  The
// weights wait for none of them: the producer fills the ring with the next
// product's weights and only the tokens' slices follow the barrier, so HBM
// stays busy across phases.  The waits need every CTA resident: a cooperative
// launch, one CTA per SM; each is bounded, and on expiry records
// FP8G_ERR_TIMEOUT and the CTA leaves.  Flags hold the call's token, so a new
// temporary needs no clearing; flags 1 and up are zeroed before the first
// barrier and flag 0 after the second, so a replayed graph finds them clear.
//
// Roles: warp 0 TMA producer, warp 1 MMAs, warp 2 scale copies to tensor
// memory, warp 3 watches the barriers, warps 4-11 quantise the tokens, then
// run the epilogues.
//
// Low-rank steps: after its FP8 steps a tile takes, per adapter among the
// group's tokens, bf16 steps (kind::f16) of the adapter's B rows against V =
// alpha A x (zero for the tokens of others), into the same fp32 accumulator.
#include <cuda_bf16.h>

#include <atomic>

#include "kernel_common.cuh"
#include "quant_math.cuh"
#include "stream.h"

namespace fp8g {

namespace {

constexpr int kSThreads = 384;
constexpr int kSEpiWarp0 = 4;
constexpr int kSEpiWarps = 8;
constexpr int kEpiThreads = kSEpiWarps * 32;
constexpr int kWTile = 128 * 128;  // bytes of a weight tile in shared memory
constexpr int kMaxStages = 16;
constexpr int kSfSlot = 16;        // tensor-memory columns of a stage's scales
constexpr int kMinUnits = 4;       // work units a CTA takes at least
constexpr int kJoin = 4;           // partial tiles read at a time
constexpr int kSmemMax = 232448;
constexpr int kGates = 3;
constexpr int kAdWords = FP8G_MAX_ADAPTERS / 32;

enum Epi : int { kGated, kRows, kOut };
// flag arrays: barriers 0-2, partial stored (first, second product)
constexpr int kFlagPart = 3;

// One group: up to nb token rows against one weight matrix.
struct Group {
    int32_t mat, row0, n;
};

struct TailBase {
    uint64_t full[kMaxStages], empty[kMaxStages], sfr[kMaxStages], accf[2], acce[2], drain, drain_sf;
    uint64_t gate[kGates];     // barrier b passed (the watcher arrives)
    uint64_t arrived[kGates];  // this CTA arrived at barrier b (the epilogue arrives)
    uint32_t tmem;
    int abort_flag;
    int n_groups;
};
struct TailMoe : TailBase {
    Group g[kStreamMaxGroups];
    int32_t cnt[FP8G_MAX_ROUTED_EXPERTS], off[FP8G_MAX_ROUTED_EXPERTS], goff[FP8G_MAX_ROUTED_EXPERTS];
    int32_t row[FP8G_MAX_TOP_K], grp[FP8G_MAX_TOP_K], in[FP8G_MAX_TOP_K];  // of the token at hand
};
struct TailLora : TailBase {
    int32_t unit0[kStreamLoraGroups + 1];
    uint32_t bits[kStreamLoraGroups][kAdWords];          // adapters of a group's rows
    int16_t word0[kStreamLoraGroups][kAdWords];          // slots before a word's
    int32_t n[kStreamLoraGroups];                        // slots
    int16_t adapter[kStreamLoraGroups][kStreamMaxTokens];
    int32_t rows_of[kStreamLoraGroups][kStreamMaxTokens];  // rows of a slot
    int32_t pick[4], rows[16];                           // the item at hand
    float acc[kSEpiWarps / 2][16][17];
};
template <bool LORA>
struct TailOf {
    using T = TailMoe;
};
template <>
struct TailOf<true> {
    using T = TailLora;
};

static_assert(kSmemMax - 1024 - (int)(sizeof(TailMoe) > sizeof(TailLora) ? sizeof(TailMoe) : sizeof(TailLora)) >= 6 * (2 * kWTile + 16 * 128 + 2048),
              "six stages with 16 token columns");

// A CTA's part of one tile: units [k0, k1) of its upt.
struct Tile {
    int32_t g, mt, row0, n, n16;
    int32_t mat0, mat1, w0, w1;  // matrix and first row of the two weight tiles
    bool has1;                   // the second one exists
    int32_t k0, k1, upt;
    int64_t u;                   // the tile's first unit
};

// First unit of CTA c of G sharing U units, and the CTA that owns unit u.
__device__ __forceinline__ int64_t span_begin(int64_t U, int G, int c) { return U * c / G; }
__device__ __forceinline__ int span_owner(int64_t U, int G, int64_t u) {
    return (int)(((u + 1) * G - 1) / U);
}

// This CTA's units [u, end) of a product of U units shared by G CTAs.
struct Walk {
    int64_t u, end, U;
    int G;
};

template <bool LORA>
__device__ __forceinline__ int64_t units_of(const StreamParams &p, const typename TailOf<LORA>::T &t,
                                            int ph) {
    if constexpr (LORA)
        return t.unit0[t.n_groups];
    else
        return (int64_t)t.n_groups * p.ph[ph].mt * p.ph[ph].ks;
}

template <bool LORA>
__device__ __forceinline__ Walk walk_of(const StreamParams &p, const typename TailOf<LORA>::T &t, int ph) {
    Walk w;
    w.U = units_of<LORA>(p, t, ph);
    w.G = (int)max((int64_t)1, min((int64_t)gridDim.x, w.U / kMinUnits));
    const int c = blockIdx.x;
    w.u = c < w.G ? span_begin(w.U, w.G, c) : 0;
    w.end = c < w.G ? span_begin(w.U, w.G, c + 1) : 0;
    return w;
}

template <int EPI>
__device__ __forceinline__ bool next_tile(const StreamParams &p, const StreamPhase &h,
                                          const typename TailOf<EPI == kOut>::T &t, Walk &w, Tile &o) {
    if (w.u >= w.end) return false;
    int64_t first;
    if constexpr (EPI == kOut) {
        int g = 0;
        while (t.unit0[g + 1] <= w.u) ++g;
        o.g = g;
        o.upt = h.ks + t.n[g] * p.kr;
        first = t.unit0[g];
        o.row0 = g * p.nb;
        o.n = min(p.nb, p.T - o.row0);
        o.mat0 = 0;
    } else {
        o.upt = h.ks;
        o.g = (int)(w.u / ((int64_t)h.mt * h.ks));
        first = (int64_t)o.g * h.mt * h.ks;
        const Group gr = t.g[o.g];
        o.row0 = gr.row0;
        o.n = gr.n;
        o.mat0 = EPI == kGated ? 2 * gr.mat : gr.mat;
    }
    const int32_t rel = (int32_t)(w.u - first);
    o.mt = rel / o.upt;
    o.k0 = rel - o.mt * o.upt;
    o.k1 = (int32_t)min((int64_t)o.upt, o.k0 + (w.end - w.u));
    o.u = w.u - o.k0;
    o.n16 = (o.n + 15) & ~15;
    if constexpr (EPI == kGated) {
        o.mat1 = o.mat0 + 1;
        o.w0 = o.w1 = o.mt * 128;
        o.has1 = true;
    } else {
        o.mat1 = o.mat0;
        o.w0 = o.mt * 128 * h.sub;
        o.w1 = o.w0 + 128;
        o.has1 = h.sub == 2 && o.w1 < h.rows;
    }
    w.u += o.k1 - o.k0;
    return true;
}

// --------------------------------------------------------------- flags
__device__ __forceinline__ void flag_set(uint64_t *f, uint64_t v) {
    asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(f), "l"(v) : "memory");
}
__device__ __forceinline__ uint64_t flag_get(const uint64_t *f) {
    uint64_t v;
    asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(f) : "memory");
    return v;
}
// Global memory written by ordinary stores before, read by TMA after (or the
// reverse order of proxies): on both sides of a flag.
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

// Whole warp: until f[c] holds the token for every c in [lo, hi).  Bounded.
__device__ __forceinline__ bool flags_wait(const StreamParams &p, const uint64_t *f, int lo, int hi,
                                           volatile int *abort_flag, unsigned detail) {
    const int lane = threadIdx.x & 31;
    int ok = 1;
    uint64_t t0 = 0;
    for (int c = lo + lane; c < hi && ok; c += 32) {
        while (flag_get(f + c) != p.token) {
            if (t0 == 0) t0 = ptx::globaltimer();
            if (*abort_flag) {
                ok = 0;
                break;
            }
            if (ptx::globaltimer() - t0 > p.timeout_ns) {
                *abort_flag = 1;
                record_error(p, FP8G_ERR_TIMEOUT, detail);
                ok = 0;
                break;
            }
        }
    }
    ok = __all_sync(0xffffffffu, ok);
    __syncwarp();  // what the lanes acquired is ordered before what the warp does next
    return ok != 0;
}

// All epilogue warps: the AND of their flags, and a barrier among them (each of
// them takes part in every call, so none is left waiting).
__device__ __forceinline__ bool epi_all(bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "barrier.cta.red.and.pred p, 1, %2, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(ok ? 1u : 0u), "n"(kEpiThreads)
        : "memory");
    return r != 0;
}

// All epilogue warps: this CTA's writes so far are done; raise its flag of
// barrier b and let the watcher look at the others'.
__device__ __forceinline__ void arrive(const StreamParams &p, TailBase &t, int b) {
    fence_proxy_async_all();
    (void)epi_all(true);
    if (threadIdx.x == kSEpiWarp0 * 32) {
        flag_set(p.flags + (int64_t)b * gridDim.x + blockIdx.x, p.token);
        ptx::mbar_arrive(ptx::smem_addr(&t.arrived[b]));
    }
}

// --------------------------------------------------------------- tables
__device__ __forceinline__ int warp_scan(int v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
    }
    return v;
}

// The groups, from the call's indices.  Call with all threads.
__device__ __forceinline__ void make_tables(const StreamParams &p, TailMoe &t) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < p.n_mat; e += kSThreads) t.cnt[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < p.n_idx; i += kSThreads) {
        const int e = __ldg(p.idx + i);
        if (e >= p.n_mat && blockIdx.x == 0) record_error(p, FP8G_ERR_INVALID_ARG, (unsigned)i);
        if (e >= 0 && e < p.n_mat) atomicAdd(&t.cnt[e], 1);
    }
    __syncthreads();
    if (warp == 0) {
        int rr = 0, gg = 0;
        for (int e0 = 0; e0 < p.n_mat; e0 += 32) {
            const int e = e0 + lane;
            const int c = e < p.n_mat ? t.cnt[e] : 0, ng = (c + p.nb - 1) / p.nb;
            const int s = warp_scan(c, lane), sg = warp_scan(ng, lane);
            if (e < p.n_mat) {
                t.off[e] = rr + s - c;
                t.goff[e] = gg + sg - ng;
            }
            for (int i = 0; i < ng; ++i)
                t.g[gg + sg - ng + i] = Group{e, rr + s - c + i * p.nb, min(p.nb, c - i * p.nb)};
            rr += __shfl_sync(0xffffffffu, s, 31);
            gg += __shfl_sync(0xffffffffu, sg, 31);
        }
        if (lane == 0) t.n_groups = gg;
    }
}

__device__ __forceinline__ void make_tables(const StreamParams &p, TailLora &t) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ng = (p.T + p.nb - 1) / p.nb;
    for (int i = threadIdx.x; i < kStreamLoraGroups * kAdWords; i += kSThreads) t.bits[0][i] = 0;
    for (int i = threadIdx.x; i < kStreamLoraGroups * kStreamMaxTokens; i += kSThreads) t.rows_of[0][i] = 0;
    __syncthreads();
    if (p.kr > 0) {
        for (int i = threadIdx.x; i < p.T; i += kSThreads) {
            const int l = __ldg(p.idx + i);
            if (l >= p.n_mat && blockIdx.x == 0) record_error(p, FP8G_ERR_INVALID_ARG, (unsigned)i);
            if (l >= 0 && l < p.n_mat) atomicOr(&t.bits[i / p.nb][l >> 5], 1u << (l & 31));
        }
        __syncthreads();
    }
    if (warp < ng) {  // lane i: adapters 32 i .. 32 i + 31
        const uint32_t w = t.bits[warp][lane];
        const int c = __popc(w), s = warp_scan(c, lane);
        int at = s - c;
        t.word0[warp][lane] = (int16_t)at;
        for (uint32_t m = w; m != 0; m &= m - 1)
            t.adapter[warp][at++] = (int16_t)(32 * lane + __ffs((int)m) - 1);
        if (lane == 31) t.n[warp] = s;
    }
    __syncthreads();
    if (p.kr > 0)
        for (int i = threadIdx.x; i < p.T; i += kSThreads) {
            const int l = __ldg(p.idx + i), g = i / p.nb;
            if (l < 0 || l >= p.n_mat) continue;
            const int s = t.word0[g][l >> 5] + __popc(t.bits[g][l >> 5] & ((1u << (l & 31)) - 1u));
            atomicAdd(&t.rows_of[g][s], 1);
        }
    if (threadIdx.x == 0) {
        int u = 0;
        for (int g = 0; g < ng; ++g) {
            t.unit0[g] = u;
            u += p.ph[0].mt * (p.ph[0].ks + t.n[g] * p.kr);
        }
        t.unit0[ng] = u;
        t.n_groups = ng;
    }
}

// ----------------------------------------------------- quantising the tokens
// Epilogue warps.  An item is a token and 2048 of its values, eight a thread
// (a 1x32 block is four threads).  Blocks past K in the last 128-wide step get
// scale 1.
__device__ __forceinline__ int quant_segments(const StreamParams &p, int ks) {
    return (ks * 16 + kEpiThreads - 1) / kEpiThreads;
}

__device__ __forceinline__ void load_x8(const StreamParams &p, int64_t off, float4 &a, float4 &b) {
    if (p.x_bf16)
        load8<true>(p.x, off, a, b);
    else
        load8<false>(p.x, off, a, b);
}

struct Quant8 {
    uint2 q;
    uint8_t sf;
    bool in;
};
__device__ __forceinline__ Quant8 quant_8(const StreamParams &p, int t, int c) {
    float4 v0 = make_float4(0.f, 0.f, 0.f, 0.f), v1 = v0;
    Quant8 r;
    r.in = c * 8 < p.K;
    if (r.in) load_x8(p, (int64_t)t * p.K + c * 8, v0, v1);
    float am = absmax8(v0, v1);
    am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
    am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
    const float s = pow2_scale<0>(am);
    r.q = quant8_pow2<0>(v0, v1, s);
    r.sf = (uint8_t)(__float_as_uint(s) >> 23);
    return r;
}

// Scale byte of row r (of a group's tile), value group c: chunk c / 16, block c / 4 % 4.
__device__ __forceinline__ int64_t sf_at(int64_t group, int ks, int r, int c) {
    return (group * ks + (c >> 4)) * 512 + 16 * (r & 31) + 4 * (r >> 5) + ((c >> 2) & 3);
}

__device__ __forceinline__ void prepare(const StreamParams &p, TailMoe &t) {
    const int tid = threadIdx.x - kSEpiWarp0 * 32, warp = tid >> 5, lane = tid & 31;
    const int ks = p.ph[0].ks, segs = quant_segments(p, ks);
    int last = -1;
    for (int it = blockIdx.x; it < p.T * segs; it += gridDim.x) {
        const int tok = it / segs, c = (it - tok * segs) * kEpiThreads + tid;
        const Quant8 q = quant_8(p, tok, c);
        if (tok != last) {
            // the token's rows in expert order: the pairs before it of the same expert
            (void)epi_all(true);
            for (int j = warp; j < p.k; j += kSEpiWarps) {
                const int i = tok * p.k + j;
                int e = __ldg(p.idx + i);
                if (e >= p.n_mat) e = -1;
                int before = 0;
                if (e >= 0) {
#pragma unroll 4
                    for (int o = lane; o < i; o += 32) before += __ldg(p.idx + o) == e;
                }
                before = __reduce_add_sync(0xffffffffu, before);
                if (lane == 0) {
                    t.row[j] = e >= 0 ? t.off[e] + before : -1;
                    t.grp[j] = e >= 0 ? t.goff[e] + before / p.nb : 0;
                    t.in[j] = before % p.nb;
                }
            }
            (void)epi_all(true);
            if (it == tok * segs)
                for (int j = tid; j < p.k; j += kEpiThreads) p.pos[tok * p.k + j] = t.row[j];
            last = tok;
        }
        if (c < ks * 16)
            for (int j = 0; j < p.k; ++j) {
                const int row = t.row[j];
                if (row < 0) continue;
                if (q.in) *reinterpret_cast<uint2 *>(p.xq + (int64_t)row * p.K + c * 8) = q.q;
                if ((c & 3) == 0) p.xsf[sf_at(t.grp[j], ks, t.in[j], c)] = q.sf;
            }
    }
}

__device__ __forceinline__ void prepare(const StreamParams &p, TailLora &) {
    const int tid = threadIdx.x - kSEpiWarp0 * 32;
    const int ks = p.ph[0].ks, segs = quant_segments(p, ks);
    for (int it = blockIdx.x; it < p.T * segs; it += gridDim.x) {
        const int tok = it / segs, c = (it - tok * segs) * kEpiThreads + tid;
        const Quant8 q = quant_8(p, tok, c);
        if (c >= ks * 16) continue;
        if (q.in) *reinterpret_cast<uint2 *>(p.xq + (int64_t)tok * p.K + c * 8) = q.q;
        if ((c & 3) == 0) p.xsf[sf_at(tok / p.nb, ks, tok % p.nb, c)] = q.sf;
    }
}

// ------------------------------------------------------------ V = alpha A x
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&b);
}
__device__ __forceinline__ float bf16_rest(float v) { return v - __bfloat162float(__float2bfloat16_rn(v)); }

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Eight values of x as bf16 pairs; of fp32 x the rounded values (hi) and what
// they leave, rounded (lo).
__device__ __forceinline__ void x_pairs(const StreamParams &p, int64_t off, bool in, uint4 &hi, uint4 &lo) {
    hi = lo = make_uint4(0u, 0u, 0u, 0u);
    if (!in) return;
    if (p.x_bf16) {
        hi = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.x) + off));
        return;
    }
    float4 a, b;
    load8<false>(p.x, off, a, b);
    hi = make_uint4(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w), pack_bf16(b.x, b.y), pack_bf16(b.z, b.w));
    lo = make_uint4(pack_bf16(bf16_rest(a.x), bf16_rest(a.y)), pack_bf16(bf16_rest(a.z), bf16_rest(a.w)),
                    pack_bf16(bf16_rest(b.x), bf16_rest(b.y)), pack_bf16(bf16_rest(b.z), bf16_rest(b.w)));
}

// Epilogue warps.  An item is 16 rows of a slot against 16 ranks of its
// adapter; the K range goes over the eight warps, each a 16 x 16 product by
// mma.sync, joined in warp order.  A lane's 16-byte load covers 8 consecutive K
// of a row; the same K permutation on both operands leaves the product as it
// is.  Bound by the latency of its loads (an adapter's 16 ranks are 131 KB at
// K = 4096): kU K steps of 32 are in flight per warp.
__device__ __forceinline__ void low_rank(const StreamParams &p, TailLora &t) {
    const int tid = threadIdx.x - kSEpiWarp0 * 32, warp = tid >> 5, lane = tid & 31;
    const int rblocks = (p.rank + 15) / 16;
    const __nv_bfloat16 *A = static_cast<const __nv_bfloat16 *>(p.a);
    for (int item = blockIdx.x;; item += gridDim.x) {
        (void)epi_all(true);  // the previous item's shared data are read
        if (warp == 0) {
            // item -> group, slot, 16 rows, rank block
            int at = 0;
            if (lane == 0) t.pick[0] = -1;
            for (int g = 0; g < t.n_groups; ++g)
                for (int s0 = 0; s0 < t.n[g]; s0 += 32) {
                    const int s = s0 + lane;
                    const int c = s < t.n[g] ? (t.rows_of[g][s] + 15) / 16 * rblocks : 0;
                    const int incl = warp_scan(c, lane), first = at + incl - c;
                    if (item >= first && item < first + c) {
                        t.pick[0] = g;
                        t.pick[1] = s;
                        t.pick[2] = (item - first) / rblocks * 16;
                        t.pick[3] = (item - first) % rblocks;
                    }
                    at += __shfl_sync(0xffffffffu, incl, 31);
                }
            if (lane < 16) t.rows[lane] = -1;
            __syncwarp();
            if (t.pick[0] >= 0) {
                const int g = t.pick[0], l = t.adapter[g][t.pick[1]];
                int seen = 0;
                for (int i0 = 0; i0 < p.nb; i0 += 32) {
                    const int i = g * p.nb + i0 + lane;
                    const bool m = i0 + lane < p.nb && i < p.T && __ldg(p.idx + i) == l;
                    const uint32_t b = __ballot_sync(0xffffffffu, m);
                    const int w = seen + __popc(b & ((1u << lane) - 1u)) - t.pick[2];
                    if (m && w >= 0 && w < 16) t.rows[w] = i0 + lane;
                    seen += __popc(b);
                }
            }
        }
        (void)epi_all(true);
        const int g = t.pick[0];
        if (g < 0) break;  // the same for all warps
        const int slot = t.pick[1], l = t.adapter[g][slot], rb = t.pick[3], row0 = g * p.nb;
        __nv_bfloat16 *hi = static_cast<__nv_bfloat16 *>(p.v) +
                            (int64_t)(g * p.slot_cap + slot) * p.halves * p.nb * p.r64 + rb * 16;
        const int64_t half = p.halves == 2 ? (int64_t)p.nb * p.r64 : 32;
        const uint4 z = make_uint4(0u, 0u, 0u, 0u);
        if (t.pick[2] == 0) {
            // the slot's first rows: zeros for the tokens of other adapters, and
            // in the columns past the rank
            const int cols = (p.halves == 2 ? p.r64 : 32) / 8;
            for (int i = tid; i < p.nb; i += kEpiThreads) {
                uint4 *d = reinterpret_cast<uint4 *>(hi + (int64_t)i * p.r64);
                uint4 *e = reinterpret_cast<uint4 *>(hi + half + (int64_t)i * p.r64);
                if (row0 + i >= p.T || __ldg(p.idx + row0 + i) != l) d[0] = d[1] = e[0] = e[1] = z;
                if (rb == 0)
                    for (int c = 2 * rblocks; c < cols; ++c) d[c] = e[c] = z;
            }
        }
        const int gr = lane >> 2, c8 = 8 * (lane & 3);
        const int i0 = t.rows[gr], i1 = t.rows[gr + 8];
        const int64_t x0 = (int64_t)(row0 + max(i0, 0)) * p.K + c8;
        const int64_t x1 = (int64_t)(row0 + max(i1, 0)) * p.K + c8;
        const int r0 = rb * 16 + gr, r1 = r0 + 8;
        const __nv_bfloat16 *a0 = A + ((int64_t)l * p.rank + min(r0, p.rank - 1)) * p.K + c8;
        const __nv_bfloat16 *a1 = A + ((int64_t)l * p.rank + min(r1, p.rank - 1)) * p.K + c8;
        float d0[4] = {}, d1[4] = {};
        const int steps = p.K / 32;  // K is a multiple of 32
        constexpr int kU = 4;
        for (int s0 = warp * kU; s0 < steps; s0 += kSEpiWarps * kU) {
            uint4 xa[kU], xb[kU], ya[kU], yb[kU], wa[kU], wb[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const bool in = s0 + u < steps;
                const int64_t k = in ? (int64_t)(s0 + u) * 32 : 0;
                x_pairs(p, x0 + k, in && i0 >= 0, xa[u], ya[u]);
                x_pairs(p, x1 + k, in && i1 >= 0, xb[u], yb[u]);
                wa[u] = in && r0 < p.rank ? __ldg(reinterpret_cast<const uint4 *>(a0 + k)) : z;
                wb[u] = in && r1 < p.rank ? __ldg(reinterpret_cast<const uint4 *>(a1 + k)) : z;
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const uint32_t f0[4] = {xa[u].x, xb[u].x, xa[u].y, xb[u].y};
                const uint32_t f1[4] = {xa[u].z, xb[u].z, xa[u].w, xb[u].w};
                mma_16816(d0, f0, wa[u].x, wa[u].y);
                mma_16816(d1, f0, wb[u].x, wb[u].y);
                mma_16816(d0, f1, wa[u].z, wa[u].w);
                mma_16816(d1, f1, wb[u].z, wb[u].w);
                if (!p.x_bf16) {
                    const uint32_t h0[4] = {ya[u].x, yb[u].x, ya[u].y, yb[u].y};
                    const uint32_t h1[4] = {ya[u].z, yb[u].z, ya[u].w, yb[u].w};
                    mma_16816(d0, h0, wa[u].x, wa[u].y);
                    mma_16816(d1, h0, wb[u].x, wb[u].y);
                    mma_16816(d0, h1, wa[u].z, wa[u].w);
                    mma_16816(d1, h1, wb[u].z, wb[u].w);
                }
            }
        }
        // the warps' products: warp w + 4 to warp w, then the four in order
        const int c2 = 2 * (lane & 3);
        float(*acc)[17] = t.acc[warp & 3];
        if (warp >= 4) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                acc[gr + 8 * (e >> 1)][c2 + (e & 1)] = d0[e];
                acc[gr + 8 * (e >> 1)][8 + c2 + (e & 1)] = d1[e];
            }
        }
        (void)epi_all(true);
        if (warp < 4) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                acc[gr + 8 * (e >> 1)][c2 + (e & 1)] += d0[e];
                acc[gr + 8 * (e >> 1)][8 + c2 + (e & 1)] += d1[e];
            }
        }
        (void)epi_all(true);
        {
            const int i = tid >> 4, c = tid & 15, row = t.rows[i];
            float v = 0.0f;
#pragma unroll
            for (int q = 0; q < kSEpiWarps / 2; ++q) v += t.acc[q][i][c];
            if (p.alpha != nullptr) v *= __ldg(p.alpha + l);
            if (rb * 16 + c >= p.rank) v = 0.0f;
            if (row >= 0) {
                const float rest = bf16_rest(v);  // none for an infinite or NaN V
                hi[(int64_t)row * p.r64 + c] = __float2bfloat16_rn(v);
                hi[half + (int64_t)row * p.r64 + c] = __float2bfloat16_rn(isfinite(rest) ? rest : 0.0f);
            }
        }
    }
}

// ------------------------------------------------------------------ roles
// The ring's position, carried from one product to the next.
struct Ring {
    int stage = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(const StreamParams &p) {
        if (++stage == p.stages) {
            stage = 0;
            phase ^= 1u;
        }
    }
};

template <int EPI>
struct Loader {
    using Tail = typename TailOf<EPI == kOut>::T;
    const StreamParams &p;
    const StreamPhase &h;
    Tail &t;
    uint32_t sbase;

    // Weights and their scales (or an adapter's rows) of a step, with the
    // bytes of the whole stage announced.
    __device__ __forceinline__ void weights(const Tile &o, int k, int stage) const {
        const uint32_t fb = ptx::smem_addr(&t.full[stage]);
        const uint32_t s0 = sbase + stage * p.stage_bytes, sf = s0 + 2 * kWTile + p.x_bytes;
        const uint32_t nw = o.has1 ? 2 : 1;
        if (EPI != kOut || k < h.ks) {
            const uint32_t w_tx = kWTile - kWTile / 8 * p.gap8;
            ptx::mbar_arrive_expect_tx(fb, nw * (w_tx + 512u) + o.n16 * 128u + 512u);
            const int64_t c0 = ((int64_t)o.mat0 * h.ks + k) * h.n_rt + o.w0 / 128;
            ptx::tma_load_3d(s0, &h.W, fb, k * kBK, o.w0, o.mat0);
            ptx::bulk_load(sf, h.sfw + c0 * 512, 512, fb);
            if (o.has1) {
                const int64_t c1 = ((int64_t)o.mat1 * h.ks + k) * h.n_rt + o.w1 / 128;
                ptx::tma_load_3d(s0 + kWTile, &h.W, fb, k * kBK, o.w1, o.mat1);
                ptx::bulk_load(sf + 512, h.sfw + c1 * 512, 512, fb);
            }
        } else if constexpr (EPI == kOut) {
            const int ls = k - h.ks, sl = ls / p.kr, c = (ls - sl * p.kr) * 64;
            const int l = t.adapter[o.g][sl];
            ptx::mbar_arrive_expect_tx(fb, nw * kWTile + p.halves * o.n16 * 128u);
            ptx::tma_load_3d(s0, &p.B, fb, c, o.w0, l);
            if (o.has1) ptx::tma_load_3d(s0 + kWTile, &p.B, fb, c, o.w1, l);
        }
    }
    // The tokens' slice and its scales (or V's) of a step.
    __device__ __forceinline__ void tokens(const Tile &o, int k, int stage) const {
        const uint32_t fb = ptx::smem_addr(&t.full[stage]);
        const uint32_t s0 = sbase + stage * p.stage_bytes, x0 = s0 + 2 * kWTile;
        if (EPI != kOut || k < h.ks) {
            ptx::bulk_load(x0 + p.x_bytes + 1024, h.sfx + ((int64_t)o.g * h.ks + k) * 512, 512, fb);
            for (int i = 0; i < o.n16; i += 16)
                ptx::tma_load_2d(x0 + i * 128, &h.X, fb, k * kBK, o.row0 + i);
        } else if constexpr (EPI == kOut) {
            const int ls = k - h.ks, sl = ls / p.kr, c = (ls - sl * p.kr) * 64;
            const int v0 = (o.g * p.slot_cap + sl) * p.halves * p.nb;
            for (int b = 0; b < p.halves; ++b)
                for (int i = 0; i < o.n16; i += 16)
                    ptx::tma_load_2d(x0 + (b * p.nb + i) * 128, &p.V, fb, c, v0 + b * p.nb + i);
        }
    }
};

// Producer (one thread): a product's stages.  The first ring's worth of weights
// goes out as stages come free; the tokens' slices follow gate `b` (of low-rank
// steps gate b + 1).  False: aborting.
template <int EPI>
__device__ __forceinline__ bool produce(const StreamParams &p, typename TailOf<EPI == kOut>::T &t, int ph,
                                        int b, Ring &r, uint32_t sbase) {
    volatile int *abort_flag = &t.abort_flag;
    const StreamPhase &h = p.ph[ph];
    const Loader<EPI> load{p, h, t, sbase};
    const Walk w0 = walk_of<EPI == kOut>(p, t, ph);
    Tile o;
    int ahead = 0;
    {
        Walk w = w0;
        Ring q = r;
        while (ahead < p.stages && next_tile<EPI>(p, h, t, w, o))
            for (int k = o.k0; k < o.k1 && ahead < p.stages; ++k, ++ahead) {
                if (!wait_bar(ptx::smem_addr(&t.empty[q.stage]), q.phase ^ 1u, abort_flag, p, q.stage))
                    return false;
                load.weights(o, k, q.stage);
                q.next(p);
            }
    }
    Walk w = w0;
    int done = 0, open = 0;
    while (next_tile<EPI>(p, h, t, w, o))
        for (int k = o.k0; k < o.k1; ++k, ++done) {
            if (done >= ahead) {
                if (!wait_bar(ptx::smem_addr(&t.empty[r.stage]), r.phase ^ 1u, abort_flag, p, r.stage))
                    return false;
                load.weights(o, k, r.stage);
            }
            const int need = EPI == kOut && k >= h.ks ? 2 : 1;
            while (open < need) {
                if (!wait_bar(ptx::smem_addr(&t.gate[b + open]), 0, abort_flag, p, 4 * 256 + b + open))
                    return false;
                fence_proxy_async_all();
                ++open;
            }
            load.tokens(o, k, r.stage);
            r.next(p);
        }
    return true;
}

// Scale copies (one thread).  From a thread of their own: issued by the MMA
// thread each copy holds up the MMAs behind it.  A stage's columns are
// rewritten only after its next "full", when the MMAs that read them are done.
template <int EPI>
__device__ __forceinline__ bool copy_scales(const StreamParams &p, typename TailOf<EPI == kOut>::T &t, int ph,
                                            Ring &r, uint32_t sbase, uint32_t sf_tmem) {
    const StreamPhase &h = p.ph[ph];
    Walk w = walk_of<EPI == kOut>(p, t, ph);
    Tile o;
    while (next_tile<EPI>(p, h, t, w, o))
        for (int k = o.k0; k < o.k1; ++k) {
            if (!wait_bar(ptx::smem_addr(&t.full[r.stage]), r.phase, &t.abort_flag, p, 2 * 256 + r.stage))
                return false;
            ptx::tc_fence_after();
            if (EPI != kOut || k < h.ks) {
                const uint32_t sf = sf_tmem + r.stage * kSfSlot;
                const uint32_t cs = sbase + r.stage * p.stage_bytes + 2 * kWTile + p.x_bytes;
                ptx::tc_cp_32x128b_warpx4(sf, ptx::desc_sf_chunk(cs));
                if (o.has1) ptx::tc_cp_32x128b_warpx4(sf + 4, ptx::desc_sf_chunk(cs + 512));
                ptx::tc_cp_32x128b_warpx4(sf + 8, ptx::desc_sf_chunk(cs + 1024));
            }
            ptx::tc_commit(ptx::smem_addr(&t.sfr[r.stage]));
            r.next(p);
        }
    return true;
}

// Accumulator of the lt-th tile this CTA works on, and the parity of its use.
__device__ __forceinline__ int acc_of(const StreamParams &p, int lt, uint32_t &par) {
    par = (uint32_t)((p.nacc == 2 ? lt >> 1 : lt) & 1);
    return p.nacc == 2 ? (lt & 1) : 0;
}

template <int EPI>
__device__ __forceinline__ bool issue_mmas(const StreamParams &p, typename TailOf<EPI == kOut>::T &t, int ph,
                                           Ring &r, int &lt, uint32_t sbase, uint32_t tmem,
                                           uint32_t sf_tmem) {
    volatile int *abort_flag = &t.abort_flag;
    const StreamPhase &h = p.ph[ph];
    Walk w = walk_of<EPI == kOut>(p, t, ph);
    Tile o;
    for (; next_tile<EPI>(p, h, t, w, o); ++lt) {
        uint32_t par;
        const int acc = acc_of(p, lt, par);
        if (!wait_bar(ptx::smem_addr(&t.acce[acc]), par ^ 1u, abort_flag, p, 256 + 64 + acc)) return false;
        ptx::tc_fence_after();
        const uint32_t d0 = tmem + acc * 2 * p.nb, d1 = d0 + p.nb;
        const uint32_t n3 = (uint32_t)(o.n16 >> 3) << 17;
        const uint32_t id8 = ptx::idesc_mxf8(128, 0, 0) | n3 | p.w_fmt, id16 = ptx::idesc_bf16(128, 0) | n3;
        for (int k = o.k0; k < o.k1; ++k) {
            if (!wait_bar(ptx::smem_addr(&t.sfr[r.stage]), r.phase, abort_flag, p, 256 + r.stage))
                return false;
            ptx::tc_fence_after();
            const uint32_t s0 = sbase + r.stage * p.stage_bytes, x0 = s0 + 2 * kWTile;
            if (EPI != kOut || k < h.ks) {
                const uint32_t sf = sf_tmem + r.stage * kSfSlot;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t id = id8 | ((uint32_t)j << 4) | ((uint32_t)j << 29);
                    const uint32_t on = (k != o.k0 || j != 0) ? 1u : 0u;
                    const uint64_t dx = ptx::desc_kmajor_sw128(x0 + 32 * j);
                    ptx::mma_mxf8(d0, ptx::desc_kmajor_sw128(s0 + 32 * j), dx, id, sf, sf + 8, on);
                    if (o.has1)
                        ptx::mma_mxf8(d1, ptx::desc_kmajor_sw128(s0 + kWTile + 32 * j), dx, id, sf + 4, sf + 8,
                                      on);
                }
            } else {
                const int ls = k - h.ks, c = (ls - ls / p.kr * p.kr) * 64;
                const int nk = (min(64, p.rank - c) + 15) / 16;
                // the lo half: rows of its own, or columns 32-63
                const uint32_t lo = p.halves == 2 ? p.nb * 128 : 64;
                for (int j = 0; j < nk; ++j) {
                    const uint64_t dh = ptx::desc_kmajor_sw128(x0 + 32 * j);
                    const uint64_t dl = ptx::desc_kmajor_sw128(x0 + lo + 32 * j);
                    const uint64_t w0 = ptx::desc_kmajor_sw128(s0 + 32 * j);
                    const uint32_t on = (k != o.k0 || j != 0) ? 1u : 0u;
                    ptx::mma_bf16(d0, w0, dh, id16, on);
                    ptx::mma_bf16(d0, w0, dl, id16, 1u);
                    if (o.has1) {
                        const uint64_t w1 = ptx::desc_kmajor_sw128(s0 + kWTile + 32 * j);
                        ptx::mma_bf16(d1, w1, dh, id16, on);
                        ptx::mma_bf16(d1, w1, dl, id16, 1u);
                    }
                }
            }
            ptx::tc_commit(ptx::smem_addr(&t.empty[r.stage]));
            r.next(p);
        }
        ptx::tc_commit(ptx::smem_addr(&t.accf[acc]));
    }
    return true;
}

__device__ __forceinline__ float gate_act(float g, int gate) {
    if (gate == FP8G_GATE_SILU) return g / (1.0f + expf(-g));
    if (gate == FP8G_GATE_GELU) return 0.5f * g * (1.0f + erff(g * 0.70710678118654752f));
    return g < 0.0f ? 0.0f : g;
}

// 16 columns of a finished tile: v[s][i] is this lane's weight row f of weight
// tile s, token column c + i.
template <int EPI, int SUBS>
__device__ __forceinline__ void store_cols(const StreamParams &p, const StreamPhase &h, const Tile &o, int c,
                                           int f, int q, int lane, const float (&v)[SUBS][16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int col = c + i;
        if (col >= o.n) break;  // warp-uniform
        const int64_t at = (int64_t)(o.row0 + col) * h.rows + f;
        if constexpr (EPI == kGated) {
            // this warp's 32 features are one 1x32 block (rows is a multiple of 32)
            uint32_t code = 127u;  // blocks past the matrix: scale 1
            if (f < h.rows) {
                const float x = __fmul_rn(gate_act(v[0][i], p.gate), v[SUBS - 1][i]);
                const uint32_t mag = isnan(x) ? 0u : __float_as_uint(fabsf(x));
                const float s = pow2_scale<0>(__uint_as_float(__reduce_max_sync(0xffffffffu, mag)));
                p.hq[at] = (uint8_t)fp8x2<0>(__fmul_rn(x, __frcp_rn(s)), 0.0f);
                code = __float_as_uint(s) >> 23;
            }
            if (lane == 0)
                p.hsf[((int64_t)o.g * h.mt + o.mt) * 512 + 16 * (col & 31) + 4 * (col >> 5) + q] =
                    (uint8_t)code;
        } else if (f < h.rows) {
            if constexpr (EPI == kRows) {
                __stcg(p.y + at, v[0][i]);
            } else {
                const float x = p.bias != nullptr ? __fadd_rn(v[0][i], __ldg(p.bias + f)) : v[0][i];
                if (p.out_f32)
                    static_cast<float *>(p.out)[at] = x;
                else
                    static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(x);
            }
        }
    }
}

template <int EPI>
__device__ __forceinline__ bool epilogue(const StreamParams &p, typename TailOf<EPI == kOut>::T &t, int ph,
                                         int &lt, uint32_t tmem) {
    volatile int *abort_flag = &t.abort_flag;
    const StreamPhase &h = p.ph[ph];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int q = warp & 3, half = (warp - kSEpiWarp0) >> 2;
    const uint32_t tq = tmem + ((uint32_t)(q * 32) << 16);
    const int row_l = q * 32 + lane;  // weight row within a tile
    // two weight tiles: this warp takes tile `half`; gated, or one tile: every
    // other 16 columns (of both tiles, gated)
    constexpr int kSubs = EPI == kGated ? 2 : 1;
    const bool by_cols = EPI == kGated || h.sub == 1;
    const int c_first = by_cols ? half * 16 : 0, c_step = by_cols ? 32 : 16;
    const int my_sub = by_cols ? 0 : half;
    uint64_t *part_flags = p.flags + (int64_t)(kFlagPart + ph) * gridDim.x;
    const int64_t part_size = (int64_t)2 * p.nb * 128;
    Walk w = walk_of<EPI == kOut>(p, t, ph);
    Tile o;
    bool ok = true;
    for (; next_tile<EPI>(p, h, t, w, o); ++lt) {
        uint32_t par;
        const int acc = acc_of(p, lt, par);
        ok = ok && wait_bar_warp(ptx::smem_addr(&t.accf[acc]), par, abort_flag, p, 3 * 256 + acc, 32);
        if (!epi_all(ok)) return false;
        ptx::tc_fence_after();
        const bool live = my_sub == 0 || o.has1;  // this warp has a weight tile
        const uint32_t ta = tq + acc * 2 * p.nb;
        if (o.k0 != 0) {
            // not the tile's first units: the partial to its owner
            float *part = p.part + blockIdx.x * part_size;
            if (live)
                for (int c = c_first; c < o.n; c += c_step)
#pragma unroll
                    for (int s = 0; s < kSubs; ++s) {
                        const int sub = EPI == kGated ? s : my_sub;
                        uint32_t r[16];
                        ptx::tmem_ld_32x32b_x16(ta + sub * p.nb + c, r);
                        ptx::tmem_ld_wait();
                        float *dst = part + ((int64_t)sub * p.nb + c) * 128 + row_l;
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (c + i < o.n) __stcg(dst + i * 128, __uint_as_float(r[i]));
                    }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&t.acce[acc]));
            (void)epi_all(true);
            if (threadIdx.x == kSEpiWarp0 * 32) flag_set(part_flags + blockIdx.x, p.token);
            continue;
        }
        // the owner: the partials of the CTAs after it
        const int c_hi = o.k1 == o.upt ? (int)blockIdx.x : span_owner(w.U, w.G, o.u + o.upt - 1);
        if (c_hi > (int)blockIdx.x)
            ok = flags_wait(p, part_flags, blockIdx.x + 1, c_hi + 1, abort_flag, 5 * 256);
        if (live && ok)
            for (int c = c_first; c < o.n; c += c_step) {
                float v[kSubs][16];
#pragma unroll
                for (int s = 0; s < kSubs; ++s) {
                    const int sub = EPI == kGated ? s : my_sub;
                    uint32_t r[16];
                    ptx::tmem_ld_32x32b_x16(ta + sub * p.nb + c, r);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[s][i] = __uint_as_float(r[i]);
                    // in unit order; several CTAs' loads in flight at a time
                    for (int a = blockIdx.x + 1; a <= c_hi; a += kJoin) {
                        float x[kJoin][16];
#pragma unroll
                        for (int j = 0; j < kJoin; ++j) {
                            const float *src =
                                p.part + (a + j) * part_size + ((int64_t)sub * p.nb + c) * 128 + row_l;
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                x[j][i] = a + j <= c_hi && c + i < o.n ? __ldcg(src + i * 128) : 0.0f;
                        }
#pragma unroll
                        for (int j = 0; j < kJoin; ++j)
                            if (a + j <= c_hi)
#pragma unroll
                                for (int i = 0; i < 16; ++i) v[s][i] += x[j][i];
                    }
                }
                store_cols<EPI, kSubs>(p, h, o, c, (my_sub ? o.w1 : o.w0) + row_l, q, lane, v);
            }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&t.acce[acc]));
    }
    return epi_all(ok);
}

// out[t, h] = sum_j w[t, j] y[pos[t, j], h], j in order; four values a thread.
__device__ __forceinline__ void combine(const StreamParams &p) {
    const int H = p.ph[1].rows;
    const int64_t n = (int64_t)p.T * (H / 4);
    for (int64_t i = (int64_t)blockIdx.x * kEpiThreads + threadIdx.x - kSEpiWarp0 * 32; i < n;
         i += (int64_t)gridDim.x * kEpiThreads) {
        const int tok = (int)(i / (H / 4)), c = (int)(i - (int64_t)tok * (H / 4)) * 4;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int j = 0; j < p.k; ++j) {
            const int r = __ldcg(p.pos + tok * p.k + j);
            if (r < 0) continue;
            const float a = __ldg(p.weights + tok * p.k + j);
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(p.y + (int64_t)r * H + c));
            s.x = fmaf(a, v.x, s.x);
            s.y = fmaf(a, v.y, s.y);
            s.z = fmaf(a, v.z, s.z);
            s.w = fmaf(a, v.w, s.w);
        }
        const int64_t at = (int64_t)tok * H + c;
        if (p.out_f32)
            *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) = s;
        else
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + at) =
                make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
    }
}

template <bool LORA>
__global__ void __launch_bounds__(kSThreads, 1) stream_kernel(const __grid_constant__ StreamParams p) {
    using Tail = typename TailOf<LORA>::T;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = ptx::smem_addr(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (raw_base & 1023u)) & 1023u);
    const uint32_t sbase = ptx::smem_addr(smem);
    Tail &t = *reinterpret_cast<Tail *>(smem + p.stages * p.stage_bytes);
    volatile int *abort_flag = &t.abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kFirst = LORA ? kOut : kGated;

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
        for (int b = 0; b < kGates; ++b) {
            ptx::mbar_init(ptx::smem_addr(&t.gate[b]), 1);
            ptx::mbar_init(ptx::smem_addr(&t.arrived[b]), 1);
        }
        ptx::mbar_init(ptx::smem_addr(&t.drain), 1);
        ptx::mbar_init(ptx::smem_addr(&t.drain_sf), 1);
        t.abort_flag = 0;
        ptx::fence_mbar_init();
        // this CTA's flags but the first barrier's (which publishes this)
        for (int f = 1; f < kStreamFlags; ++f) p.flags[(int64_t)f * gridDim.x + blockIdx.x] = 0;
    }
    if (warp == 0 && lane == 0) {
        ptx::prefetch_tmap(&p.ph[0].W);
        ptx::prefetch_tmap(&p.ph[0].X);
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_addr(&t.tmem), 512);
        ptx::tmem_relinquish();
    }
    make_tables(p, t);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = t.tmem;
    const uint32_t sf_tmem = tmem + p.nacc * 2 * p.nb;

    if (warp == 0) {
        if (lane == 0) {
            Ring r;
            if (produce<kFirst>(p, t, 0, 0, r, sbase)) {
                if constexpr (!LORA) (void)produce<kRows>(p, t, 1, 1, r, sbase);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            Ring r;
            int lt = 0;
            if (issue_mmas<kFirst>(p, t, 0, r, lt, sbase, tmem, sf_tmem)) {
                if constexpr (!LORA) (void)issue_mmas<kRows>(p, t, 1, r, lt, sbase, tmem, sf_tmem);
            }
        }
    } else if (warp == 2) {
        if (lane == 0) {
            Ring r;
            if (copy_scales<kFirst>(p, t, 0, r, sbase, sf_tmem)) {
                if constexpr (!LORA) (void)copy_scales<kRows>(p, t, 1, r, sbase, sf_tmem);
            }
        }
    } else if (warp == 3) {
        // ===== watcher: opens gate b when every CTA has arrived at barrier b =====
        for (int b = 0; b < (LORA ? 2 : 3); ++b) {
            if (!wait_bar_warp(ptx::smem_addr(&t.arrived[b]), 0, abort_flag, p, 6 * 256 + b, 32)) break;
            if (!flags_wait(p, p.flags + (int64_t)b * gridDim.x, 0, gridDim.x, abort_flag, 6 * 256 + 16 + b))
                break;
            if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&t.gate[b]));
            // the second barrier passed: nobody looks at the first one's flags any more
            if (b == 1 && lane == 0) p.flags[blockIdx.x] = 0;
            __syncwarp();
        }
    } else {
        // ===== tokens, then epilogues =====
        auto gate = [&](int b) {
            return wait_bar_warp(ptx::smem_addr(&t.gate[b]), 0, abort_flag, p, 7 * 256 + b, 32);
        };
        int lt = 0;
        prepare(p, t);
        arrive(p, t, 0);
        if constexpr (LORA) {
            if (p.kr > 0) low_rank(p, t);
            if (epi_all(gate(0))) {
                arrive(p, t, 1);
                (void)epilogue<kOut>(p, t, 0, lt, tmem);
                (void)gate(1);
            }
        } else {
            if (epilogue<kGated>(p, t, 0, lt, tmem) && epi_all(gate(0))) {
                arrive(p, t, 1);
                if (epilogue<kRows>(p, t, 1, lt, tmem) && epi_all(gate(1))) {
                    arrive(p, t, 2);
                    if (epi_all(gate(2))) combine(p);
                }
            }
        }
    }

    __syncwarp();
    __syncthreads();
    if (*abort_flag) {
        // wait (bounded) for this CTA's MMAs, then give copies in flight a
        // bounded time before shared memory is released
        if (threadIdx.x == 0) p.flags[blockIdx.x] = 0;
        if ((warp == 1 || warp == 2) && lane == 0) {
            const uint32_t db = ptx::smem_addr(warp == 1 ? &t.drain : &t.drain_sf);
            ptx::tc_commit(db);
            const uint64_t t0 = ptx::globaltimer();
            while (!ptx::mbar_try_wait(db, 0) && ptx::globaltimer() - t0 < p.timeout_ns) {
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

template <bool LORA>
cudaError_t launch_one(const StreamParams &p, int grid, cudaStream_t s) {
    auto kern = stream_kernel<LORA>;
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
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kSThreads);
    // always more than half an SM's shared memory: one CTA per SM
    cfg.dynamicSmemBytes = (size_t)p.stages * p.stage_bytes + sizeof(typename TailOf<LORA>::T) + 1024;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

void stream_sizes(StreamParams &p, int nb, bool lora, int v_halves) {
    p.nb = nb;
    // two accumulators of two tiles each beside the scales, where they fit
    p.nacc = nb <= 64 ? 2 : 1;
    p.x_bytes = nb * 128 * v_halves;
    p.stage_bytes = 2 * kWTile + p.x_bytes + 2048;  // 1536 bytes of scales; 1024-byte multiples
    const int room = kSmemMax - 1024 - (int)(lora ? sizeof(TailLora) : sizeof(TailMoe));
    p.stages = room / p.stage_bytes;
    const int cols = (512 - p.nacc * 2 * nb) / kSfSlot;
    if (p.stages > cols) p.stages = cols;
    if (p.stages > kMaxStages) p.stages = kMaxStages;
}

size_t stream_part_bytes(const StreamParams &p, int grid) {
    return (size_t)grid * 2 * p.nb * 128 * sizeof(float);
}

size_t stream_flag_bytes(int grid) { return (size_t)kStreamFlags * grid * sizeof(uint64_t); }

uint64_t stream_token() {
    // odd multiples of a large odd constant: never 0, all different for 2^63 calls
    static std::atomic<uint64_t> calls{0};
    return (2 * calls.fetch_add(1, std::memory_order_relaxed) + 1) * 0x9E3779B97F4A7C15ull;
}

cudaError_t launch_stream(bool lora, const StreamParams &p, int grid, cudaStream_t s) {
    return lora ? launch_one<true>(p, grid, s) : launch_one<false>(p, grid, s);
}

}  // namespace fp8g
