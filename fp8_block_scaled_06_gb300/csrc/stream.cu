// Few tokens against block-scaled weights that are read once: the MoE layer
// (gate/up product, gated activation, down product, weighted sum) and the
// projection with low-rank adapters.  Two launches: one prepares the tokens
// (codes in the order of their experts or adapters), the other runs the products.
//
//   D[f, t] = sum_k (s W)[f, k] (s X)[t, k]
//
// The weights are the MMA's 128-row operand and the tokens its columns
// (tcgen05.mma kind::mxf8f6f4, M = 128, N = the group's tokens rounded up to
// 16): with few tokens a tile costs what its weights cost to load, and no CUDA
// core touches them.  A step is 128 K of a pair of 128-row weight tiles (32 KB:
// the gate and the up rows of the same features, or two neighbouring tiles).
//
// Tickets.  A ticket is a tile of a product (or a part of its K steps, where the
// tiles are too few to draw on all of HBM; about 100 SMs can).  One CTA per SM
// takes tickets off a counter in order: SMs that HBM serves better take more,
// and the counter is the whole schedule.  A part that is not the tile's last to
// finish leaves its fp32 sums in memory; the last one adds all parts in order,
// so results do not depend on which that is.
//
// The layer's two products share the line of tickets: all gate/up tiles by
// expert, then all down tiles by expert.  A down ticket's weights are loaded as
// soon as it is taken; only its tokens wait until the expert's gate/up tiles
// are done, which by then lie a whole product back in the line, so HBM is busy
// all along.  A wait is always for tickets taken earlier, by CTAs that are
// running, which in turn wait only for earlier ones: no CTA needs another one to
// be scheduled, whatever else the GPU runs.  Waits are bounded all the same.
//
// Adapters.  The epilogue warps first compute V = alpha A x (items off a counter,
// as the tickets), in two or three bf16 pieces.  After its FP8 steps a tile takes, per
// adapter among the group's tokens, bf16 steps (kind::f16) of the adapter's B
// rows against all pieces of V, into the same fp32 accumulator; a step covers
// the 16-column windows that hold the adapter's tokens (V is zero in the others'
// columns; lora_value.cuh has what follows for a B that is not finite).  B comes
// through the ring as the weights do: read through L1, of which 20 KB are left
// beside the ring, into registers for mma.sync, the same term took 128 rows of 32
// adapters of rank 64 from 48 to 66 us.
//
// Measured, per call on the device back to back, beside the bytes at 6.78 TB/s:
// one token, two experts of 4096 x 14336, 67 us (54); 5 tokens over 64 experts of
// 2080 x 1440, 60 (43); 16 tokens over 32 4-bit experts of 4096 x 2048, 72 (56);
// 64 tokens over 8 experts of 4096 x 14336, 227 (214).  While it streams it reads
// 6.6 to 7.1 TB/s; what is left is 6 us from the call before to the first weights
// in shared memory, the wait of the down product's first tokens, and 6 us from the
// last weights to the end.  Adapters: 33 rows at 4096 x 4096, rank 16, 18.5 us (3)
// with the weights in L2, 22.6 from memory; 128 rows of 32 adapters, rank 64, at 4096
// x 14336, 42 (21): 26 the projection (112 tiles, so 40 of 152 SMs have none; an SM
// takes in 58 GB/s, of which half are tokens), 3 V, 13 the 32 low-rank steps, of which
// 9 are the roles' own instructions a step (measured without the loads and MMAs).
//
// Roles: warp 0 takes tickets and loads weights, warp 3 the tokens' slices and
// the scales, warp 2 copies scales to tensor memory, warp 1 issues MMAs, warps
// 4-11 run the epilogues.  Two loading threads because a thread takes about
// 0.08 us to issue a copy, and a step has six.
#include <cuda_bf16.h>

#include <cstddef>
#include <type_traits>

#include "kernel_common.cuh"
#include "lora_pieces.cuh"
#include "lora_value.cuh"
#include "quant_math.cuh"
#include "stream.h"

namespace fp8g {

namespace {

constexpr int kSThreads = 384;
constexpr int kSEpiWarp0 = 4;
constexpr int kSEpiWarps = 8;
constexpr int kEpiThreads = kSEpiWarps * 32;
constexpr int kPrepThreads = 256;
constexpr int kPrepWarps = kPrepThreads / 32;
constexpr int kWTile = 128 * 128;  // bytes of a weight tile in shared memory
constexpr int kMaxStages = 16;
constexpr int kSfSlot = 16;        // tensor-memory columns of a stage's scales
// Steps of a part at least (33 rows at 1024 x 2048: 15.3 us, with parts of four 17.8).
constexpr int kMinSteps = 8;
constexpr int kCols = 8;           // token columns at a time in an epilogue (few: its code runs cold)
constexpr int kPairs = 256;        // pairs (token, expert) of a table of the weighted sum
constexpr int kTickets = 4;        // tickets in flight in a CTA
constexpr int kSmemMax = 232448;

enum Epi : int { kGated, kRows, kOut };

// ----------------------------------------------------------------- tables
// One group: up to nb token rows against one weight matrix.
struct Group {
    int16_t mat, row0, n, pad;
};
struct MoeTables {
    int32_t n_groups;
    Group g[kStreamMaxGroups];
    int32_t cnt[FP8G_MAX_ROUTED_EXPERTS];
};
struct LoraTables {
    int32_t n_groups;
    int32_t n[kStreamLoraGroups];  // slots
    int32_t windows[kStreamLoraGroups];  // windows of a slot's columns (Step)
    int32_t items;                       // of V, in all groups
    int16_t adapter[kStreamLoraGroups][kStreamMaxTokens];
    // a group's rows are taken in the order of their slots (those without an
    // adapter last): a slot's are columns first[s] .. first[s + 1] - 1
    int16_t first[kStreamLoraGroups][kStreamMaxTokens + 1];
    int16_t row_of[kStreamLoraRows];  // column -> row of the call
    union {
        alignas(16) uint32_t key[kStreamLoraRows];  // while the tables are made: lora_key
        float acc[4][16][17];  // products to join (V)
    };
};

__device__ __forceinline__ int warp_scan(int v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
    }
    return v;
}

// The groups, from the call's indices, by all threads of a block; ends with a
// barrier.
__device__ __forceinline__ void make_tables(const StreamParams &p, MoeTables &t) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (p.n_idx <= 32 && p.n_idx <= p.nb) {
        // one warp, a pair a lane: a block's barriers and shared-memory sums take
        // longer than everything else here
        if (warp == 0) {
            int e = lane < p.n_idx ? __ldg(p.idx + lane) : -1;
            if (e >= p.n_mat) e = -1;
            const uint32_t same = __match_any_sync(0xffffffffu, e);
            const bool first = e >= 0 && lane == __ffs((int)same) - 1;
            const uint32_t firsts = __ballot_sync(0xffffffffu, first);
            int row0 = 0, g = 0;  // rows and groups of smaller experts
            for (uint32_t m = firsts; m != 0; m &= m - 1) {
                const int o = __ffs((int)m) - 1;
                const int eo = __shfl_sync(0xffffffffu, e, o), c = __popc(__shfl_sync(0xffffffffu, same, o));
                if (eo < e) {
                    row0 += c;
                    ++g;
                }
            }
            if (first) t.g[g] = Group{(int16_t)e, (int16_t)row0, (int16_t)__popc(same), 0};
            if (lane == 0) t.n_groups = __popc(firsts);
        }
        __syncthreads();
        return;
    }
    for (int e = threadIdx.x; e < p.n_mat; e += blockDim.x) t.cnt[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < p.n_idx; i += blockDim.x) {
        const int e = __ldg(p.idx + i);
        if (e >= 0 && e < p.n_mat) atomicAdd(&t.cnt[e], 1);
    }
    __syncthreads();
    if (warp == 0) {
        int rr = 0, gg = 0;
        for (int e0 = 0; e0 < p.n_mat; e0 += 32) {
            const int e = e0 + lane;
            const int c = e < p.n_mat ? t.cnt[e] : 0, ng = (c + p.nb - 1) / p.nb;
            const int s = warp_scan(c, lane), sg = warp_scan(ng, lane);
            for (int i = 0; i < ng; ++i)
                t.g[gg + sg - ng + i] = Group{(int16_t)e, (int16_t)(rr + s - c + i * p.nb),
                                              (int16_t)min(p.nb, c - i * p.nb), 0};
            rr += __shfl_sync(0xffffffffu, s, 31);
            gg += __shfl_sync(0xffffffffu, sg, 31);
        }
        if (lane == 0) t.n_groups = gg;
    }
    __syncthreads();
}

// Rows in the order of their columns: by adapter (none: last), then by row.
__device__ __forceinline__ uint32_t lora_key(const StreamParams &p, int i) {
    const int l = p.rank > 0 ? __ldg(p.idx + i) : -1;
    return (uint32_t)(l < 0 || l >= p.n_mat ? FP8G_MAX_ADAPTERS : l) * kStreamLoraRows + i;
}

// A row's column is the number of smaller keys in its group (128 at most: counted
// by the row's thread; sorting in several steps with barriers took 3 us longer).
// Then a warp a group: a slot starts where the adapter changes.
__device__ __forceinline__ void make_tables(const StreamParams &p, LoraTables &t) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ng = (p.T + p.nb - 1) / p.nb;
    for (int i = threadIdx.x; i < ((p.T + 3) & ~3); i += (int)blockDim.x)
        t.key[i] = i < p.T ? lora_key(p, i) : 0xFFFFFFFFu;
    if (threadIdx.x == 0) {
        t.n_groups = ng;
        t.items = 0;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.T; i += (int)blockDim.x) {
        const int lo = i / p.nb * p.nb, hi = min(p.T, lo + p.nb);  // nb is a multiple of 16
        const uint32_t mine = t.key[i];
        int col = 0;
#pragma unroll 4
        for (int j = lo; j < hi; j += 4) {
            const uint4 k = *reinterpret_cast<const uint4 *>(t.key + j);
            col += (k.x < mine) + (k.y < mine) + (k.z < mine) + (k.w < mine);
        }
        t.row_of[lo + col] = (int16_t)i;
    }
    __syncthreads();
    if (warp < ng) {
        const int g = warp, lo = g * p.nb, n = min(p.nb, p.T - lo);
        int slots = 0, with = 0;  // slots, rows with an adapter
        uint32_t before = 0xFFFFFFFFu;  // adapter of the last column
        for (int c0 = 0; c0 < n; c0 += 32) {
            const int c = c0 + lane;
            const uint32_t l = c < n ? t.key[t.row_of[lo + c]] / kStreamLoraRows : FP8G_MAX_ADAPTERS;
            uint32_t prev = __shfl_up_sync(0xffffffffu, l, 1);
            if (lane == 0) prev = before;
            before = __shfl_sync(0xffffffffu, l, 31);
            const bool on = l < FP8G_MAX_ADAPTERS, first = on && l != prev;
            const uint32_t b = __ballot_sync(0xffffffffu, first);
            if (first) {
                const int s = slots + __popc(b & ((1u << lane) - 1u));
                t.adapter[g][s] = (int16_t)l;
                t.first[g][s] = (int16_t)c;
            }
            slots += __popc(b);
            with += __popc(__ballot_sync(0xffffffffu, on));
        }
        if (lane == 0) {
            t.n[g] = slots;
            t.first[g][slots] = (int16_t)with;
        }
        __syncwarp();
        int items = 0, most = 0;
        for (int s = lane; s < slots; s += 32) {
            const int from = t.first[g][s], to = t.first[g][s + 1];
            items += (to - from + 15) / 16;
            most = max(most, ((to + 15) & ~15) - (from & ~15));
        }
        most = __reduce_max_sync(0xffffffffu, most);
        items = __reduce_add_sync(0xffffffffu, items);
        if (lane == 0) {
            t.windows[g] = (max(most, 1) + p.v_cols - 1) / p.v_cols;
            atomicAdd(&t.items, items * ((p.rank + 15) / 16));
        }
    }
    __syncthreads();
}

// ----------------------------------------------------- preparing the tokens
// An item is a token and 2048 of its values, eight a thread (a 1x32 block is
// four threads).  Blocks past K in the last 128-wide step get scale 1.
__host__ __device__ inline int quant_segments(int ks) { return (ks * 16 + kPrepThreads - 1) / kPrepThreads; }

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

// Block (token, segment): the token's codes at its rows in expert order.
__global__ void __launch_bounds__(kPrepThreads) moe_prep_kernel(const __grid_constant__ StreamParams p) {
    __shared__ int32_t cnt[FP8G_MAX_ROUTED_EXPERTS];
    __shared__ int32_t row[FP8G_MAX_TOP_K], grp[FP8G_MAX_TOP_K], in[FP8G_MAX_TOP_K], any;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ks = p.ph[0].ks, segs = quant_segments(ks);
    const int tok = blockIdx.x / segs, seg = blockIdx.x - tok * segs, c = seg * kPrepThreads + tid;
    for (int e = tid; e < p.n_mat; e += kPrepThreads) cnt[e] = 0;
    if (tid == 0) any = 0;
    __syncthreads();
    ptx::grid_dep_wait();  // launched programmatically: global memory from here on
    ptx::grid_dep_launch();
    const int first = tid < p.n_idx ? __ldg(p.idx + tid) : -1;  // on the way beside the token
    const Quant8 q = quant_8(p, tok, c);
    for (int i = blockIdx.x * kPrepThreads + tid; i < p.n_counters; i += gridDim.x * kPrepThreads)
        p.counters[i] = 0;
    for (int i = tid; i < p.n_idx; i += kPrepThreads) {
        const int e = i == tid ? first : __ldg(p.idx + i);
        if (e >= p.n_mat && blockIdx.x == 0) record_error(p, FP8G_ERR_INVALID_ARG, (unsigned)i);
        if (e >= 0 && e < p.n_mat) {
            atomicAdd(&cnt[e], 1);
            any = 1;
        }
    }
    __syncthreads();
    // the token's rows: those of smaller experts, then the pairs before it of its own
    for (int j = warp; j < p.k; j += kPrepWarps) {
        const int i = tok * p.k + j;
        int e = __ldg(p.idx + i);
        if (e >= p.n_mat) e = -1;
        int before = 0, rows = 0, groups = 0;
        if (e >= 0) {
#pragma unroll 4
            for (int o = lane; o < i; o += 32) before += __ldg(p.idx + o) == e;
            for (int o = lane; o < e; o += 32) {
                rows += cnt[o];
                groups += (cnt[o] + p.nb - 1) / p.nb;
            }
        }
        before = __reduce_add_sync(0xffffffffu, before);
        rows = __reduce_add_sync(0xffffffffu, rows);
        groups = __reduce_add_sync(0xffffffffu, groups);
        if (lane == 0) {
            row[j] = e >= 0 ? rows + before : -1;
            grp[j] = groups + before / p.nb;
            in[j] = before % p.nb;
            if (seg == 0) p.pos[i] = row[j];
        }
    }
    __syncthreads();
    if (c < ks * 16)
        for (int j = 0; j < p.k; ++j) {
            if (row[j] < 0) continue;
            if (q.in) *reinterpret_cast<uint2 *>(p.xq + (int64_t)row[j] * p.K + c * 8) = q.q;
            if ((c & 3) == 0) p.xsf[sf_at(grp[j], ks, in[j], c)] = q.sf;
        }
    // no token has an expert: no tile will write the output
    if (!any && c * 8 < p.K) {
        const int64_t at = (int64_t)tok * p.K + c * 8;
        const uint4 z = make_uint4(0u, 0u, 0u, 0u);
        uint4 *d = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.out) + at * (p.out_f32 ? 4 : 2));
        d[0] = z;
        if (p.out_f32) d[1] = z;
    }
}

// Block (token, segment): the token's codes at its column.
__global__ void __launch_bounds__(kPrepThreads) lora_prep_kernel(const __grid_constant__ StreamParams p) {
    const int tid = threadIdx.x;
    const int ks = p.ph[0].ks, segs = quant_segments(ks);
    const int tok = blockIdx.x / segs, c = (blockIdx.x - tok * segs) * kPrepThreads + tid;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const Quant8 q = quant_8(p, tok, c);
    for (int i = blockIdx.x * kPrepThreads + tid; i < p.n_counters; i += gridDim.x * kPrepThreads)
        p.counters[i] = 0;
    if (c == 0 && p.kr > 0 && __ldg(p.idx + tok) >= p.n_mat) record_error(p, FP8G_ERR_INVALID_ARG, (unsigned)(p.first_row + tok));
    // the row's column: the smaller keys of its group
    const int g = tok / p.nb, j = g * p.nb + tid;
    const int col = __syncthreads_count(tid < p.nb && j < p.T && lora_key(p, j) < lora_key(p, tok));
    if (c >= ks * 16) return;
    if (q.in) *reinterpret_cast<uint2 *>(p.xq + ((int64_t)g * p.nb + col) * p.K + c * 8) = q.q;
    if ((c & 3) == 0) p.xsf[sf_at(g, ks, col, c)] = q.sf;
}

// ---------------------------------------------------------------- products
template <bool LORA>
struct TablesOf {
    using T = MoeTables;
};
template <>
struct TablesOf<true> {
    using T = LoraTables;
};

// Shared memory after the ring.
template <bool LORA>
struct Tail {
    uint64_t full[kMaxStages], empty[kMaxStages], sfr[kMaxStages], accf[2], acce[2], drain, drain_sf;
    uint64_t tk_full[kTickets], tk_empty[kTickets];
    int32_t ticket[kTickets];
    uint32_t tmem;
    int abort_flag;
    int last;
    int32_t parts[2], tickets[2];  // parts of a tile, tickets, per product
    int32_t pair_at[LORA ? 1 : kPairs];
    float pair_w[LORA ? 1 : kPairs];
    int32_t item, pick[4];  // item of V at hand
    uint32_t low[LORA ? kMaxStages : 1];  // a stage's low-rank step: first column, columns, MMAs of each piece
    typename TablesOf<LORA>::T tab;
};

static_assert(offsetof(LoraTables, key) % 16 == 0 && alignof(Tail<true>) % 16 == 0, "keys are read in fours");
static_assert(kSmemMax - 1024 - (int)(sizeof(Tail<false>) > sizeof(Tail<true>) ? sizeof(Tail<false>)
                                                                               : sizeof(Tail<true>)) >=
                  6 * (2 * kWTile + 16 * 128 + 2048),
              "six stages with 16 token columns");

// Parts of the tiles of a product: as many as give every SM a ticket at most.  (One
// token, two experts, down product of 32 tiles of 112 steps: 4 parts 67.3 us per
// call, 10 parts, two tickets an SM, 70.7.  64 tiles of 32 steps, adapters, one
// row at 4096 x 8192: 2 parts 17.3, unsplit 18.9.  64 tokens, 128 down tiles of 112
// steps: unsplit 227, 2 parts 249.)
__host__ __device__ inline int parts_of(int tiles, int ks, int num_sms) {
    if (tiles == 0 || tiles * 2 > num_sms || tiles > kStreamSplitTiles) return 1;
    const int most = ks / kMinSteps;
    return min(num_sms / tiles, most > 1 ? most : 1);
}

// What a ticket stands for: steps [k0, k1) of a tile, then (adapters) its low-rank
// steps [l0, l1).  Every part has its share of both (the low-rank ones all in the
// last part: 33 rows of 16 adapters at 4096 x 4096 21.7 us instead of 18.6); the
// FP8 steps start its accumulators.
struct Tile {
    int32_t ph, g, mt, part, tile;
    int32_t row0, n, n16;
    int32_t mat0, mat1, w0, w1;  // matrix and first row of the two weight tiles
    bool has1;                   // the second one exists
    int32_t k0, k1, l0, l1;
};

template <bool LORA>
__device__ __forceinline__ bool decode(const StreamParams &p, const Tail<LORA> &t, int ticket, Tile &o) {
    o.ph = !LORA && ticket >= t.tickets[0];
    if (o.ph) ticket -= t.tickets[0];
    if (ticket >= t.tickets[o.ph]) return false;
    const StreamPhase &h = p.ph[o.ph];
    const int parts = t.parts[o.ph];
    o.tile = ticket / parts;
    o.part = ticket - o.tile * parts;
    o.g = o.tile / h.mt;
    o.mt = o.tile - o.g * h.mt;
    o.k0 = h.ks * o.part / parts;
    o.k1 = h.ks * (o.part + 1) / parts;
    o.l0 = o.l1 = 0;
    if constexpr (LORA) {
        const int low = t.tab.n[o.g] * p.kr * t.tab.windows[o.g];
        o.l0 = low * o.part / parts;
        o.l1 = low * (o.part + 1) / parts;
        o.row0 = o.g * p.nb;
        o.n = min(p.nb, p.T - o.row0);
        o.mat0 = 0;
    } else {
        const Group gr = t.tab.g[o.g];
        o.row0 = gr.row0;
        o.n = gr.n;
        o.mat0 = o.ph ? gr.mat : 2 * gr.mat;
    }
    o.n16 = (o.n + 15) & ~15;
    if (!LORA && o.ph == 0) {
        o.mat1 = o.mat0 + 1;
        o.w0 = o.w1 = o.mt * 128;
        o.has1 = true;
    } else {
        o.mat1 = o.mat0;
        o.w0 = o.mt * 128 * h.sub;
        o.w1 = o.w0 + 128;
        o.has1 = h.sub == 2 && o.w1 < h.rows;
    }
    return true;
}

// A low-rank step: a slot's 64 ranks from c on for n token columns from lo on, the
// 16-column windows of the slot's rows (of up to v_cols columns where V's pieces
// take rows of their own; V is zero in the others' columns).
struct Step {
    int slot, c, lo, n;
    bool none;  // the slot has no rows in this window
};
// A role's way through a tile's low-rank steps: windows in rank blocks in slots.
struct LowRank {
    int slot = 0, c = 0, w = 0;
    __device__ __forceinline__ void next(const StreamParams &p, int nw) {
        if (++w < nw) return;
        w = 0;
        if (++c < p.kr) return;
        c = 0;
        ++slot;
    }
    template <bool LORA>
    __device__ __forceinline__ void start(const StreamParams &p, const Tail<LORA> &t, const Tile &o) {
        if constexpr (LORA) {
            // (divisions take longer than a step's MMAs: once a tile)
            const int nw = t.tab.windows[o.g], per = p.kr * nw;
            slot = o.l0 / per;
            c = (o.l0 - slot * per) / nw;
            w = o.l0 - slot * per - c * nw;
        }
    }
};
__device__ __forceinline__ Step step_of(const StreamParams &p, const LoraTables &t, const Tile &o, LowRank &q) {
    const int lo = t.first[o.g][q.slot] & ~15, hi = (t.first[o.g][q.slot + 1] + 15) & ~15;
    Step s{q.slot, q.c * 64, lo, hi - lo, false};
    if (p.v_cols < p.nb) {
        const int from = lo + q.w * p.v_cols;
        s.none = from >= hi;
        s.lo = s.none ? lo : from;
        s.n = s.none ? 16 : min(p.v_cols, hi - from);
    }
    q.next(p, t.windows[o.g]);
    return s;
}

// The ring's position, and the ticket queue's.
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
struct Queue {
    int i = 0;
    __device__ __forceinline__ int slot() const { return i % kTickets; }
    __device__ __forceinline__ uint32_t phase() const { return (uint32_t)(i / kTickets) & 1u; }
};

// The next ticket's tile, for one thread (WARP: a whole warp); false: none, or
// aborting.
template <bool LORA, bool WARP>
__device__ __forceinline__ bool take(const StreamParams &p, Tail<LORA> &t, Queue &q, Tile &o, unsigned who) {
    const uint32_t bar = ptx::smem_addr(&t.tk_full[q.slot()]);
    if (!(WARP ? wait_bar_warp(bar, q.phase(), &t.abort_flag, p, who * 256 + 200, 32)
               : wait_bar(bar, q.phase(), &t.abort_flag, p, who * 256 + 200)))
        return false;
    const int ticket = *reinterpret_cast<volatile int32_t *>(&t.ticket[q.slot()]);
    if (WARP) __syncwarp();
    if (!WARP || (threadIdx.x & 31) == 0) ptx::mbar_arrive(ptx::smem_addr(&t.tk_empty[q.slot()]));
    ++q.i;
    return decode(p, t, ticket, o);
}

__device__ __forceinline__ int atom_add_acq_rel(int32_t *a, int v) {
    int old;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(old) : "l"(a), "r"(v) : "memory");
    return old;
}
__device__ __forceinline__ int ld_acquire(const int32_t *a) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(a) : "memory");
    return v;
}
// Between ordinary stores and TMA loads of the same memory (on both sides of
// the counter that orders them).
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

// Until *counter is n (one thread).  Bounded; false: aborting.
template <bool LORA>
__device__ __forceinline__ bool wait_count(const StreamParams &p, Tail<LORA> &t, const int32_t *counter, int n) {
    volatile int *abort_flag = &t.abort_flag;
    const uint64_t t0 = ptx::globaltimer();
    while (ld_acquire(counter) != n) {
        if (*abort_flag) return false;
        if (ptx::globaltimer() - t0 > p.timeout_ns) {
            *abort_flag = 1;
            record_error(p, FP8G_ERR_TIMEOUT, 4 * 256 + 100);
            return false;
        }
    }
    return true;
}

// Warp 0: tickets and weight tiles (or an adapter's rows).
template <bool LORA>
__device__ __forceinline__ void load_weights(const StreamParams &p, Tail<LORA> &t, uint32_t sbase) {
    volatile int *abort_flag = &t.abort_flag;
    const uint32_t w_tx = kWTile - kWTile / 8 * p.gap8;
    Ring r;
    Queue q;
    int next = atomicAdd(p.counters, 1);
    while (true) {
        const int ticket = next;
        if (!wait_bar(ptx::smem_addr(&t.tk_empty[q.slot()]), q.phase() ^ 1u, abort_flag, p, 201)) return;
        *reinterpret_cast<volatile int32_t *>(&t.ticket[q.slot()]) = ticket;
        ptx::mbar_arrive(ptx::smem_addr(&t.tk_full[q.slot()]));
        ++q.i;
        Tile o;
        if (!decode(p, t, ticket, o)) return;
        const StreamPhase &h = p.ph[o.ph];
        // the next ticket: late enough that a CTA does not hold a tile others could
        // start, early enough that the answer is there when this tile's loads are out
        const int steps = o.k1 - o.k0 + o.l1 - o.l0, ask = max(0, steps - 2);
        for (int k = o.k0; k < o.k1; ++k) {
            if (k - o.k0 == ask) next = atomicAdd(p.counters, 1);
            if (!wait_bar(ptx::smem_addr(&t.empty[r.stage]), r.phase ^ 1u, abort_flag, p, r.stage)) return;
            const uint32_t fb = ptx::smem_addr(&t.full[r.stage]), s0 = sbase + r.stage * p.stage_bytes;
            ptx::mbar_arrive_expect_tx(fb, o.has1 ? 2 * w_tx : w_tx);
            ptx::tma_load_3d(s0, &h.W, fb, k * kBK, o.w0, o.mat0);
            if (o.has1) ptx::tma_load_3d(s0 + kWTile, &h.W, fb, k * kBK, o.w1, o.mat1);
            r.next(p);
        }
        if constexpr (LORA) {
            LowRank low;
            if (o.l0 < o.l1) low.start(p, t, o);
            for (int l = o.l0; l < o.l1; ++l) {
                if (o.k1 - o.k0 + l - o.l0 == ask) next = atomicAdd(p.counters, 1);
                const Step st = step_of(p, t.tab, o, low);
                const int adapter = t.tab.adapter[o.g][st.slot];
                if (!wait_bar(ptx::smem_addr(&t.empty[r.stage]), r.phase ^ 1u, abort_flag, p, r.stage)) return;
                const uint32_t fb = ptx::smem_addr(&t.full[r.stage]), s0 = sbase + r.stage * p.stage_bytes;
                ptx::mbar_arrive_expect_tx(fb, o.has1 ? 2 * kWTile : kWTile);
                ptx::tma_load_3d(s0, &p.B, fb, st.c, o.w0, adapter);
                if (o.has1) ptx::tma_load_3d(s0 + kWTile, &p.B, fb, st.c, o.w1, adapter);
                r.next(p);
            }
        }
    }
}

// Warp 3: the tokens' slices (or V's), and all scale chunks (tokens', first
// weight tile's, second's).  A down product's tokens wait for the gate/up tiles
// of their group.  P: pieces of V.
template <bool LORA, int P>
__device__ __forceinline__ void load_tokens(const StreamParams &p, Tail<LORA> &t, uint32_t sbase) {
    volatile int *abort_flag = &t.abort_flag;
    Ring r;
    Queue q;
    Tile o;
    int ready = -1;  // groups up to this one are known to be done
    bool v_done = false;
    while (take<LORA, false>(p, t, q, o, 4)) {
        const StreamPhase &h = p.ph[o.ph];
        if (o.ph == 1 && o.g > ready) {
            if (!wait_count(p, t, p.done_group + o.g, p.ph[0].mt)) return;
            fence_proxy_async_all();
            ready = o.g;
        }
        const int64_t step = (int64_t)h.n_rt * 512;
        const uint8_t *c0 = h.sfw + (int64_t)o.mat0 * h.ks * step + o.w0 / 128 * 512;
        const uint8_t *c1 = h.sfw + (int64_t)o.mat1 * h.ks * step + o.w1 / 128 * 512;
        const bool pair = o.has1 && c1 == c0 + 512;
        const uint8_t *cx = h.sfx + (int64_t)o.g * h.ks * 512;
        // boxes of 64 rows, or of 16 where few are wanted (a box may reach past
        // the group's rows, but not past the nb rows that a stage has room for)
        const int box = o.n16 > 32 && p.nb % 64 == 0 ? 64 : 16, boxes = (o.n16 + box - 1) / box;
        const CUtensorMap *map = box == 64 ? &h.X64 : &h.X;
        for (int k = o.k0; k < o.k1; ++k) {
            if (!wait_bar(ptx::smem_addr(&t.empty[r.stage]), r.phase ^ 1u, abort_flag, p, 4 * 256 + r.stage))
                return;
            const uint32_t fb = ptx::smem_addr(&t.full[r.stage]);
            const uint32_t x0 = sbase + r.stage * p.stage_bytes + p.w_bytes, sf = x0 + p.x_bytes;
            ptx::mbar_arrive_expect_tx(fb, boxes * box * 128u + (o.has1 ? 1536u : 1024u));
            for (int i = 0; i < boxes; ++i)
                ptx::tma_load_2d(x0 + i * box * 128, map, fb, k * kBK, o.row0 + i * box);
            ptx::bulk_load(sf, cx + (int64_t)k * 512, 512, fb);
            ptx::bulk_load(sf + 512, c0 + k * step, pair ? 1024 : 512, fb);
            if (o.has1 && !pair) ptx::bulk_load(sf + 1024, c1 + k * step, 512, fb);
            r.next(p);
        }
        if constexpr (LORA) {
            LowRank low;
            if (o.l0 < o.l1) {
                low.start(p, t, o);
                if (!v_done) {  // every item of V
                    if (!wait_count(p, t, p.counters + 2, t.tab.items)) return;
                    fence_proxy_async_all();
                    v_done = true;
                }
            }
            for (int l = o.l0; l < o.l1; ++l) {
                const Step st = step_of(p, t.tab, o, low);
                if (!wait_bar(ptx::smem_addr(&t.empty[r.stage]), r.phase ^ 1u, abort_flag, p, 4 * 256 + r.stage))
                    return;
                const uint32_t fb = ptx::smem_addr(&t.full[r.stage]);
                const uint32_t x0 = sbase + r.stage * p.stage_bytes + p.w_bytes;
                t.low[r.stage] = (uint32_t)(st.lo | st.n << 8 |
                                            (st.none ? 0 : (min(64, p.rank - st.c) + 15) / 16) << 16);
                const int v0 = (o.g * p.slot_cap + st.slot) * p.blocks;
                ptx::mbar_arrive_expect_tx(fb, p.blocks * st.n * 128u);
                if (st.n == 16)
                    ptx::tma_load_3d(x0, &p.V, fb, st.c, st.lo, v0);
                else if (P == 3 && st.n == 32 && p.blocks > 1)
                    ptx::tma_load_3d(x0, &p.V32, fb, st.c, st.lo, v0);
                else
                    for (int b = 0; b < p.blocks; ++b)
                        for (int i = 0; i < st.n; i += 16)
                            ptx::tma_load_3d(x0 + (b * st.n + i) * 128, &p.V1, fb, st.c, st.lo + i, v0 + b);
                r.next(p);
            }
        }
    }
}

// Warp 2.  From a thread of their own: issued by the MMA thread each copy holds
// up the MMAs behind it.  A stage's columns are rewritten only after its next
// "full", when the MMAs that read them are done.
template <bool LORA>
__device__ __forceinline__ void copy_scales(const StreamParams &p, Tail<LORA> &t, uint32_t sbase,
                                            uint32_t sf_tmem) {
    Ring r;
    Queue q;
    Tile o;
    while (take<LORA, false>(p, t, q, o, 2))
        for (int i = o.l0 - o.l1 + o.k0 - o.k1, low = o.l0 - o.l1; i < 0; ++i) {
            if (!wait_bar(ptx::smem_addr(&t.full[r.stage]), r.phase, &t.abort_flag, p, 2 * 256 + r.stage))
                return;
            ptx::tc_fence_after();
            if (!LORA || i < low) {
                const uint32_t sf = sf_tmem + r.stage * kSfSlot;
                const uint32_t cs = sbase + r.stage * p.stage_bytes + p.w_bytes + p.x_bytes;
                ptx::tc_cp_32x128b_warpx4(sf, ptx::desc_sf_chunk(cs + 512));
                if (o.has1) ptx::tc_cp_32x128b_warpx4(sf + 4, ptx::desc_sf_chunk(cs + 1024));
                ptx::tc_cp_32x128b_warpx4(sf + 8, ptx::desc_sf_chunk(cs));
            }
            ptx::tc_commit(ptx::smem_addr(&t.sfr[r.stage]));
            r.next(p);
        }
}

// Accumulator of the lt-th tile this CTA works on, and the parity of its use.
__device__ __forceinline__ int acc_of(const StreamParams &p, int lt, uint32_t &par) {
    par = (uint32_t)((p.nacc == 2 ? lt >> 1 : lt) & 1);
    return p.nacc == 2 ? (lt & 1) : 0;
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// Warp 1.  The whole warp goes through the loop and one lane issues: operands
// that the compiler knows to be the same in all lanes are in uniform registers
// already (from a branch for lane 0 alone a step's eight MMAs took 0.4 us to
// issue, more than 4-bit weights take to load).  MMAs into one accumulator follow
// each other at about 140 cycles however few their columns, so a tile has two
// where tensor memory allows (chains): MMAs alternate and the epilogue adds them.
template <bool LORA, int P>
__device__ __forceinline__ void issue_mmas(const StreamParams &p, Tail<LORA> &t, uint32_t sbase, uint32_t tmem,
                                           uint32_t sf_tmem) {
    volatile int *abort_flag = &t.abort_flag;
    Ring r;
    Queue q;
    Tile o;
    // matrix descriptors of stage 0; a stage on: stage16 more
    const uint64_t w_desc = ptx::desc_kmajor_sw128(sbase), x_desc = ptx::desc_kmajor_sw128(sbase + p.w_bytes);
    const uint32_t stage16 = (uint32_t)p.stage_bytes >> 4, tile16 = kWTile >> 4;
    const uint32_t tile_cols = p.chains * p.nb, odd = p.chains == 2 ? p.nb : 0;
    auto wait = [&](uint64_t *bar, uint32_t phase, unsigned detail) {
        const uint32_t b = ptx::smem_addr(bar);
        if (__all_sync(0xffffffffu, ptx::mbar_try_wait(b, phase))) return true;
        return wait_bar_warp(b, phase, abort_flag, p, detail);
    };
    for (int lt = 0; take<LORA, true>(p, t, q, o, 1); ++lt) {
        uint32_t par;
        const int acc = acc_of(p, lt, par);
        if (!wait(&t.acce[acc], par ^ 1u, 256 + 64 + acc)) return;
        ptx::tc_fence_after();
        const int k0 = uniform(o.k0), k1 = uniform(o.k1), n16 = uniform(o.n16);
        const bool has1 = uniform(o.has1) != 0;
        const uint32_t d0 = tmem + acc * p.acc_cols, d1 = d0 + tile_cols;
        const uint32_t id8 = ptx::idesc_mxf8(128, 0, 0) | (uint32_t)(n16 >> 3) << 17 | p.w_fmt;
        for (int k = k0; k < k1; ++k) {
            if (!wait(&t.sfr[r.stage], r.phase, 256 + r.stage)) return;
            ptx::tc_fence_after();
            const uint32_t at = r.stage * stage16;
            const uint32_t first = k == k0 ? 0u : 1u;
            const uint32_t sf = sf_tmem + r.stage * kSfSlot;
            if (elect_one()) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t id = id8 | ((uint32_t)j << 4) | ((uint32_t)j << 29);
                    const uint32_t on = j < p.chains ? first : 1u, c = (j & 1) ? odd : 0;
                    ptx::mma_mxf8(d0 + c, w_desc + at + 2 * j, x_desc + at + 2 * j, id, sf, sf + 8, on);
                    if (has1)
                        ptx::mma_mxf8(d1 + c, w_desc + at + tile16 + 2 * j, x_desc + at + 2 * j, id, sf + 4,
                                      sf + 8, on);
                }
            }
            if (elect_one()) ptx::tc_commit(ptx::smem_addr(&t.empty[r.stage]));
            __syncwarp();
            r.next(p);
        }
        if constexpr (LORA) {
            for (int l = uniform(o.l1 - o.l0); l > 0; --l) {
                if (!wait(&t.sfr[r.stage], r.phase, 256 + r.stage)) return;
                ptx::tc_fence_after();
                const int all = uniform((int)t.low[r.stage]);
                const int lo = all & 255, n = all >> 8 & 255, nk = all >> 16;
                const uint32_t id16 = ptx::idesc_bf16(128, 0) | (uint32_t)(n >> 3) << 17;
                const uint32_t at = r.stage * stage16;
                // pieces (LoraV), the second one into the second accumulator
                const uint64_t x0 = x_desc + at;
                const uint64_t x1 = x0 + (P == 3 && p.per == 3 ? 2 : p.per == 2 ? 4 : n * 8);
                const uint64_t x2 = x0 + (p.per == 3 ? 4 : p.per == 2 ? n * 8 : 2 * n * 8);
                const uint32_t da = d0 + lo, db = da + odd;
                if (elect_one()) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (j >= nk) break;
                        const uint64_t w0 = w_desc + at + 2 * j, w1 = w0 + tile16;
                        ptx::mma_bf16(da, w0, x0 + 2 * j, id16, 1u);
                        if (has1) ptx::mma_bf16(da + tile_cols, w1, x0 + 2 * j, id16, 1u);
                        ptx::mma_bf16(db, w0, x1 + 2 * j, id16, 1u);
                        if (has1) ptx::mma_bf16(db + tile_cols, w1, x1 + 2 * j, id16, 1u);
                        if (P == 2) continue;
                        ptx::mma_bf16(da, w0, x2 + 2 * j, id16, 1u);
                        if (has1) ptx::mma_bf16(da + tile_cols, w1, x2 + 2 * j, id16, 1u);
                    }
                }
                if (elect_one()) ptx::tc_commit(ptx::smem_addr(&t.empty[r.stage]));
                __syncwarp();
                r.next(p);
            }
        }
        if (elect_one()) ptx::tc_commit(ptx::smem_addr(&t.accf[acc]));
        __syncwarp();
    }
}

// ---------------------------------------------------------------- epilogue
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

// All epilogue warps: after this CTA's stores, add 1 to *counter; whether that
// made it `full`.  What the others stored before their additions can then be read.
template <bool LORA>
__device__ __forceinline__ bool count_in(Tail<LORA> &t, int32_t *counter, int full) {
    (void)epi_all(true);
    if (threadIdx.x == kSEpiWarp0 * 32) t.last = atom_add_acq_rel(counter, 1) + 1 == full;
    (void)epi_all(true);
    return t.last != 0;
}

// ------------------------------------------------------------ V = alpha A x
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&b);
}
// An item is up to 16 rows of a slot against 16 ranks of its adapter; the K range
// goes over the eight warps, each a 16 x 16 product by mma.sync (ranks x rows),
// joined in warp order.  A lane's 16-byte load covers 8 consecutive K of a row;
// the same K permutation on both operands leaves the product as it is.  kU K
// steps of 32 are on the way in a warp.  With two warps to a scheduler what
// bounds this, next to the loads' latency (an adapter's 16 ranks are 131 KB at
// K = 4096), is the number of instructions: rows and ranks past the end read
// others' values, into products that are not stored, and no load has a condition.
// FEW: eight rows at most.
template <int P, bool BF16, bool FEW>
__device__ __forceinline__ void low_rank_item(const StreamParams &p, LoraTables &t, const int32_t *pick) {
    const int tid = threadIdx.x - kSEpiWarp0 * 32, warp = tid >> 5, lane = tid & 31;
    const int g = pick[0], slot = pick[1], l = t.adapter[g][slot], rb = pick[3];
    const int col0 = t.first[g][slot] + pick[2], n = min(16, t.first[g][slot + 1] - col0);  // this item's columns
    __nv_bfloat16 *hi = static_cast<__nv_bfloat16 *>(p.v) +
                        (int64_t)(g * p.slot_cap + slot) * p.blocks * p.nb * p.r64 + rb * 16;
    const int64_t block = (int64_t)p.nb * p.r64;
    if (pick[2] == 0) {
        // the slot's first rows: zeros for the tokens of other adapters, and
        // in the columns past the rank
        const int rblocks = (p.rank + 15) / 16, all = p.per == 1 ? p.r64 / 16 : p.per == 2 ? 2 : 1;
        const int s_lo = t.first[g][slot], s_hi = t.first[g][slot + 1];
        for (int i = tid; i < p.nb; i += kEpiThreads) {
            __nv_bfloat16 *d = hi + (int64_t)i * p.r64;
            if (i < s_lo || i >= s_hi) zero_v<P>(d, 1, p.per, block);
            if (rb == 0) zero_v<P>(d + 16 * rblocks, all - rblocks, p.per, block);
        }
    }
    const int gr = lane >> 2, c8 = 8 * (lane & 3);
    const int64_t lo = (int64_t)g * p.nb + col0;
    const int64_t x0 = (int64_t)t.row_of[lo + min(gr, n - 1)] * p.K + c8;
    const int64_t x1 = (int64_t)t.row_of[lo + min(gr + 8, n - 1)] * p.K + c8;
    const int r0 = min(rb * 16 + gr, p.rank - 1), r1 = min(rb * 16 + gr + 8, p.rank - 1);
    const __nv_bfloat16 *A = static_cast<const __nv_bfloat16 *>(p.a) + (int64_t)l * p.rank * p.K + c8;
    const __nv_bfloat16 *a0 = A + (int64_t)r0 * p.K, *a1 = A + (int64_t)r1 * p.K;
    float d0[4] = {}, d1[4] = {};  // rows 0-7, 8-15
    constexpr int kU = BF16 ? (FEW ? 6 : 4) : 2;
    auto go = [&](auto count, int s0) {
        constexpr int U = decltype(count)::value;
        uint4 wa[U], wb[U];
        X8<BF16> xa[U];
        [[maybe_unused]] X8<BF16> xb[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (s0 + u) * 32;
            wa[u] = __ldg(reinterpret_cast<const uint4 *>(a0 + k));
            wb[u] = __ldg(reinterpret_cast<const uint4 *>(a1 + k));
            xa[u].load(p.x, x0 + k);
            if constexpr (!FEW) xb[u].load(p.x, x1 + k);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t f0[4] = {wa[u].x, wb[u].x, wa[u].y, wb[u].y};
            const uint32_t f1[4] = {wa[u].z, wb[u].z, wa[u].w, wb[u].w};
#pragma unroll
            for (int i = 0; i < X8<BF16>::kMost; ++i) {
                if (i == P) break;
                const uint4 x = xa[u].template next<P>();
                mma_16816(d0, f0, x.x, x.y);
                mma_16816(d0, f1, x.z, x.w);
                if constexpr (!FEW) {
                    const uint4 y = xb[u].template next<P>();
                    mma_16816(d1, f0, y.x, y.y);
                    mma_16816(d1, f1, y.z, y.w);
                }
            }
        }
    };
    const int steps = p.K / 32;  // K is a multiple of 32
    int s0 = warp * kU;
    for (; s0 + kU <= steps; s0 += kSEpiWarps * kU) go(std::integral_constant<int, kU>{}, s0);
#pragma unroll 1
    for (; s0 < steps; ++s0) go(std::integral_constant<int, 1>{}, s0);
    // the warps' products: warp w + 4 to warp w, then the four in order
    const int c2 = 2 * (lane & 3);
    float(*acc)[17] = t.acc[warp & 3];  // [row][rank]
    if (warp >= 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            acc[c2 + (e & 1)][gr + 8 * (e >> 1)] = d0[e];
            if constexpr (!FEW) acc[8 + c2 + (e & 1)][gr + 8 * (e >> 1)] = d1[e];
        }
    }
    (void)epi_all(true);
    if (warp < 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            acc[c2 + (e & 1)][gr + 8 * (e >> 1)] += d0[e];
            if constexpr (!FEW) acc[8 + c2 + (e & 1)][gr + 8 * (e >> 1)] += d1[e];
        }
    }
    (void)epi_all(true);
    const int i = tid >> 4, c = tid & 15;
    float v = 0.0f;
#pragma unroll
    for (int q = 0; q < kSEpiWarps / 2; ++q) v += t.acc[q][i][c];
    if (p.alpha != nullptr) v *= __ldg(p.alpha + l);
    if (rb * 16 + c >= p.rank) v = 0.0f;
    if (i < n) store_v<P>(hi + (int64_t)(col0 + i) * p.r64 + c, v, p.per, block);
}

template <int P>
__device__ __forceinline__ void low_rank(const StreamParams &p, LoraTables &t, int32_t *pick, int item) {
    const int rblocks = (p.rank + 15) / 16;
    if ((threadIdx.x >> 5) == kSEpiWarp0) {
        // item -> group, slot, 16 rows, rank block
        const int lane = threadIdx.x & 31;
        int at = 0;
        for (int g = 0; g < t.n_groups; ++g)
            for (int s0 = 0; s0 < t.n[g]; s0 += 32) {
                const int s = s0 + lane;
                const int c = s < t.n[g] ? (t.first[g][s + 1] - t.first[g][s] + 15) / 16 * rblocks : 0;
                const int incl = warp_scan(c, lane), first = at + incl - c;
                if (item >= first && item < first + c) {
                    pick[0] = g;
                    pick[1] = s;
                    pick[2] = (item - first) / rblocks * 16;
                    pick[3] = (item - first) % rblocks;
                }
                at += __shfl_sync(0xffffffffu, incl, 31);
            }
    }
    (void)epi_all(true);
    const int left = t.first[pick[0]][pick[1] + 1] - t.first[pick[0]][pick[1]] - pick[2];
    if (!p.x_bf16)
        low_rank_item<P, false, false>(p, t, pick);
    else if (left <= 8)
        low_rank_item<P, true, true>(p, t, pick);
    else
        low_rank_item<P, true, false>(p, t, pick);
}

__device__ __forceinline__ float gate_act(float g, int gate) {
    if (gate == FP8G_GATE_SILU) return g / (1.0f + expf(-g));
    if (gate == FP8G_GATE_GELU) return 0.5f * g * (1.0f + erff(g * 0.70710678118654752f));
    return g < 0.0f ? 0.0f : g;
}

// kCols columns of a finished tile: v[s][i] is this lane's weight row f of weight
// tile s, token column c + i.  (Plain stores go on with all columns and leave out
// those past the group, so that their latencies overlap; the layer's, mostly of
// a column or two, end at the last one.)  spoilt (kOut): set where an
// adapter's B is not finite: no value of its windows is then, so the first of the
// kCols columns tells (a comparison for each took 512 rows from 112.0 to 114.8 us).
template <bool LORA, int EPI, int SUBS>
__device__ __forceinline__ void store_cols(const StreamParams &p, const StreamPhase &h, const Tail<LORA> &t,
                                           const Tile &o, int c, int c_hi, int f, int q, int lane, float bias,
                                           const float (&v)[SUBS][kCols], bool &spoilt) {
    if constexpr (EPI != kOut) {
#pragma unroll
        for (int i = 0; i < kCols; ++i) {
            const int col = c + i;
            if (col >= c_hi) break;  // warp-uniform
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
                __stcg(p.y + at, v[0][i]);
            }
        }
    } else {
        spoilt |= !isfinite(v[0][0]);
        int row[kCols];
#pragma unroll
        for (int i = 0; i < kCols; ++i) row[i] = c + i < c_hi ? t.tab.row_of[o.row0 + c + i] : 0;
#pragma unroll
        for (int i = 0; i < kCols; ++i) {
            const int64_t at = (int64_t)row[i] * h.rows + f;
            const float x = p.bias != nullptr ? __fadd_rn(v[0][i], bias) : v[0][i];
            if (f >= h.rows || c + i >= c_hi) continue;
            if (p.out_f32)
                static_cast<float *>(p.out)[at] = x;
            else
                static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(x);
        }
    }
}

// The NaN among a warp's values of a tile, lane: feature f, computed again
// (lora_value.cuh); columns as finish_tile takes them.  (Arguments by value: a Tile
// by reference would live in memory, 0.5 us a call.)
__device__ __noinline__ void again(const StreamParams &p, Tail<true> &t, int g, int f, int c_first, int c_step) {
    const StreamPhase &h = p.ph[0];
    const int lane = threadIdx.x & 31, slots = t.tab.n[g], row0 = g * p.nb, n = min(p.nb, p.T - row0);
    if (slots == 0) return;
    // V as other SMs wrote it
    if (!__all_sync(0xffffffffu, wait_count(p, t, p.counters + 2, t.tab.items))) return;
    LoraValue v;
    v.K = p.K;
    v.fmt = p.fmt;
    v.sfx_step = 512;
    v.sfw_step = (int64_t)h.n_rt * 512;
    v.pieces = p.pieces;
    v.per = p.per;
    v.block = (int64_t)p.nb * p.r64;
    for (int c = c_first; c < n; c += c_step)
        for (int col = c; col < min(n, c + kCols); ++col) {
            const int64_t at = (int64_t)t.tab.row_of[row0 + col] * h.rows + f;
            float *out = static_cast<float *>(p.out) + at;
            __nv_bfloat16 *out16 = static_cast<__nv_bfloat16 *>(p.out) + at;
            bool bad = false;
            if (f < h.rows) bad = isnan(p.out_f32 ? *out : __bfloat162float(*out16));
            int s = 0;
            while (s < slots && col >= t.tab.first[g][s + 1]) ++s;
            v.rank = s < slots ? p.rank : 0;
            v.x = p.xq + (int64_t)(row0 + col) * p.K;
            v.sfx = h.sfx + (int64_t)g * h.ks * 512 + scale_byte(col);
            v.v = static_cast<const __nv_bfloat16 *>(p.v) +
                  ((int64_t)(g * p.slot_cap + s) * p.blocks * p.nb + col) * p.r64;
            for (uint32_t m = __ballot_sync(0xffffffffu, bad); m != 0; m &= m - 1) {
                const int src = __ffs((int)m) - 1;
                const int64_t fs = f - lane + src;
                v.w = p.w + fs * (p.K / 8 * (8 - p.gap8));
                v.sfw = h.sfw + fs / 128 * 512 + scale_byte(fs);
                v.b = static_cast<const __nv_bfloat16 *>(p.b) +
                      (s < slots ? (t.tab.adapter[g][s] * (int64_t)h.rows + fs) * p.rank : 0);
                float x = lora_value(v);
                if (p.bias != nullptr) x = __fadd_rn(x, __ldg(p.bias + fs));
                if (lane != src) continue;
                if (p.out_f32)
                    *out = x;
                else
                    *out16 = __float2bfloat16_rn(x);
            }
        }
}

// out[t, h] = sum_j w[t, j] y[pos[t, j], h] of one tile of h, j in order; four
// values a thread.  y: rows in memory, or where the tiles are split the sums of
// the tiles' parts (in order).  The pairs' rows and weights go through shared
// memory a table at a time, so that only the loads of y are on the way, several
// tokens' at once; a call of one table makes it before its first tile.
template <bool LORA>
__device__ __forceinline__ void fill_pairs(const StreamParams &p, Tail<LORA> &t, int tok0, int n) {
    for (int i = (int)threadIdx.x - kSEpiWarp0 * 32; i < n * p.k; i += kEpiThreads) {
        const int pos = __ldcg(p.pos + tok0 * p.k + i);
        int at = pos;
        if (t.parts[1] > 1 && pos >= 0) {
            // group and column of the row: its partial tiles' first value
            int g = 0;
            while (pos >= t.tab.g[g].row0 + t.tab.g[g].n) ++g;
            at = g << 8 | (pos - t.tab.g[g].row0);
        }
        t.pair_at[i] = at;
        t.pair_w[i] = __ldg(p.weights + tok0 * p.k + i);
    }
}
template <bool LORA>
__device__ __forceinline__ void combine(const StreamParams &p, Tail<LORA> &t, const Tile &o) {
    const StreamPhase &h = p.ph[1];
    const int H = h.rows, tid = threadIdx.x - kSEpiWarp0 * 32, parts = t.parts[1];
    const int per = h.sub * 32, teams = kEpiThreads / per;  // threads for a token's values
    const int f = tid % per * 4, c = o.w0 + f, team = tid / per;
    const int64_t part_size = (int64_t)2 * p.nb * 128;
    const int step = min(p.T, kPairs / p.k);  // tokens of a table
    for (int tok0 = 0; tok0 < p.T; tok0 += step) {
        const int n = min(step, p.T - tok0);
        if (step < p.T) {
            (void)epi_all(true);
            fill_pairs(p, t, tok0, n);
            (void)epi_all(true);
        }
        if (c >= H) continue;
        constexpr int kTok = 4;
        for (int a = team; a < n; a += teams * kTok) {
            float4 s[kTok];
#pragma unroll
            for (int u = 0; u < kTok; ++u) s[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int j = 0; j < p.k; ++j) {
                float4 v[kTok];
                if (parts == 1) {
#pragma unroll
                    for (int u = 0; u < kTok; ++u) {
                        const int tok = a + u * teams, at = tok < n ? t.pair_at[tok * p.k + j] : -1;
                        v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (at >= 0) v[u] = __ldcg(reinterpret_cast<const float4 *>(p.y + (int64_t)at * H + c));
                    }
                } else {
#pragma unroll
                    for (int u = 0; u < kTok; ++u) {
                        const int tok = a + u * teams, at = tok < n ? t.pair_at[tok * p.k + j] : -1;
                        v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (at < 0) continue;
                        const float *src = h.part + ((int64_t)((at >> 8) * h.mt + o.mt) * parts) * part_size +
                                           ((int64_t)(f >> 7) * p.nb + (at & 255)) * 128 + (f & 127);
#pragma unroll 8
                        for (int q = 0; q < parts; ++q) {
                            const float4 x = __ldcg(reinterpret_cast<const float4 *>(src + q * part_size));
                            v[u].x += x.x;
                            v[u].y += x.y;
                            v[u].z += x.z;
                            v[u].w += x.w;
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < kTok; ++u) {
                    const int tok = a + u * teams;
                    if (tok >= n || t.pair_at[tok * p.k + j] < 0) continue;
                    const float w = t.pair_w[tok * p.k + j];
                    s[u].x = fmaf(w, v[u].x, s[u].x);
                    s[u].y = fmaf(w, v[u].y, s[u].y);
                    s[u].z = fmaf(w, v[u].z, s[u].z);
                    s[u].w = fmaf(w, v[u].w, s[u].w);
                }
            }
#pragma unroll
            for (int u = 0; u < kTok; ++u) {
                const int tok = a + u * teams;
                if (tok >= n) continue;
                const int64_t at = (int64_t)(tok0 + tok) * H + c;
                if (p.out_f32)
                    *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) = s[u];
                else
                    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + at) =
                        make_uint2(pack_bf16(s[u].x, s[u].y), pack_bf16(s[u].z, s[u].w));
            }
        }
    }
}

// One ticket: its accumulator `acc` is complete.
template <bool LORA, int EPI>
__device__ __forceinline__ void finish_tile(const StreamParams &p, Tail<LORA> &t, const Tile &o, int acc,
                                            uint32_t tmem) {
    const StreamPhase &h = p.ph[EPI == kRows ? 1 : 0];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int q = warp & 3, half = (warp - kSEpiWarp0) >> 2;
    const int row_l = q * 32 + lane;  // weight row within a tile
    // two weight tiles: this warp takes tile `half`; gated, or one tile: every
    // other kCols columns (of both tiles, gated)
    constexpr int kSubs = EPI == kGated ? 2 : 1;
    constexpr int kJoin = EPI == kGated ? 2 : 4;  // parts read at a time
    const bool by_cols = EPI == kGated || h.sub == 1;
    const int c_first = by_cols ? half * kCols : 0, c_step = by_cols ? 2 * kCols : kCols;
    const int my_sub = by_cols ? 0 : half;
    const bool live = my_sub == 0 || o.has1;  // this warp has a weight tile
    const uint32_t ta = tmem + ((uint32_t)(q * 32) << 16) + acc * p.acc_cols;
    // kCols columns from c on of weight tile sub, its chains added
    auto load = [&](int sub, int c, float (&d)[kCols]) {
        const uint32_t at = ta + sub * p.chains * p.nb + c;
        uint32_t r[kCols], x[kCols];
        ptx::tmem_ld_32x32b_x8(at, r);
        if (p.chains == 2) ptx::tmem_ld_32x32b_x8(at + p.nb, x);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < kCols; ++i)
            d[i] = p.chains == 2 ? __uint_as_float(r[i]) + __uint_as_float(x[i]) : __uint_as_float(r[i]);
    };
    const int parts = t.parts[EPI == kRows ? 1 : 0];
    const int f = (my_sub ? o.w1 : o.w0) + row_l;
    const float bias = EPI == kOut && p.bias != nullptr && f < h.rows ? __ldg(p.bias + f) : 0.0f;
    const int64_t part_size = (int64_t)2 * p.nb * 128;
    float *part0 = h.part + (int64_t)o.tile * parts * part_size;  // the tile's parts
    bool last = true, spoilt = false;
    if (parts > 1) {
        float *part = part0 + o.part * part_size;
        if (live)
            for (int c = c_first; c < o.n; c += c_step)
#pragma unroll
                for (int s = 0; s < kSubs; ++s) {
                    const int sub = EPI == kGated ? s : my_sub;
                    float d[kCols];
                    load(sub, c, d);
                    float *dst = part + ((int64_t)sub * p.nb + c) * 128 + row_l;
#pragma unroll
                    for (int i = 0; i < kCols; ++i)
                        if (c + i < o.n) __stcg(dst + i * 128, d[i]);
                }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&t.acce[acc]));
        if constexpr (EPI == kRows) {
            // every part of every group of this tile of h: the weighted sum
            // reads the parts themselves
            if (count_in(t, p.done_tile + o.mt, t.tab.n_groups * parts)) combine(p, t, o);
            return;
        }
        last = count_in(t, h.part_cnt + o.tile, parts);
    }
    if (last && live)
        for (int c = c_first; c < o.n; c += c_step) {
            float v[kSubs][kCols];
#pragma unroll
            for (int s = 0; s < kSubs; ++s) {
                const int sub = EPI == kGated ? s : my_sub;
                if (parts == 1) {
                    load(sub, c, v[s]);
                } else {
                    // in order; several parts' loads in flight at a time
#pragma unroll
                    for (int i = 0; i < kCols; ++i) v[s][i] = 0.0f;
                    for (int a = 0; a < parts; a += kJoin) {
                        float x[kJoin][kCols];
#pragma unroll
                        for (int j = 0; j < kJoin; ++j) {
                            const float *src = part0 + (a + j) * part_size + ((int64_t)sub * p.nb + c) * 128 + row_l;
#pragma unroll
                            for (int i = 0; i < kCols; ++i)
                                x[j][i] = a + j < parts && c + i < o.n ? __ldcg(src + i * 128) : 0.0f;
                        }
#pragma unroll
                        for (int j = 0; j < kJoin; ++j)
#pragma unroll
                            for (int i = 0; i < kCols; ++i) v[s][i] += x[j][i];
                    }
                }
            }
            store_cols<LORA, EPI, kSubs>(p, h, t, o, c, o.n, f, q, lane, bias, v, spoilt);
        }
    if (parts == 1) {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&t.acce[acc]));
    }
    if constexpr (EPI == kGated) {
        if (last) {
            fence_proxy_async_all();
            (void)epi_all(true);
            if (threadIdx.x == kSEpiWarp0 * 32) (void)atom_add_acq_rel(p.done_group + o.g, 1);
        }
    } else if constexpr (EPI == kRows) {
        // the last group to finish this tile of h sums the tokens' experts
        if (count_in(t, p.done_tile + o.mt, t.tab.n_groups)) combine(p, t, o);
    } else {
        if (__any_sync(0xffffffffu, spoilt)) again(p, t, o.g, f, c_first, c_step);
    }
}

// (512: 128 registers a thread, which leaves room on the SM for the next call's
// preparing blocks while this one ends.  With its own 384 threads' worth, 140 to 158,
// device times are the same and calls back to back slower: 5 tokens over 64 experts 60.7
// -> 62.6 us, 16 over 32 4-bit ones 77.2 -> 78.2.)
template <bool LORA, int P>
__global__ void __launch_bounds__(512, 1) stream_kernel(const __grid_constant__ StreamParams p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = ptx::smem_addr(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (raw_base & 1023u)) & 1023u);
    const uint32_t sbase = ptx::smem_addr(smem);
    Tail<LORA> &t = *reinterpret_cast<Tail<LORA> *>(smem + p.stages * p.stage_bytes);
    volatile int *abort_flag = &t.abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            ptx::mbar_init(ptx::smem_addr(&t.full[s]), 2);
            ptx::mbar_init(ptx::smem_addr(&t.empty[s]), 1);
            ptx::mbar_init(ptx::smem_addr(&t.sfr[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(ptx::smem_addr(&t.accf[a]), 1);
            ptx::mbar_init(ptx::smem_addr(&t.acce[a]), kSEpiWarps);
        }
        for (int i = 0; i < kTickets; ++i) {
            ptx::mbar_init(ptx::smem_addr(&t.tk_full[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&t.tk_empty[i]), 3 + kSEpiWarps);
        }
        ptx::mbar_init(ptx::smem_addr(&t.drain), 1);
        ptx::mbar_init(ptx::smem_addr(&t.drain_sf), 1);
        t.abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        ptx::prefetch_tmap(&p.ph[0].W);
        ptx::prefetch_tmap(&p.ph[0].X);
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_addr(&t.tmem), 512);
        ptx::tmem_relinquish();
    }
    // Launched programmatically: the preparing kernel may still run, but what
    // was complete before it began, the indices among it, can be read (it lets
    // this kernel start only after its own wait).
    make_tables(p, t.tab);
    if (threadIdx.x == 0)
        for (int i = 0; i < (LORA ? 1 : 2); ++i) {
            const int tiles = t.tab.n_groups * p.ph[i].mt;
            t.parts[i] = parts_of(tiles, p.ph[i].ks, (int)gridDim.x);
            t.tickets[i] = tiles * t.parts[i];
        }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = t.tmem;
    const uint32_t sf_tmem = tmem + p.nacc * p.acc_cols;

    if (warp == 0) {
        if (lane == 0) {
            // the weights that some CTA will want first, to L2 while the tokens
            // are prepared (one-byte formats)
            Tile o;
            if (p.gap8 == 0 && decode(p, t, (int)blockIdx.x, o)) {
                const int k1 = min(min(o.k1, o.k0 + p.stages), p.ph[o.ph].ks);
                for (int k = o.k0; k < k1; ++k) {
                    ptx::tma_prefetch_3d(&p.ph[o.ph].W, k * kBK, o.w0, o.mat0);
                    if (o.has1) ptx::tma_prefetch_3d(&p.ph[o.ph].W, k * kBK, o.w1, o.mat1);
                }
            }
            ptx::grid_dep_wait();
            ptx::grid_dep_launch();
            load_weights(p, t, sbase);
        }
    } else if (warp == 1) {
        issue_mmas<LORA, P>(p, t, sbase, tmem, sf_tmem);
    } else if (warp == 2) {
        if (lane == 0) copy_scales(p, t, sbase, sf_tmem);
    } else if (warp == 3) {
        if (lane == 0) {
            ptx::grid_dep_wait();
            load_tokens<LORA, P>(p, t, sbase);
        }
    } else if (warp < kSEpiWarp0 + kSEpiWarps) {
        ptx::grid_dep_wait();
        if constexpr (LORA) {
            // items of V first, taken off a counter as the tickets are
            while (true) {
                (void)epi_all(true);
                if (threadIdx.x == kSEpiWarp0 * 32) t.item = atomicAdd(p.counters + 1, 1);
                (void)epi_all(true);
                const int item = t.item;
                if (item >= t.tab.items) break;
                low_rank<P>(p, t.tab, t.pick, item);
                fence_proxy_async_all();
                (void)epi_all(true);
                if (threadIdx.x == kSEpiWarp0 * 32) (void)atom_add_acq_rel(p.counters + 2, 1);
            }
        }
        if constexpr (!LORA)
            if (p.T <= kPairs / p.k) fill_pairs(p, t, 0, p.T);  // (read after the barriers below)
        Queue q;
        Tile o;
        for (int lt = 0;; ++lt) {
            const bool more = take<LORA, true>(p, t, q, o, 3);
            if (!epi_all(more)) break;
            uint32_t par;
            const int acc = acc_of(p, lt, par);
            if (!epi_all(wait_bar_warp(ptx::smem_addr(&t.accf[acc]), par, abort_flag, p, 3 * 256 + acc, 32))) break;
            ptx::tc_fence_after();
            if constexpr (LORA) {
                finish_tile<true, kOut>(p, t, o, acc, tmem);
            } else {
                if (o.ph == 0)
                    finish_tile<false, kGated>(p, t, o, acc, tmem);
                else
                    finish_tile<false, kRows>(p, t, o, acc, tmem);
            }
        }
    }

    __syncwarp();
    __syncthreads();
    if (*abort_flag) {
        // wait (bounded) for this CTA's MMAs, then give copies in flight a
        // bounded time before shared memory is released
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

template <bool LORA, int P>
cudaError_t launch_one(const StreamParams &p, int grid, cudaStream_t s) {
    auto kern = stream_kernel<LORA, P>;
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
    // more than half an SM's shared memory: one CTA per SM
    const size_t smem = (size_t)p.stages * p.stage_bytes + sizeof(Tail<LORA>) + 1024;
    return launch_programmatic_smem(kern, dim3((unsigned)grid), dim3(kSThreads), smem, s, p);
}

}  // namespace

void stream_sizes(StreamParams &p, int nb, int sub, bool lora, int v_blocks) {
    p.nb = nb;
    // Tensor memory beside the scales (up to eight stages' 128 columns): two
    // accumulators, so that a tile's epilogue overlaps the next tile, then two
    // chains each
    const int room_cols = 512 - 8 * kSfSlot;
    p.nacc = 2 * sub * nb <= room_cols ? 2 : 1;
    p.chains = p.nacc * sub * 2 * nb <= room_cols ? 2 : 1;
    p.acc_cols = sub * p.chains * nb;
    p.w_bytes = sub * kWTile;
    // V's pieces in rows of their own: room for all columns of two, or of
    // kStreamMaxTokens for half of them; of three for 32 (more stages; slots of more
    // columns take further steps)
    p.v_cols = v_blocks == 3 ? (nb < 32 ? nb : 32) : v_blocks == 2 && nb == kStreamMaxTokens ? nb / 2 : nb;
    const int x_rows = v_blocks * p.v_cols;
    p.x_bytes = (x_rows > nb ? x_rows : nb) * 128;
    // the scales' chunks (512 bytes each: tokens, weight tiles), in 1024-byte multiples
    p.stage_bytes = p.w_bytes + p.x_bytes + (sub == 2 ? 2048 : 1024);
    const int room = kSmemMax - 1024 - (int)(lora ? sizeof(Tail<true>) : sizeof(Tail<false>));
    p.stages = room / p.stage_bytes;
    const int cols = (512 - p.nacc * p.acc_cols) / kSfSlot;
    if (p.stages > cols) p.stages = cols;
    if (p.stages > kMaxStages) p.stages = kMaxStages;
}

size_t stream_part_bytes(const StreamParams &p, int num_sms) {
    return (size_t)num_sms * 2 * p.nb * 128 * sizeof(float);  // split tiles: at most a part per SM
}

cudaError_t launch_stream(bool lora, const StreamParams &p, int num_sms, cudaStream_t s) {
    const int segs = quant_segments(p.ph[0].ks);
    cudaError_t e;
    if (lora) {
        e = launch_programmatic(lora_prep_kernel, dim3((unsigned)(p.T * segs)), dim3(kPrepThreads), s, p);
        if (e == cudaSuccess)
            e = p.pieces == 3 ? launch_one<true, 3>(p, num_sms, s) : launch_one<true, 2>(p, num_sms, s);
    } else {
        e = launch_programmatic(moe_prep_kernel, dim3((unsigned)(p.T * segs)), dim3(kPrepThreads), s, p);
        if (e == cudaSuccess) e = launch_one<false, 0>(p, num_sms, s);
    }
    return e;
}

}  // namespace fp8g
