// MoE router: the k largest of a token's E expert logits, their weights, and
// the order the grouped GEMM takes its rows in.
//
//   chosen(t) = the k largest logits l[t, :], largest first, ties to the lower
//               expert; a NaN or -inf logit is never chosen (id -1, weight 0)
//   weight    = scale * softmax over all experts | softmax over the chosen |
//               sigmoid | sigmoid / sum of the chosen sigmoids
//   order     = the pairs (t, j) by expert, then by t k + j
//
// Up to 64 experts four lanes take a token (route_quad), more: a warp takes one, its
// logits in registers as order-preserving integers (lane i: experts i, i + 32, ...),
// with two warp reductions in each of the k rounds (redux: the largest key, then the
// lowest expert that has it).  Either way a logit is read once, and what bounds the
// kernel is not memory (32768 x 64 fp32 logits, 8 MB, are read in 1.3 us) but issuing
// instructions: of four lanes' comparisons, about 100 pairs of 64-bit words a lane,
// softmax, ranks and stores, 1800 a warp; a block of 32 warps an SM issues in 57 % of
// its slots (DRAM 7 %), and 24 of 152 SMs have no block.
//
// Device times per call, back to back in a graph (k = 8, softmax over all): one token
// of 8 experts 2.1 us, of 64 3.9, 77 with the order 6.6: latency; 2048 with it 8.6,
// 32768 10.5 without and 17.0 with it, 262144 130; 77, 2048 and 32768 tokens of 256
// experts 20.5, 22.1 and 69.  (Inserting into a list of eight instead of merging, 168
// pairs: the first kernel alone 18.4 us in place of 13.7.)
//
// Order: a stable counting sort.  A token chooses an expert at most once, so a
// warp's choices of an expert are a mask over its eight tokens: a pair's rank
// is the masks' set bits before it.  A block counts; the second kernel (none when
// one block holds every token) adds the counts of the blocks before and stores
// the pairs at base + rank (6.5 us more for 262144 pairs; ranking them there by
// matching in a warp, 3 us more still).  No atomic decides a position, so the order is
// the same in every run.
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace fp8g {

namespace {

constexpr int kWarps = 32;
constexpr int kBlockTokens = 256;  // tokens of a block at most
constexpr int kFewTokens = 64;     // of a block where that leaves SMs idle

__device__ __forceinline__ float neg_inf() { return __int_as_float((int)0xFF800000u); }

struct RouteArgs {
    const void *logits;
    int64_t ld;  // elements between rows
    int32_t T, E, k, score;
    float scale;
    int32_t *ids;
    float *weights;
    int32_t *counts, *rows, *slots;  // all null: no order wanted
    int32_t *hist;                   // [blocks][E]: pairs of a block's tokens
    uint8_t *rank;                   // [T k]: of a pair among its block's of its expert
    int32_t vec;                     // four logits of a row at a time
    int32_t tokens;                  // of a block
};

// Order-preserving key of a logit, 0 where it cannot be chosen.
__device__ __forceinline__ uint32_t route_key(float l) {
    if (!(l > neg_inf())) return 0u;  // NaN, -inf
    const uint32_t b = __float_as_uint(l + 0.0f);  // -0 ties with +0
    return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t key) {
    return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// exp(l - top) with top the largest; infinite tops count as equal.
__device__ __forceinline__ float rel_exp(float l, float top) {
    return l == top ? 1.0f : expf(l - top);
}

// 1 / (1 + exp(-l)) times exp(-m), m at most 0.  In the normalised sigmoid, with m
// the largest chosen logit or 0, the factor cancels in the quotient and the largest
// numerator is at least 1/2 however low the logits (with m = 0 all are 0 from -89
// down, and so is their sum).  em: exp(m).
__device__ __forceinline__ float sigmoid_over(float l, float m, float em) {
    return 1.0f / (em + expf(m - l));
}
__device__ __forceinline__ float sigmoid_shift(int score, float top) {
    return score == FP8G_SCORE_SIGMOID_NORM ? fminf(top, 0.0f) : 0.0f;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// One token: its choices to ids / weights; the lanes j < k return the chosen
// expert (-1: none).
template <int NV, bool BF16>
__device__ __forceinline__ int route_token(const RouteArgs &a, int t, int lane) {
    uint32_t key[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = lane + 32 * i;
        float l = neg_inf();
        if (e < a.E) {
            const int64_t off = (int64_t)t * a.ld + e;
            if constexpr (BF16)
                l = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.logits)[off]);
            else
                l = static_cast<const float *>(a.logits)[off];
        }
        key[i] = route_key(l);
    }
    uint32_t all = 0;  // the largest key
    float sum = 0.0f;
    if (a.score == FP8G_SCORE_SOFTMAX) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) m = max(m, key[i]);
        all = __reduce_max_sync(0xffffffffu, m);
        const float top = key_value(all);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (key[i] != 0u) sum += rel_exp(key_value(key[i]), top);
        sum = warp_sum(sum);
    }
    int mine = -1;
    uint32_t mine_key = 0;
    for (int j = 0; j < a.k; ++j) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        const uint32_t m = __reduce_max_sync(0xffffffffu, best);
        if (m == 0u) break;
        const uint32_t e = __reduce_min_sync(0xffffffffu,
                                             best == m ? (uint32_t)(lane + 32 * at) : 0xFFFFFFFFu);
        if ((e & 31u) == (uint32_t)lane) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if ((uint32_t)i == e >> 5) key[i] = 0u;
        }
        if (j == 0) all = m;
        if (lane == j) {
            mine = (int)e;
            mine_key = m;
        }
    }
    float w = 0.0f;
    if (mine >= 0) {
        const float l = key_value(mine_key), top = key_value(all), m = sigmoid_shift(a.score, top);
        w = a.score <= FP8G_SCORE_SOFTMAX_TOPK ? rel_exp(l, top) : sigmoid_over(l, m, m < 0.0f ? expf(m) : 1.0f);
    }
    if (a.score == FP8G_SCORE_SOFTMAX_TOPK || a.score == FP8G_SCORE_SIGMOID_NORM) sum = warp_sum(w);
    if (lane < a.k) {
        if (a.score != FP8G_SCORE_SIGMOID && mine >= 0) w = __fdiv_rn(w, sum);
        a.ids[(int64_t)t * a.k + lane] = mine;
        a.weights[(int64_t)t * a.k + lane] = mine >= 0 ? w * a.scale : 0.0f;
    }
    return mine;
}

__device__ __forceinline__ uint64_t umax64(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t umin64(uint64_t a, uint64_t b) { return a > b ? b : a; }

// Larger first.
__device__ __forceinline__ void order2(uint64_t &a, uint64_t &b) {
    const uint64_t hi = umax64(a, b);
    b = umin64(a, b);
    a = hi;
}
// Batcher's odd-even merge sort, largest first (K = 4, 8, 16: 5, 19, 63 pairs).
template <int K>
__device__ __forceinline__ void sort_desc(uint64_t (&v)[K]) {
#pragma unroll
    for (int p = 1; p < K; p <<= 1)
#pragma unroll
        for (int k = p; k >= 1; k >>= 1)
#pragma unroll
            for (int i = 0; i < K; ++i)
                if (i >= k % p && (i - k % p) / k % 2 == 0 && i + k < K && i / (2 * p) == (i + k) / (2 * p))
                    order2(v[i], v[i + k]);
}
// The K largest of two such lists: the larger halves' maxima are bitonic.
template <int K>
__device__ __forceinline__ void merge_desc(uint64_t (&v)[K], const uint64_t (&o)[K]) {
#pragma unroll
    for (int j = 0; j < K; ++j) v[j] = umax64(v[j], o[K - 1 - j]);
#pragma unroll
    for (int h = K / 2; h > 0; h >>= 1)
#pragma unroll
        for (int j = 0; j < K; ++j)
            if ((j & h) == 0) order2(v[j], v[j + h]);
}

// Four lanes take a token: lane q a quarter of the experts, as (key, ~expert)
// words, K at a time: sorted, merged into its K best, and those over the lanes
// in two rounds.  All four end with the token's list `best`; lane q scores and
// stores choices q, q + 4, ...  t < 0: no token (the lane takes part in the
// shuffles only).
template <int NE, int K, bool BF16>
__device__ __forceinline__ void route_quad(const RouteArgs &a, int t, int q, uint64_t (&best)[K]) {
    uint32_t key[NE];
    const int64_t row = (int64_t)max(t, 0) * a.ld;
    const int live = t < 0 ? 0 : a.E;
    if (a.vec) {  // experts 16 c + 4 q and the next three
#pragma unroll
        for (int c = 0; c < NE / 4; ++c) {
            const int e = 16 * c + 4 * q;
            float l[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
            if (e < live) {
                if constexpr (BF16) {
                    const uint2 r = __ldg(reinterpret_cast<const uint2 *>(
                        static_cast<const __nv_bfloat16 *>(a.logits) + row + e));
                    l[0] = __uint_as_float(r.x << 16);
                    l[1] = __uint_as_float(r.x & 0xFFFF0000u);
                    l[2] = __uint_as_float(r.y << 16);
                    l[3] = __uint_as_float(r.y & 0xFFFF0000u);
                } else {
                    const float4 r =
                        __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(a.logits) + row + e));
                    l[0] = r.x;
                    l[1] = r.y;
                    l[2] = r.z;
                    l[3] = r.w;
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) key[4 * c + i] = route_key(l[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = 16 * (i / 4) + 4 * q + i % 4;
            float l = neg_inf();
            if (e < live) {
                if constexpr (BF16)
                    l = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.logits)[row + e]);
                else
                    l = static_cast<const float *>(a.logits)[row + e];
            }
            key[i] = route_key(l);
        }
    }
#pragma unroll
    for (int c = 0; c < (NE + K - 1) / K; ++c) {
        uint64_t v[K];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int i = c * K + j;
            v[j] = i < NE && key[i < NE ? i : 0] != 0u
                       ? (uint64_t)key[i < NE ? i : 0] << 32 | (uint32_t)~(16 * (i / 4) + 4 * q + i % 4)
                       : 0;
        }
        sort_desc<K>(v);
        if (c == 0) {
#pragma unroll
            for (int j = 0; j < K; ++j) best[j] = v[j];
        } else {
            merge_desc<K>(best, v);
        }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        uint64_t v[K];
#pragma unroll
        for (int j = 0; j < K; ++j) v[j] = __shfl_xor_sync(0xffffffffu, best[j], o);
        merge_desc<K>(best, v);
    }
    const float top = key_value((uint32_t)(best[0] >> 32));
    float sum = 0.0f;
    if (a.score == FP8G_SCORE_SOFTMAX) {
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (key[i] != 0u) sum += rel_exp(key_value(key[i]), top);
    }
    const float m = sigmoid_shift(a.score, top), em = m < 0.0f ? expf(m) : 1.0f;
    float w[K / 4];
    uint64_t mine[K / 4];
#pragma unroll
    for (int j = 0; j < K / 4; ++j) {
        const uint64_t lo = q & 1 ? best[4 * j + 1] : best[4 * j], hi = q & 1 ? best[4 * j + 3] : best[4 * j + 2];
        mine[j] = 4 * j + q < a.k ? (q & 2 ? hi : lo) : 0;
        const uint32_t kj = (uint32_t)(mine[j] >> 32);
        w[j] = 0.0f;
        if (kj != 0u)
            w[j] = a.score <= FP8G_SCORE_SOFTMAX_TOPK ? rel_exp(key_value(kj), top)
                                                      : sigmoid_over(key_value(kj), m, em);
        if (a.score == FP8G_SCORE_SOFTMAX_TOPK || a.score == FP8G_SCORE_SIGMOID_NORM) sum += w[j];
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    if (t < 0) return;
#pragma unroll
    for (int j = 0; j < K / 4; ++j)
        if (4 * j + q < a.k) {
            const bool on = (mine[j] >> 32) != 0;
            const float v = a.score == FP8G_SCORE_SIGMOID ? w[j] : __fdiv_rn(w[j], sum);
            a.ids[(int64_t)t * a.k + 4 * j + q] = on ? (int)~(uint32_t)mine[j] : -1;
            a.weights[(int64_t)t * a.k + 4 * j + q] = on ? v * a.scale : 0.0f;
        }
}

// Shared memory of a block that wants the order.
struct Order {
    int32_t *cnt, *base, *total;
    uint32_t *mask;   // [warps][E / 4]: a byte an expert: which of the warp's (8) tokens chose it
    uint16_t *start;  // [warps][E]: pairs of the expert in earlier warps
    int words;        // of a warp's masks
    __device__ __forceinline__ Order(int32_t *sm, int E) {
        cnt = sm;
        base = sm + E;
        total = sm + 2 * E;
        words = (E + 3) / 4;
        mask = reinterpret_cast<uint32_t *>(sm + 2 * E + 1);
        start = reinterpret_cast<uint16_t *>(mask + kWarps * words);
    }
    __device__ __forceinline__ void note(int warp, int i, int e) {  // the warp's token i chose e
        atomicOr(mask + warp * words + (e >> 2), 1u << (8 * (e & 3) + i));
    }
    // Rank of that pair among the block's of its expert, after starts().
    __device__ __forceinline__ int rank(int warp, int i, int e, int E) const {
        const uint32_t m = mask[warp * words + (e >> 2)] >> (8 * (e & 3));
        return start[warp * E + e] + __popc(m & ((1u << i) - 1u));
    }
    // Starts and counts of the block, by all threads, after every note.
    __device__ __forceinline__ void starts(int E) {
        __syncthreads();
        const int warps = (int)blockDim.x >> 5;
        for (int e = threadIdx.x; e < E; e += blockDim.x) {
            int run = 0;
#pragma unroll 8
            for (int w = 0; w < warps; ++w) {
                start[w * E + e] = (uint16_t)run;
                run += __popc(mask[w * words + (e >> 2)] >> (8 * (e & 3)) & 255u);
            }
            cnt[e] = run;
        }
        __syncthreads();
    }
};
size_t order_smem(int E) { return (size_t)(2 * E + 1 + kWarps * ((E + 3) / 4)) * 4 + (size_t)kWarps * E * 2; }

// Exclusive prefix over experts of cnt (in place to base), by warp 0; the sum
// goes to *total.  Call with all threads.
__device__ __forceinline__ void expert_prefix(const int32_t *cnt, int32_t *base, int E,
                                              int32_t *total) {
    __syncthreads();
    if (threadIdx.x < 32) {
        int run = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + (int)threadIdx.x;
            const int c = e < E ? cnt[e] : 0;
            int s = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, s, o);
                if ((int)threadIdx.x >= o) s += v;
            }
            if (e < E) base[e] = run + s - c;
            run += __shfl_sync(0xffffffffu, s, 31);
        }
        if (threadIdx.x == 0) *total = run;
    }
    __syncthreads();
}

// K 0: a warp takes a token at a time, up to eight in a row, NV = ceil(E / 32);
// else four lanes take one, NV = ceil(E / 4), K at least a.k.
template <int NV, int K, bool BF16>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(RouteArgs a) {
    extern __shared__ int32_t sm[];
    Order o(sm, a.E);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = (int)blockDim.x >> 5;
    const bool ordered = a.rows != nullptr;
    if (ordered) {
        for (int i = threadIdx.x; i < warps * o.words; i += blockDim.x) o.mask[i] = 0u;
        __syncthreads();
    }
    ptx::grid_dep_wait();  // launched programmatically: global memory from here on
    const int t0 = blockIdx.x * a.tokens, n = min(a.T - t0, a.tokens);
    const int per = K == 0 ? (n + warps - 1) / warps : 8;  // tokens of a warp
    // this lane's choices: (expert, token of the warp), and the pair's number
    constexpr int kMine = K == 0 ? 8 : K / 4;
    int mine[kMine];
    const int q = threadIdx.x & 3, quad = lane >> 2;
    if constexpr (K == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            mine[i] = -1;
            if (i < per && warp * per + i < n) mine[i] = route_token<NV, BF16>(a, t0 + warp * per + i, lane);
        }
    } else {
        const int i = (int)(threadIdx.x >> 2);
        uint64_t best[K];
        route_quad<NV, K, BF16>(a, i < n ? t0 + i : -1, q, best);
#pragma unroll
        for (int j = 0; j < K / 4; ++j) {
            const uint64_t lo = q & 1 ? best[4 * j + 1] : best[4 * j], hi = q & 1 ? best[4 * j + 3] : best[4 * j + 2];
            const uint64_t b = q & 2 ? hi : lo;
            mine[j] = i < n && 4 * j + q < a.k && (b >> 32) != 0 ? (int)~(uint32_t)b : -1;
        }
    }
    if (!ordered) {
        ptx::grid_dep_launch();
        return;
    }
#pragma unroll
    for (int j = 0; j < kMine; ++j)
        if (mine[j] >= 0) o.note(warp, K == 0 ? j : quad, mine[j]);
    o.starts(a.E);
    const bool alone = gridDim.x == 1;
    if (alone) {
        expert_prefix(o.cnt, o.base, a.E, o.total);
        for (int e = threadIdx.x; e < a.E; e += blockDim.x) a.counts[e] = o.cnt[e];
    } else {
        for (int e = threadIdx.x; e < a.E; e += blockDim.x) a.hist[(int64_t)blockIdx.x * a.E + e] = o.cnt[e];
    }
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
        if (mine[j] < 0) continue;
        const int i = K == 0 ? j : quad;
        const int token = t0 + warp * per + i, pair = token * a.k + (K == 0 ? lane : 4 * j + q);
        const int r = o.rank(warp, i, mine[j], a.E);
        if (alone) {
            a.rows[o.base[mine[j]] + r] = token;
            a.slots[o.base[mine[j]] + r] = pair;
        } else {
            a.rank[pair] = (uint8_t)r;
        }
    }
    if (alone)  // places past the last pair
        for (int i = *o.total + (int)threadIdx.x; i < n * a.k; i += blockDim.x) a.rows[i] = a.slots[i] = -1;
    ptx::grid_dep_launch();
}

// More than one block of tokens: the places, from every block's counts.
__global__ void __launch_bounds__(kWarps * 32) route_order_kernel(RouteArgs a, int blocks) {
    extern __shared__ int32_t sm[];
    int32_t *cnt = sm, *base = sm + a.E, *total = sm + 2 * a.E;
    int32_t *before = total + 1;  // pairs of expert e in earlier blocks
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) cnt[e] = before[e] = 0;
    __syncthreads();
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int t0 = blockIdx.x * a.tokens, n = min(a.T - t0, a.tokens) * a.k, i0 = t0 * a.k;
    // this thread's first pairs, on the way while the counts are added
    constexpr int kFirst = 2;
    int e[kFirst], r[kFirst];
#pragma unroll
    for (int j = 0; j < kFirst; ++j) {
        const int i = (int)threadIdx.x + j * (int)blockDim.x;
        e[j] = i < n ? __ldcg(a.ids + i0 + i) : -1;
        r[j] = i < n ? __ldcg(a.rank + i0 + i) : 0;
    }
    // whole sums: the order of the additions does not matter
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int x = lane; x < a.E; x += 32) {
        int s = 0, p = 0;
#pragma unroll 4
        for (int b = warp; b < blocks; b += kWarps) {
            const int c = __ldcg(a.hist + (int64_t)b * a.E + x);
            s += c;
            if (b < (int)blockIdx.x) p += c;
        }
        atomicAdd(&cnt[x], s);
        atomicAdd(&before[x], p);
    }
    expert_prefix(cnt, base, a.E, total);
    for (int x = threadIdx.x; x < a.E; x += blockDim.x) {
        if (blockIdx.x == 0) a.counts[x] = cnt[x];
        base[x] += before[x];
    }
    __syncthreads();
    auto place = [&](int i, int x, int rank) {
        if (x < 0) return;
        a.rows[base[x] + rank] = (i0 + i) / a.k;
        a.slots[base[x] + rank] = i0 + i;
    };
#pragma unroll
    for (int j = 0; j < kFirst; ++j) place((int)threadIdx.x + j * (int)blockDim.x, e[j], r[j]);
    for (int i = (int)threadIdx.x + kFirst * (int)blockDim.x; i < n; i += (int)blockDim.x)
        place(i, __ldcg(a.ids + i0 + i), __ldcg(a.rank + i0 + i));
    // places past the last pair
    for (int i = (int)threadIdx.x; i < n; i += (int)blockDim.x)
        if (i0 + i >= *total) a.rows[i0 + i] = a.slots[i0 + i] = -1;
}

template <int NV, int K>
cudaError_t launch_nv(const RouteArgs &a, bool bf16, int blocks, int threads, size_t smem,
                      cudaStream_t s) {
    return bf16 ? launch_programmatic_smem(route_kernel<NV, K, true>, dim3(blocks), dim3(threads), smem, s, a)
                : launch_programmatic_smem(route_kernel<NV, K, false>, dim3(blocks), dim3(threads), smem, s, a);
}

}  // namespace

// Tokens of a block.  64 where the blocks' counts, which every block of the order
// adds up, stay few: with the order (64 experts, k = 8) 2048 tokens take 8.6 us, with
// 256 16.4; 8192 9.0 and 16.6; 32768 25.9, with 256 17.0.  Up to 256 tokens one block
// makes the order by itself (256: 13.6 us; a temporary and a second launch cost the
// host 6 us).
static int route_tokens(int64_t T, bool ordered) {
    if (ordered && (T <= kBlockTokens || T > 128 * kFewTokens)) return kBlockTokens;
    return kFewTokens;
}
int route_blocks(int64_t T, bool ordered) {
    const int n = route_tokens(T, ordered);
    return (int)((T + n - 1) / n);
}

cudaError_t launch_moe_route(const void *logits, int bf16, int64_t ld, int32_t T, int32_t E, int32_t k,
                             int32_t score, float scale, int32_t *ids, float *weights,
                             int32_t *counts, int32_t *rows, int32_t *slots, int32_t *hist,
                             cudaStream_t s) {
    const int tokens = route_tokens(T, rows != nullptr), blocks = route_blocks(T, rows != nullptr);
    const uintptr_t unit = bf16 ? 8 : 16;  // bytes of four logits
    const int vec = E % 4 == 0 && ld % 4 == 0 && reinterpret_cast<uintptr_t>(logits) % unit == 0;
    uint8_t *rank = reinterpret_cast<uint8_t *>(hist + (int64_t)blocks * E);
    const RouteArgs a{logits, ld, T, E, k, score, scale, ids, weights, counts, rows, slots, hist, rank, vec,
                      tokens};
    const size_t smem = rows == nullptr ? 0 : order_smem(E);  // E <= 256: 27 KB
    cudaError_t e;
    const int most = T < tokens ? T : tokens;  // tokens of a block
    const bool b16 = bf16 != 0;
    // a warp a token against four lanes a token, 64 experts, k = 8: 2.8 and 3.9 us for
    // one token, 4.0 and 3.8 for 32, 6.8 and 4.3 for 256, 25.4 and 10.5 for 32768
    if (E <= 64) {
        const int threads = (most * 4 + 31) / 32 * 32;
        if (E <= 32)
            e = k <= 4   ? launch_nv<8, 4>(a, b16, blocks, threads, smem, s)
                : k <= 8 ? launch_nv<8, 8>(a, b16, blocks, threads, smem, s)
                         : launch_nv<8, 16>(a, b16, blocks, threads, smem, s);
        else
            e = k <= 4   ? launch_nv<16, 4>(a, b16, blocks, threads, smem, s)
                : k <= 8 ? launch_nv<16, 8>(a, b16, blocks, threads, smem, s)
                         : launch_nv<16, 16>(a, b16, blocks, threads, smem, s);
    } else {
        const int threads = 32 * (most < kWarps ? most : kWarps);
        e = E <= 128 ? launch_nv<4, 0>(a, b16, blocks, threads, smem, s)
                     : launch_nv<8, 0>(a, b16, blocks, threads, smem, s);
    }
    if (e != cudaSuccess || rows == nullptr || blocks == 1) return e;
    return launch_programmatic_smem(route_order_kernel, dim3(blocks), dim3(kWarps * 32),
                                    (size_t)(3 * E + 1) * 4, s, a, blocks);
}

}  // namespace fp8g
