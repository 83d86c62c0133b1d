// MoE router: the k largest of a token's E expert logits, their weights, and
// the order the grouped GEMM takes its rows in.
//
//   chosen(t) = the k largest logits l[t, :], largest first, ties to the lower
//               expert; a NaN or -inf logit is never chosen (id -1, weight 0)
//   weight    = scale * softmax over all experts | softmax over the chosen |
//               sigmoid | sigmoid / sum of the chosen sigmoids
//   order     = the pairs (t, j) by expert, then by t k + j
//
// A warp takes a token, its logits in registers as order-preserving integers
// (lane i: experts i, i + 32, ...).  Each of the k rounds is two warp
// reductions (redux: the largest key, then the lowest expert that has it), so
// a token costs about 2 k reductions and one pass over its logits: the kernel
// reads every logit once and is bound by latency, not by memory (32768 x 64
// fp32 logits are 8 MB).
//
// Order: a stable counting sort.  A block counts its tokens' choices per
// expert; the second kernel (none when one block holds every token) adds the
// counts of the blocks before it, ranks each pair among its warp's and its
// block's, and stores it.  No atomic decides a position, so the order is the
// same in every run.
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace fp8g {

namespace {

constexpr int kWarps = 32;
constexpr int kTokensPerBlock = 256;
constexpr int kQuadTokens = 32;  // more tokens than this: four lanes a token

__device__ __forceinline__ float neg_inf() { return __int_as_float((int)0xFF800000u); }

struct RouteArgs {
    const void *logits;
    int64_t ld;  // elements between rows
    int32_t T, E, k, score;
    float scale;
    int32_t *ids;
    float *weights;
    int32_t *counts, *rows, *slots;  // all null: no order wanted
    int32_t *hist;                   // [blocks][E]
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
        const float l = key_value(mine_key);
        w = a.score <= FP8G_SCORE_SOFTMAX_TOPK ? rel_exp(l, key_value(all)) : 1.0f / (1.0f + expf(-l));
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

// Four lanes take a token: lane q the experts q, q + 4, ...  Each keeps its
// K best as a descending list of (key, ~expert) words, a new one passing down
// the list by compare-exchange; two rounds of bitonic merges over the lanes
// give all four the token's list.  Returns it in `best`; t < 0: no token (the
// lane takes part in the shuffles only).
template <int NE, int K, bool BF16>
__device__ __forceinline__ void route_quad(const RouteArgs &a, int t, int q, uint64_t (&best)[K]) {
    uint32_t key[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = q + 4 * i;
        key[i] = 0u;
        if (t >= 0 && e < a.E) {
            const int64_t off = (int64_t)t * a.ld + e;
            if constexpr (BF16)
                key[i] = route_key(__bfloat162float(static_cast<const __nv_bfloat16 *>(a.logits)[off]));
            else
                key[i] = route_key(static_cast<const float *>(a.logits)[off]);
        }
    }
#pragma unroll
    for (int j = 0; j < K; ++j) best[j] = 0;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        uint64_t w = key[i] == 0u ? 0 : (uint64_t)key[i] << 32 | (uint32_t)~(q + 4 * i);
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const uint64_t lo = umin64(best[j], w);
            best[j] = umax64(best[j], w);
            w = lo;
        }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        uint64_t c[K];
#pragma unroll
        for (int j = 0; j < K; ++j)
            c[j] = umax64(best[j], __shfl_xor_sync(0xffffffffu, best[K - 1 - j], o));
#pragma unroll
        for (int h = K / 2; h > 0; h >>= 1)
#pragma unroll
            for (int j = 0; j < K; ++j)
                if ((j & h) == 0) {
                    const uint64_t hi = umax64(c[j], c[j + h]);
                    c[j + h] = umin64(c[j], c[j + h]);
                    c[j] = hi;
                }
#pragma unroll
        for (int j = 0; j < K; ++j) best[j] = c[j];
    }
    // the scores, in the order of the choices (the same on all four lanes)
    const float top = key_value((uint32_t)(best[0] >> 32));
    float sum = 0.0f;
    if (a.score == FP8G_SCORE_SOFTMAX) {
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (key[i] != 0u) sum += rel_exp(key_value(key[i]), top);
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    }
    float w[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
        const uint32_t kj = (uint32_t)(best[j] >> 32);
        w[j] = 0.0f;
        if (j < a.k && kj != 0u)
            w[j] = a.score <= FP8G_SCORE_SOFTMAX_TOPK ? rel_exp(key_value(kj), top)
                                                      : 1.0f / (1.0f + expf(-key_value(kj)));
        if (a.score == FP8G_SCORE_SOFTMAX_TOPK || a.score == FP8G_SCORE_SIGMOID_NORM) sum += w[j];
    }
    if (t < 0) return;
#pragma unroll
    for (int j = 0; j < K; ++j)
        if ((j & 3) == q && j < a.k) {
            const bool on = (best[j] >> 32) != 0;
            const float v = a.score == FP8G_SCORE_SIGMOID ? w[j] : __fdiv_rn(w[j], sum);
            a.ids[(int64_t)t * a.k + j] = on ? (int)~(uint32_t)best[j] : -1;
            a.weights[(int64_t)t * a.k + j] = on ? v * a.scale : 0.0f;
        }
}

// The pairs [i0, i0 + n) of the ids, ranked among themselves by expert, to
// their places: base[e] is the first place of this block's pairs of expert e.
// wh [kWarps][E] counts per warp.  Call with all threads.
__device__ __forceinline__ void place_pairs(const RouteArgs &a, const int32_t *ids, int64_t i0, int n,
                                            const int32_t *base, int32_t *wh, int64_t total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarps = blockDim.x >> 5;
    const int per = ((n + nwarps - 1) / nwarps + 31) & ~31;  // pairs per warp, whole steps
    for (int i = threadIdx.x; i < nwarps * a.E; i += blockDim.x) wh[i] = 0;
    __syncthreads();
    const int lo = warp * per, hi = min(n, lo + per);
    for (int i = lo + lane; i < hi; i += 32) {
        const int e = ids[i0 + i];
        if (e >= 0) atomicAdd(&wh[warp * a.E + e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        int run = base[e];
        for (int w = 0; w < nwarps; ++w) {
            const int c = wh[w * a.E + e];
            wh[w * a.E + e] = run;
            run += c;
        }
    }
    __syncthreads();
    for (int i = lo; i < hi; i += 32) {
        const int f = i + lane;
        const int e = f < hi ? ids[i0 + f] : -1;
        const uint32_t same = __match_any_sync(0xffffffffu, e);
        if (e >= 0) {
            const int at = wh[warp * a.E + e] + __popc(same & ((1u << lane) - 1u));
            const int64_t pair = i0 + f;
            a.rows[at] = (int32_t)(pair / a.k);
            a.slots[at] = (int32_t)pair;
        }
        __syncwarp();
        if (e >= 0 && lane == 31 - __clz(same)) wh[warp * a.E + e] += __popc(same);
        __syncwarp();
    }
    // places past the last pair
    for (int i = threadIdx.x; i < n; i += blockDim.x)
        if (i0 + i >= total) {
            a.rows[i0 + i] = -1;
            a.slots[i0 + i] = -1;
        }
}

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

// K 0: a warp takes a token, NV = ceil(E / 32); else four lanes take one, NV =
// ceil(E / 4), K at least a.k.
template <int NV, int K, bool BF16>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(RouteArgs a) {
    extern __shared__ int32_t sm[];  // cnt [E], base [E], total, warp counts [kWarps][E]
    int32_t *cnt = sm, *base = sm + a.E, *total = sm + 2 * a.E, *wh = sm + 2 * a.E + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool ordered = a.rows != nullptr;
    if (ordered)
        for (int e = threadIdx.x; e < a.E; e += blockDim.x) cnt[e] = 0;
    __syncthreads();
    ptx::grid_dep_wait();  // launched programmatically: global memory from here on
    const int t0 = blockIdx.x * kTokensPerBlock, t1 = min(a.T, t0 + kTokensPerBlock);
    if constexpr (K == 0) {
        for (int t = t0 + warp; t < t1; t += blockDim.x >> 5) {
            const int e = route_token<NV, BF16>(a, t, lane);
            if (ordered && e >= 0) atomicAdd(&cnt[e], 1);
        }
    } else {
        const int t = t0 + (int)(threadIdx.x >> 2), q = threadIdx.x & 3;
        uint64_t best[K];
        route_quad<NV, K, BF16>(a, t < t1 ? t : -1, q, best);
        if (ordered && t < t1) {
#pragma unroll
            for (int j = 0; j < K; ++j)
                if ((j & 3) == q && j < a.k && (best[j] >> 32) != 0) atomicAdd(&cnt[~(uint32_t)best[j]], 1);
        }
    }
    if (!ordered) {
        ptx::grid_dep_launch();
        return;
    }
    if (gridDim.x > 1) {
        __syncthreads();
        for (int e = threadIdx.x; e < a.E; e += blockDim.x)
            a.hist[(int64_t)blockIdx.x * a.E + e] = cnt[e];
        ptx::grid_dep_launch();
        return;
    }
    ptx::grid_dep_launch();
    expert_prefix(cnt, base, a.E, total);
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) a.counts[e] = cnt[e];
    place_pairs(a, a.ids, 0, a.T * a.k, base, wh, *total);
}

// More than one block of tokens: the places, from every block's counts.
__global__ void __launch_bounds__(kWarps * 32) route_order_kernel(RouteArgs a, int blocks) {
    extern __shared__ int32_t sm[];
    int32_t *cnt = sm, *base = sm + a.E, *total = sm + 2 * a.E, *wh = sm + 2 * a.E + 1;
    int32_t *before = wh + kWarps * a.E;  // pairs of expert e in earlier blocks
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) cnt[e] = before[e] = 0;
    __syncthreads();
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    // whole sums: the order of the additions does not matter
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = lane; e < a.E; e += 32) {
        int s = 0, p = 0;
        for (int b = warp; b < blocks; b += kWarps) {
            const int c = __ldcg(a.hist + (int64_t)b * a.E + e);
            s += c;
            if (b < (int)blockIdx.x) p += c;
        }
        atomicAdd(&cnt[e], s);
        atomicAdd(&before[e], p);
    }
    expert_prefix(cnt, base, a.E, total);
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        if (blockIdx.x == 0) a.counts[e] = cnt[e];
        base[e] += before[e];
    }
    __syncthreads();
    const int t0 = blockIdx.x * kTokensPerBlock, t1 = min(a.T, t0 + kTokensPerBlock);
    place_pairs(a, a.ids, (int64_t)t0 * a.k, (t1 - t0) * a.k, base, wh, *total);
}

template <int NV, int K>
cudaError_t launch_nv(const RouteArgs &a, bool bf16, int blocks, int threads, size_t smem,
                      cudaStream_t s) {
    return bf16 ? launch_programmatic_smem(route_kernel<NV, K, true>, dim3(blocks), dim3(threads), smem, s, a)
                : launch_programmatic_smem(route_kernel<NV, K, false>, dim3(blocks), dim3(threads), smem, s, a);
}

}  // namespace

int route_blocks(int64_t T) { return (int)((T + kTokensPerBlock - 1) / kTokensPerBlock); }

cudaError_t launch_moe_route(const void *logits, int bf16, int64_t ld, int32_t T, int32_t E, int32_t k,
                             int32_t score, float scale, int32_t *ids, float *weights,
                             int32_t *counts, int32_t *rows, int32_t *slots, int32_t *hist,
                             cudaStream_t s) {
    const RouteArgs a{logits, ld, T, E, k, score, scale, ids, weights, counts, rows, slots, hist};
    const int blocks = route_blocks(T);
    const size_t smem = (size_t)(2 * E + 1 + kWarps * E) * 4;  // E <= 256: 34 KB
    cudaError_t e;
    if (T > kQuadTokens && E <= 64) {
        const int threads = (int)((T < kTokensPerBlock ? T : kTokensPerBlock) * 4 + 31) / 32 * 32;
        if (E <= 32)
            e = k <= 8 ? launch_nv<8, 8>(a, bf16 != 0, blocks, threads, smem, s)
                       : launch_nv<8, 16>(a, bf16 != 0, blocks, threads, smem, s);
        else
            e = k <= 8 ? launch_nv<16, 8>(a, bf16 != 0, blocks, threads, smem, s)
                       : launch_nv<16, 16>(a, bf16 != 0, blocks, threads, smem, s);
    } else {
        const int threads = 32 * (T < kWarps ? T : kWarps);
        if (E <= 32)
            e = launch_nv<1, 0>(a, bf16 != 0, blocks, threads, smem, s);
        else if (E <= 64)
            e = launch_nv<2, 0>(a, bf16 != 0, blocks, threads, smem, s);
        else if (E <= 128)
            e = launch_nv<4, 0>(a, bf16 != 0, blocks, threads, smem, s);
        else
            e = launch_nv<8, 0>(a, bf16 != 0, blocks, threads, smem, s);
    }
    if (e != cudaSuccess || rows == nullptr || blocks == 1) return e;
    return launch_programmatic_smem(route_order_kernel, dim3(blocks), dim3(kWarps * 32),
                                    smem + (size_t)E * 4, s, a, blocks);
}

}  // namespace fp8g
