// A whole mixture-of-experts layer for a few tokens, and the packing of
// weight scales it takes.
//
//   xq = Q(x)                        E4M3, 1x32 power-of-two scales
//   g, u = xq W13[e]^T               fp32, e = ids[t, j]
//   hq = Q(act(g) u)                 act and product in fp32
//   out[t] = sum_j w[t, j] hq W2[e]^T   fp32 sum over j in order, one rounding
//
// Four launches, each overlapping the start of the next (programmatic
// launches): prepare (routing tables, tokens quantised in expert order), the
// two streaming products (stream.cu), combine.  The weights of the chosen
// experts are read once; everything else is a few hundred kilobytes.
#include <cuda_bf16.h>

#include "internal.h"
#include "kernel_common.cuh"
#include "quant_math.cuh"
#include "stream.h"

namespace fp8g {

namespace {

constexpr int kPrepThreads = 512;
constexpr int kMaxPairs = 8192;  // T k
constexpr int kMaxExperts = 256;

struct PrepArgs {
    const void *x;
    const int32_t *ids;
    int32_t T, k, E, H;
    int32_t nb;        // tokens per group
    int32_t ks;        // 128-wide K steps of x
    uint8_t *xq;       // [T k][H] codes, expert order
    uint8_t *xsf;      // [group][ks][512]
    int32_t *pos;      // [T k] row in expert order, -1: not routed
    int32_t *cnt;      // counters of both products
    int32_t n_cnt;
    unsigned int *status;
};

// Block t: token t.  Every block derives the routing tables it needs from the
// ids itself (a few thousand integers at most), as the products' CTAs do.
template <bool BF16>
__global__ void __launch_bounds__(kPrepThreads) moe_prep_kernel(PrepArgs a) {
    __shared__ int16_t id[kMaxPairs];
    __shared__ int32_t cnt[kMaxExperts], off[kMaxExperts], goff[kMaxExperts];
    __shared__ int32_t my_row[16], my_tile[16], my_in[16];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int R = a.T * a.k, t = blockIdx.x;
    for (int e = tid; e < a.E; e += kPrepThreads) cnt[e] = 0;
    __syncthreads();
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    for (int i = tid; i < R; i += kPrepThreads) {
        int e = __ldg(a.ids + i);
        if (e >= a.E) {
            if (t == 0 && atomicCAS(&a.status[0], 0u, (unsigned)FP8G_ERR_INVALID_ARG) == 0u)
                atomicExch(&a.status[1], (unsigned)i);
            e = -1;
        }
        if (e < 0) e = -1;
        id[i] = (int16_t)e;
        if (e >= 0) atomicAdd(&cnt[e], 1);
    }
    for (int i = t * kPrepThreads + tid; i < a.n_cnt; i += gridDim.x * kPrepThreads) a.cnt[i] = 0;
    __syncthreads();
    if (warp == 0) {  // exclusive prefixes over experts: rows, groups
        int rr = 0, gg = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane;
            const int c = e < a.E ? cnt[e] : 0;
            const int ng = (c + a.nb - 1) / a.nb;
            int s = c, sg = ng;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, s, o), vg = __shfl_up_sync(0xffffffffu, sg, o);
                if (lane >= o) {
                    s += v;
                    sg += vg;
                }
            }
            if (e < a.E) {
                off[e] = rr + s - c;
                goff[e] = gg + sg - ng;
            }
            rr += __shfl_sync(0xffffffffu, s, 31);
            gg += __shfl_sync(0xffffffffu, sg, 31);
        }
    }
    __syncthreads();
    // this token's places: the pairs before it with the same expert
    for (int j = warp; j < a.k; j += kPrepThreads / 32) {
        const int i = t * a.k + j, e = id[i];
        int before = 0;
        if (e >= 0)
            for (int o = lane; o < i; o += 32) before += id[o] == e;
        before = __reduce_add_sync(0xffffffffu, before);
        if (lane == 0) {
            my_row[j] = e >= 0 ? off[e] + before : -1;
            my_tile[j] = e >= 0 ? goff[e] + before / a.nb : 0;
            my_in[j] = before % a.nb;
            a.pos[i] = my_row[j];
        }
    }
    __syncthreads();
    // quantise: thread c takes values 8c .. 8c + 7, four threads a block; K
    // groups past H (the last step's tail) get scale 1
    const int groups = a.ks * 16;
    for (int c0 = 0; c0 < groups; c0 += kPrepThreads) {
        const int c = c0 + tid;
        float4 v0 = make_float4(0.f, 0.f, 0.f, 0.f), v1 = v0;
        const bool in = c * 8 < a.H;
        if (in) load8<BF16>(a.x, (int64_t)t * a.H + c * 8, v0, v1);
        float am = absmax8(v0, v1);
        am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
        am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
        const float s = pow2_scale<0>(am);
        const uint2 q = quant8_pow2<0>(v0, v1, s);
        const int kg = c >> 4, b = (c >> 2) & 3;
        for (int j = 0; j < a.k; ++j) {
            const int row = my_row[j];
            if (row < 0 || c >= groups) continue;
            if (in) *reinterpret_cast<uint2 *>(a.xq + (int64_t)row * a.H + c * 8) = q;
            if ((c & 3) == 0)
                a.xsf[((int64_t)my_tile[j] * a.ks + kg) * 512 + 16 * (my_in[j] & 31) +
                      4 * (my_in[j] >> 5) + b] = (uint8_t)(__float_as_uint(s) >> 23);
        }
    }
}

// out[t, h] = sum_j w[t, j] y[pos[t, j], h], j in order; four values a thread.
template <bool F32>
__global__ void __launch_bounds__(256) moe_combine_kernel(const float *__restrict__ y,
                                                          const int32_t *__restrict__ pos,
                                                          const float *__restrict__ w, int32_t k,
                                                          int32_t H, void *__restrict__ out) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int t = blockIdx.y, h = (blockIdx.x * 256 + threadIdx.x) * 4;
    if (h >= H) return;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < k; ++j) {
        const int r = __ldcg(pos + t * k + j);
        if (r < 0) continue;
        const float c = __ldg(w + t * k + j);
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(y + (int64_t)r * H + h));
        s.x = fmaf(c, v.x, s.x);
        s.y = fmaf(c, v.y, s.y);
        s.z = fmaf(c, v.z, s.z);
        s.w = fmaf(c, v.w, s.w);
    }
    const int64_t at = (int64_t)t * H + h;
    if constexpr (F32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(out) + at) = s;
    } else {
        __nv_bfloat162 lo = __floats2bfloat162_rn(s.x, s.y), hi = __floats2bfloat162_rn(s.z, s.w);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(out) + at) =
            make_uint2(*reinterpret_cast<uint32_t *>(&lo), *reinterpret_cast<uint32_t *>(&hi));
    }
}

bool is_aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool packed(int f) { return f == FP8G_E2M1 || f == FP8G_E2M3 || f == FP8G_E3M2; }
constexpr int64_t kMaxDim = (int64_t)1 << 31;

int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

}  // namespace

}  // namespace fp8g

using namespace fp8g;

extern "C" {

int64_t fp8g_packed_scale_bytes(int64_t matrices, int64_t rows, int64_t K) {
    if (matrices < 1 || rows < 1 || K < 1 || matrices >= kMaxDim || rows >= kMaxDim || K >= kMaxDim)
        return 0;
    const int64_t per = ((rows + 127) / 128) * ((K + 127) / 128);
    if (per > ((int64_t)1 << 50) / matrices) return 0;
    return matrices * per * 512;
}

fp8g_status fp8g_pack_scales(const float *sf, int64_t matrices, int64_t rows, int64_t K,
                             uint8_t *packed_sf, cudaStream_t stream) {
    if (sf == nullptr || packed_sf == nullptr) return FP8G_ERR_INVALID_ARG;
    if (matrices < 1 || rows < 1 || K < 1) return FP8G_ERR_INVALID_ARG;
    if (K % 32 != 0) return FP8G_ERR_UNSUPPORTED_SHAPE;
    const int64_t n_rt = (rows + 127) / 128;
    if (matrices > 65535 || n_rt > 65535 || K >= kMaxDim) return FP8G_ERR_UNSUPPORTED_SHAPE;
    if (!is_aligned(sf, 16) || !is_aligned(packed_sf, 16)) return FP8G_ERR_ALIGNMENT;
    HostDevice d;
    const fp8g_status st = host_device(d);
    if (st != FP8G_OK) return st;
    const PackArgs none{nullptr, 0, 0, 0, 0, nullptr, nullptr, 0};
    const PackArgs b{sf, rows, rows, (int32_t)n_rt, (int32_t)matrices, packed_sf, nullptr, 0};
    const cudaError_t e = launch_pack_scales(none, b, K / 32, (int32_t)((K + 127) / 128), 0, d.status,
                                             stream);
    return e == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}

fp8g_status fp8g_moe_route(const void *logits, int32_t in_dtype, int64_t ld, int64_t T, int32_t E,
                           int32_t k, int32_t score, float scale, int32_t *ids, float *weights,
                           int32_t *counts, int32_t *rows, int32_t *slots, cudaStream_t stream) {
    if (in_dtype != FP8G_IN_F32 && in_dtype != FP8G_IN_BF16) return FP8G_ERR_INVALID_ARG;
    if (score < FP8G_SCORE_SOFTMAX || score > FP8G_SCORE_SIGMOID_NORM) return FP8G_ERR_INVALID_ARG;
    if (T < 0 || E < 1 || k < 1 || k > E || ld < E) return FP8G_ERR_INVALID_ARG;
    if (E > FP8G_MAX_ROUTED_EXPERTS || k > FP8G_MAX_TOP_K || T > FP8G_MAX_ROUTED_TOKENS)
        return FP8G_ERR_UNSUPPORTED_SHAPE;
    const bool ordered = counts != nullptr;
    if ((rows != nullptr) != ordered || (slots != nullptr) != ordered) return FP8G_ERR_INVALID_ARG;
    if (T > 0 && (logits == nullptr || ids == nullptr || weights == nullptr)) return FP8G_ERR_INVALID_ARG;
    if (!is_aligned(logits, in_dtype == FP8G_IN_BF16 ? 2 : 4) || !is_aligned(ids, 4) ||
        !is_aligned(weights, 4) || !is_aligned(counts, 4) || !is_aligned(rows, 4) || !is_aligned(slots, 4))
        return FP8G_ERR_ALIGNMENT;
    HostDevice d;
    fp8g_status st = host_device(d);
    if (st != FP8G_OK) return st;
    if (T == 0) {
        if (ordered && cudaMemsetAsync(counts, 0, (size_t)E * 4, stream) != cudaSuccess)
            return FP8G_ERR_CUDA;
        return FP8G_OK;
    }
    void *hist = nullptr;
    if (ordered && route_blocks(T) > 1) {
        cudaMemPool_t pool;
        if ((st = host_pool(d.dev, pool)) != FP8G_OK) return st;
        if (cudaMallocFromPoolAsync(&hist, (size_t)route_blocks(T) * E * 4, pool, stream) != cudaSuccess)
            return FP8G_ERR_CUDA;
    }
    const cudaError_t e = launch_moe_route(logits, in_dtype == FP8G_IN_BF16, ld, (int32_t)T, E, k, score,
                                           scale, ids, weights, counts, rows, slots,
                                           static_cast<int32_t *>(hist), stream);
    const cudaError_t ef = hist != nullptr ? cudaFreeAsync(hist, stream) : cudaSuccess;
    return e == cudaSuccess && ef == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}

fp8g_status fp8_moe_layer(const void *x, int32_t x_dtype, const int32_t *ids, const float *weights,
                          const void *W13, const uint8_t *sf13, const void *W2, const uint8_t *sf2,
                          void *out, int out_dtype, int32_t w_fmt, int32_t gate, int64_t T, int32_t k,
                          int32_t E, int64_t H, int64_t F, cudaStream_t stream) {
    if (x_dtype != FP8G_IN_F32 && x_dtype != FP8G_IN_BF16) return FP8G_ERR_INVALID_ARG;
    if (out_dtype != FP8G_OUT_BF16 && out_dtype != FP8G_OUT_F32) return FP8G_ERR_INVALID_ARG;
    if (w_fmt < FP8G_E4M3 || w_fmt > FP8G_E3M2) return FP8G_ERR_INVALID_ARG;
    if (gate < FP8G_GATE_SILU || gate > FP8G_GATE_RELU) return FP8G_ERR_INVALID_ARG;
    if (T < 0 || k < 1 || E < 1 || H < 1 || F < 1) return FP8G_ERR_INVALID_ARG;
    if (W13 == nullptr || sf13 == nullptr || W2 == nullptr || sf2 == nullptr) return FP8G_ERR_INVALID_ARG;
    if (T > 0 && (x == nullptr || ids == nullptr || weights == nullptr || out == nullptr))
        return FP8G_ERR_INVALID_ARG;
    const int64_t unit = packed(w_fmt) ? 128 : 32;
    if (H % unit != 0 || F % unit != 0) return FP8G_ERR_UNSUPPORTED_SHAPE;
    if (T > FP8G_MOE_MAX_TOKENS || k > FP8G_MAX_TOP_K || E > FP8G_MAX_ROUTED_EXPERTS ||
        H >= (1 << 24) || F >= (1 << 24))
        return FP8G_ERR_UNSUPPORTED_SHAPE;
    const uintptr_t wal = packed(w_fmt) ? 32 : 16;
    if (!is_aligned(x, 16) || !is_aligned(out, 16) || !is_aligned(W13, wal) || !is_aligned(W2, wal) ||
        !is_aligned(sf13, 16) || !is_aligned(sf2, 16) || !is_aligned(ids, 4) || !is_aligned(weights, 4))
        return FP8G_ERR_ALIGNMENT;
    HostDevice d;
    fp8g_status st = host_device(d);
    if (st != FP8G_OK) return st;
    if (T == 0) return FP8G_OK;

    const int R = (int)(T * k), nb = (int)(T < kStreamMaxTokens ? round_up(T, 16) : kStreamMaxTokens);
    // groups: each expert's rows in tiles of nb
    const int max_groups = (int)((E < R ? E : R) + R / nb);
    StreamParams p1{}, p2{};
    stream_sizes(p1, nb, 1);
    stream_sizes(p2, nb, 1);
    p1.mt = (int32_t)((F + 127) / 128);
    p1.ks = (int32_t)((H + 127) / 128);
    p1.rows = (int32_t)F;
    p1.n_rt = p1.mt;
    p2.mt = (int32_t)((H + 255) / 256);
    p2.ks = p1.mt;
    p2.rows = (int32_t)H;
    p2.n_rt = p1.ks;
    const int64_t units1 = (int64_t)p1.mt * p1.ks, units2 = (int64_t)p2.mt * p2.ks;
    if (max_groups > kStreamMaxGroups || units1 * max_groups >= INT32_MAX ||
        units2 * max_groups >= INT32_MAX)
        return FP8G_ERR_UNSUPPORTED_SHAPE;

    // one temporary: [codes x][scales x][codes h][scales h][y][partials][tables]
    size_t at = 0;
    auto take = [&at](size_t bytes) {
        const size_t o = at;
        at += (bytes + 1023) / 1024 * 1024;
        return o;
    };
    const size_t o_xq = take((size_t)R * H), o_xsf = take((size_t)max_groups * p1.ks * 512);
    const size_t o_hq = take((size_t)R * F), o_hsf = take((size_t)max_groups * p1.mt * 512);
    const size_t o_y = take((size_t)R * H * 4), o_part = take(stream_part_bytes(p1, d.num_sms));
    const int n_cnt = max_groups * (p1.mt + p2.mt);
    const size_t o_cnt = take((size_t)n_cnt * 4), o_pos = take((size_t)R * 4);
    cudaMemPool_t pool;
    if ((st = host_pool(d.dev, pool)) != FP8G_OK) return st;
    void *wsv = nullptr;
    if (cudaMallocFromPoolAsync(&wsv, at, pool, stream) != cudaSuccess) return FP8G_ERR_CUDA;
    uint8_t *ws = static_cast<uint8_t *>(wsv);

    CUtensorMap m13, m2, mx, mh;
    {
        const uint32_t bw[3] = {(uint32_t)kBK, 128u, 1u}, bx[2] = {(uint32_t)kBK, 16u};
        const uint64_t d13[3] = {(uint64_t)H, (uint64_t)F, (uint64_t)(2 * E)};
        const uint64_t d2[3] = {(uint64_t)F, (uint64_t)H, (uint64_t)E};
        const uint64_t dx[2] = {(uint64_t)H, (uint64_t)R}, dh[2] = {(uint64_t)F, (uint64_t)R};
        st = host_operand_map(W13, w_fmt, 3, d13, bw, d.dev, m13);
        if (st == FP8G_OK) st = host_operand_map(W2, w_fmt, 3, d2, bw, d.dev, m2);
        if (st == FP8G_OK) st = host_operand_map(ws + o_xq, FP8G_E4M3, 2, dx, bx, d.dev, mx);
        if (st == FP8G_OK) st = host_operand_map(ws + o_hq, FP8G_E4M3, 2, dh, bx, d.dev, mh);
    }
    cudaError_t e = st == FP8G_OK ? cudaSuccess : cudaErrorInvalidValue;
    int32_t *cnt = reinterpret_cast<int32_t *>(ws + o_cnt);
    int32_t *pos = reinterpret_cast<int32_t *>(ws + o_pos);
    if (e == cudaSuccess) {
        PrepArgs a{};
        a.x = x;
        a.ids = ids;
        a.T = (int32_t)T;
        a.k = k;
        a.E = E;
        a.H = (int32_t)H;
        a.nb = nb;
        a.ks = p1.ks;
        a.xq = ws + o_xq;
        a.xsf = ws + o_xsf;
        a.pos = pos;
        a.cnt = cnt;
        a.n_cnt = n_cnt;
        a.status = d.status;
        e = x_dtype == FP8G_IN_BF16
                ? launch_programmatic(moe_prep_kernel<true>, dim3((unsigned)T), dim3(kPrepThreads), stream, a)
                : launch_programmatic(moe_prep_kernel<false>, dim3((unsigned)T), dim3(kPrepThreads), stream,
                                      a);
    }
    for (StreamParams *p : {&p1, &p2}) {
        p->w_fmt = host_mma_type(w_fmt) << 7;
        p->gap8 = host_gap8(w_fmt);
        p->idx = ids;
        p->n_idx = R;
        p->n_mat = E;
        p->part = reinterpret_cast<float *>(ws + o_part);
        p->status = d.status;
        p->timeout_ns = d.timeout_ns;
    }
    p1.sfw = sf13;
    p1.sfx = ws + o_xsf;
    p1.tile_cnt = cnt;
    p1.gate = gate;
    p1.hq = ws + o_hq;
    p1.hsf = ws + o_hsf;
    p2.sfw = sf2;
    p2.sfx = ws + o_hsf;
    p2.tile_cnt = cnt + (size_t)max_groups * p1.mt;
    p2.y = reinterpret_cast<float *>(ws + o_y);
    if (e == cudaSuccess) e = launch_stream(kStreamGated, m13, mx, mx, mx, p1, d.num_sms, stream);
    if (e == cudaSuccess) e = launch_stream(kStreamRows, m2, mh, mh, mh, p2, d.num_sms, stream);
    if (e == cudaSuccess) {
        const dim3 grid((unsigned)((H / 4 + 255) / 256), (unsigned)T);
        e = out_dtype == FP8G_OUT_F32
                ? launch_programmatic(moe_combine_kernel<true>, grid, dim3(256), stream, p2.y, pos, weights,
                                      k, (int32_t)H, out)
                : launch_programmatic(moe_combine_kernel<false>, grid, dim3(256), stream, p2.y, pos, weights,
                                      k, (int32_t)H, out);
    }
    const cudaError_t ef = cudaFreeAsync(wsv, stream);
    if (st != FP8G_OK) return st;
    return e == cudaSuccess && ef == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}

}  // extern "C"
