// A whole mixture-of-experts layer for a few tokens, and the packing of
// weight scales it takes.
//
//   xq = Q(x)                        E4M3, 1x32 power-of-two scales
//   g, u = xq W13[e]^T               fp32, e = ids[t, j]
//   hq = Q(act(g) u)                 act and product in fp32
//   out[t] = sum_j w[t, j] hq W2[e]^T   fp32 sum over j in order, one rounding
//
// Two launches (stream.cu).  The weights of the chosen experts are read once;
// everything else is a few hundred kilobytes.
#include "stream.h"

namespace fp8g {

namespace {

bool is_aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool packed(int f) { return f == FP8G_E2M1 || f == FP8G_E2M3 || f == FP8G_E3M2; }
constexpr int64_t kMaxDim = (int64_t)1 << 31;

}  // namespace

}  // namespace fp8g

using namespace fp8g;

extern "C" {

int64_t fp8g_packed_scale_bytes(int64_t matrices, int64_t rows, int64_t K) {
    if (matrices < 1 || rows < 1 || K < 1 || K % 32 != 0) return 0;
    if (matrices > 65535 || rows > 65535 * 128 || K >= kMaxDim) return 0;
    return matrices * ((rows + 127) / 128) * ((K + 127) / 128) * 512;
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
    if (T > 0 && ((rows != nullptr) != ordered || (slots != nullptr) != ordered)) return FP8G_ERR_INVALID_ARG;
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
    if (ordered && route_blocks(T, true) > 1) {
        cudaMemPool_t pool;
        if ((st = host_pool(d.dev, pool)) != FP8G_OK) return st;
        // counts of every block of tokens, then ranks of the pairs
        const size_t bytes = (size_t)route_blocks(T, true) * E * 4 + (size_t)T * k;
        if (cudaMallocFromPoolAsync(&hist, bytes, pool, stream) != cudaSuccess)
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

    const int R = (int)(T * k), nb = stream_columns(T);
    // groups: each expert's rows in tiles of nb
    const int max_groups = (int)((E < R ? E : R) + R / nb);
    StreamParams p{};
    stream_sizes(p, nb, 2, false, 1);
    StreamPhase &g = p.ph[0], &dn = p.ph[1];
    g.sub = dn.sub = 2;
    g.mt = (int32_t)((F + 127) / 128);
    g.ks = (int32_t)((H + 127) / 128);
    g.rows = (int32_t)F;
    g.n_rt = g.mt;
    dn.mt = (int32_t)((H + 255) / 256);
    dn.ks = g.mt;
    dn.rows = (int32_t)H;
    dn.n_rt = g.ks;
    if (max_groups > kStreamMaxGroups || (int64_t)max_groups * g.mt * g.ks >= INT32_MAX ||
        (int64_t)max_groups * dn.mt * dn.ks >= INT32_MAX)
        return FP8G_ERR_UNSUPPORTED_SHAPE;

    // one temporary
    size_t at = 0;
    auto take = [&at](size_t bytes) {
        const size_t o = at;
        at += (bytes + 1023) / 1024 * 1024;
        return o;
    };
    const size_t o_xq = take((size_t)R * H), o_xsf = take((size_t)max_groups * g.ks * 512);
    const size_t o_hq = take((size_t)R * F), o_hsf = take((size_t)max_groups * g.mt * 512);
    const size_t o_y = take((size_t)R * H * 4), o_pos = take((size_t)R * 4);
    const size_t o_part0 = take(stream_part_bytes(p, d.num_sms)), o_part1 = take(stream_part_bytes(p, d.num_sms));
    p.n_counters = 3 + max_groups + dn.mt + kStreamSplitTiles;
    const size_t o_cnt = take((size_t)p.n_counters * 4);
    cudaMemPool_t pool;
    if ((st = host_pool(d.dev, pool)) != FP8G_OK) return st;
    void *wsv = nullptr;
    if (cudaMallocFromPoolAsync(&wsv, at, pool, stream) != cudaSuccess) return FP8G_ERR_CUDA;
    uint8_t *ws = static_cast<uint8_t *>(wsv);
    {
        const uint32_t bw[3] = {(uint32_t)kBK, 128u, 1u}, bx[2] = {(uint32_t)kBK, 16u};
        const uint32_t by[2] = {(uint32_t)kBK, 64u};
        const uint64_t d13[3] = {(uint64_t)H, (uint64_t)F, (uint64_t)(2 * E)};
        const uint64_t d2[3] = {(uint64_t)F, (uint64_t)H, (uint64_t)E};
        const uint64_t dx[2] = {(uint64_t)H, (uint64_t)R}, dh[2] = {(uint64_t)F, (uint64_t)R};
        st = host_operand_map(W13, w_fmt, 3, d13, bw, d.dev, g.W);
        if (st == FP8G_OK) st = host_operand_map(W2, w_fmt, 3, d2, bw, d.dev, dn.W);
        if (st == FP8G_OK) st = host_operand_map(ws + o_xq, FP8G_E4M3, 2, dx, bx, d.dev, g.X);
        if (st == FP8G_OK) st = host_operand_map(ws + o_hq, FP8G_E4M3, 2, dh, bx, d.dev, dn.X);
        if (nb % 64 == 0) {
            if (st == FP8G_OK) st = host_operand_map(ws + o_xq, FP8G_E4M3, 2, dx, by, d.dev, g.X64);
            if (st == FP8G_OK) st = host_operand_map(ws + o_hq, FP8G_E4M3, 2, dh, by, d.dev, dn.X64);
        }
    }
    g.sfw = sf13;
    g.sfx = ws + o_xsf;
    dn.sfw = sf2;
    dn.sfx = ws + o_hsf;
    p.w_fmt = host_mma_type(w_fmt) << 7;
    p.gap8 = host_gap8(w_fmt);
    p.x = x;
    p.x_bf16 = x_dtype == FP8G_IN_BF16;
    p.T = (int32_t)T;
    p.K = (int32_t)H;
    p.idx = ids;
    p.n_idx = R;
    p.n_mat = E;
    p.xq = ws + o_xq;
    p.xsf = ws + o_xsf;
    p.counters = reinterpret_cast<int32_t *>(ws + o_cnt);
    p.done_group = p.counters + 3;
    p.done_tile = p.done_group + max_groups;
    g.part = reinterpret_cast<float *>(ws + o_part0);
    g.part_cnt = p.done_tile + dn.mt;
    dn.part = reinterpret_cast<float *>(ws + o_part1);
    p.out = out;
    p.out_f32 = out_dtype == FP8G_OUT_F32;
    p.status = d.status;
    p.timeout_ns = d.timeout_ns;
    p.k = k;
    p.gate = gate;
    p.weights = weights;
    p.pos = reinterpret_cast<int32_t *>(ws + o_pos);
    p.hq = ws + o_hq;
    p.hsf = ws + o_hsf;
    p.y = reinterpret_cast<float *>(ws + o_y);
    const cudaError_t e = st == FP8G_OK ? launch_stream(false, p, d.num_sms, stream) : cudaErrorInvalidValue;
    const cudaError_t ef = cudaFreeAsync(wsv, stream);
    if (st != FP8G_OK) return st;
    return e == cudaSuccess && ef == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}

}  // extern "C"
