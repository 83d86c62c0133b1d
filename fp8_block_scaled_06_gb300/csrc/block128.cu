// Entry points of the operators with fp32 scales for blocks of 128: argument
// checks, tensor maps, the choice between the kernel for few rows
// (block128_few.cu) and the one on CTA pairs (block128_gemm.cu).
#include <algorithm>

#include "block128.h"

namespace fp8g {

namespace {

bool is_aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool fp8_fmt(int f) { return f == FP8G_E4M3 || f == FP8G_E5M2; }
int64_t blocks(int64_t n) { return (n + kBlk - 1) / kBlk; }
constexpr int64_t kMaxDim = (int64_t)1 << 31;
constexpr int64_t kMaxQuantRows = (int64_t)65535 * 16;  // 16 rows at least a block: a grid's second axis

// How T tiles of num_kb K blocks go to `most` CTA pairs: rounds of whole tiles and, where
// the last would leave pairs idle, its K blocks in shares, a tile's to four pairs at
// most (the one with its end adds the others' sums, 256 KB each), by a kernel of their own:
// in one kernel, pairs whose shares differ read the rounds' operands at different times,
// and L2 served fewer (4099 x 4096 x 28672 372 us in place of 330).
// Shares cost the time of about 50 K blocks (writing and adding sums, zeroing flags, the gap
// between kernels): taken where they save 60.  Measured, us, with / without: saving 20 (4096 x
// 4096 x 4096) 69 / 58, 47 (4099 x 4096 x 14336) 178 / 175, 94 (4099 x 4096 x 28672) 330 / 346;
// weight gradient of 1024 x 1024 x 16384 43 / 75.
struct Deal {
    int64_t whole;  // tiles
    int32_t share;  // K blocks of a pair of the others (0: there are none)
    int64_t units;  // K blocks one after the other
};
Deal deal(int64_t T, int num_kb, int most, bool can_share) {
    const int64_t full = T / most, rest = T - full * most;
    Deal d{T, 0, (T + most - 1) / most * num_kb};
    if (rest == 0 || !can_share) return d;
    int64_t share = (rest * num_kb + most - 1) / most;
    if (share < (num_kb + 3) / 4) share = (num_kb + 3) / 4;
    if (num_kb - share < 60) return d;
    return Deal{full * most, (int32_t)share, full * num_kb + share + 50};
}

// Which kernel, and its shape.
struct Plan {
    bool few;
    int nt, split;  // few: rows of A of a tile, CTAs that share its K blocks
};

// The kernel for few rows against the one on CTA pairs, by estimates of their time.
// In units of about 10 cycles: pairs take 76 a K block (every tile 256 x 256, however few of
// its rows exist; 725 cycles when nothing else holds them up), the call eight K blocks more at
// its ends.  Few rows: a tile of 128 weight rows; a round begins and ends with the time of five
// K blocks (first loads, joining), of fifteen if another comes before it, each further CTA of a
// tile joins about one more; a K block takes 100 where a CTA has its SM alone, 130 where two
// share it (loads bound both).  A cluster stays in one GPC, so fewer run at once than its
// SMs would give (1, 2, .. 8 CTAs, an SM each: 152, 76, 46, 36, 28, 23, 15, 15); with two
// CTAs an SM it has half the SMs, or twice as many run.
// Measured, us, few rows / pairs: 64 x 14336 x 4096 14.5 / 17, 77 of them 20 / 17, 77 x
// 4096 x 14336 18 / 29, 256 of them 28 / 30; gated, 64 rows of F 14336, K 4096 24 / 33,
// 128 rows 47 / 34.  By CTAs of a tile: 77 x 5120 x 5120 2, 3, 4: 14.6, 12.0, 18.6; 64 x 28672
// x 8192 1, 2, 4: 43, 51, 56.
Plan plan(int64_t M, int64_t n_blocks, const Deal &d, int num_kb, bool gated, int dev) {
    int64_t least = (d.units + 8) * 76;
    Plan best{false, kBlk, 1};
    const int most = gated ? 64 : 128;
    int nt = 16;
    while (nt < most && nt < M) nt *= 2;
    const int64_t tiles = n_blocks * ((M + nt - 1) / nt);
    const int per_sm = nt < most ? 2 : 1;
    if (M > 65535 * 16) return best;  // (a grid's second axis)
    for (int s = 1; s <= 8 && s <= num_kb; ++s) {
        int64_t fit = per_sm * b128_few_clusters(s, dev);
        if (per_sm == 2) fit = std::max<int64_t>(fit, b128_few_clusters((s + 1) / 2, dev));
        if (fit == 0) continue;
        const int64_t r = (tiles + fit - 1) / fit;
        const int64_t cost = (r * ((num_kb + s - 1) / s + 10) - 5 + s) * (per_sm == 1 ? 100 : 130);
        if (cost < least) {
            least = cost;
            best = Plan{true, nt, s};
        }
    }
    return best;
}

// The kernels on CTA pairs: whole tiles, then the others in shares with a temporary for sums
// (its flags are zeroed before both, so that nothing is between them).
fp8g_status run_pairs(const B128Maps &m, B128Params &p, const Deal &dl, int out, bool vec_b, const HostDevice &d,
                      cudaStream_t stream) {
    const int32_t T = p.T, most = d.num_sms / 2;
    p.T = (int32_t)dl.whole;
    p.pairs = std::min(p.T, most);
    if (dl.share == 0) return launch_b128_pair(m, p, out, vec_b, stream) == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
    B128Params q = p;
    q.first = p.T;
    q.T = T;
    q.share = dl.share;
    q.pairs = ((q.T - q.first) * q.num_kb + q.share - 1) / q.share;
    cudaMemPool_t pool;
    const fp8g_status st = host_pool(d.dev, pool);
    if (st != FP8G_OK) return st;
    void *ws = nullptr;
    const size_t sums = (size_t)q.pairs * kB128PartBytes, flags = ((size_t)q.pairs * 16 + 1) * 4;
    if (cudaMallocFromPoolAsync(&ws, sums + flags, pool, stream) != cudaSuccess) return FP8G_ERR_CUDA;
    q.part = static_cast<float *>(ws);
    q.there = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(ws) + sums);
    cudaError_t e = cudaMemsetAsync(q.there, 0, flags, stream);
    if (e == cudaSuccess && p.T > 0) e = launch_b128_pair(m, p, out, vec_b, stream);
    if (e == cudaSuccess) e = launch_b128_share(m, q, out, vec_b, stream);
    const cudaError_t ef = cudaFreeAsync(ws, stream);
    return e == cudaSuccess && ef == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}

fp8g_status map2(const void *ptr, int64_t inner, int64_t outer, int rows, int dev, CUtensorMap &m) {
    const uint64_t d[2] = {(uint64_t)inner, (uint64_t)outer};
    const uint32_t b[2] = {(uint32_t)kBlk, (uint32_t)rows};
    return host_operand_map(ptr, FP8G_E4M3, 2, d, b, dev, m);  // (one-byte elements)
}

fp8g_status check_quant(const void *x, int64_t rows, int64_t cols, int64_t ld, int esz, int fmt) {
    if (!fp8_fmt(fmt) || rows < 0 || cols < 1 || ld < cols) return FP8G_ERR_INVALID_ARG;
    if (rows > 0 && x == nullptr) return FP8G_ERR_INVALID_ARG;
    if (cols % 16 != 0 || rows > kMaxQuantRows || cols >= kMaxDim || ld >= ((int64_t)1 << 40))
        return FP8G_ERR_UNSUPPORTED_SHAPE;
    if (!is_aligned(x, 16) || ld * esz % 16 != 0) return FP8G_ERR_ALIGNMENT;
    return FP8G_OK;
}

fp8g_status run_quant(const B128Quant &a, int fmt, cudaStream_t stream) {
    HostDevice d;
    const fp8g_status st = host_device(d);
    if (st != FP8G_OK || a.R == 0) return st;
    return launch_b128_quant(a, fmt, stream) == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}

}  // namespace

}  // namespace fp8g

using namespace fp8g;

extern "C" {

fp8g_status fp8g_quantize_block128(const void *x, int32_t in_dtype, int64_t ld, int64_t rows, int64_t cols,
                                   int32_t fmt, uint8_t *q_row, float *s_row, uint8_t *q_col, float *s_col,
                                   cudaStream_t stream) {
    if (in_dtype != FP8G_IN_F32 && in_dtype != FP8G_IN_BF16) return FP8G_ERR_INVALID_ARG;
    if ((q_row == nullptr) != (s_row == nullptr) || (q_col == nullptr) != (s_col == nullptr))
        return FP8G_ERR_INVALID_ARG;
    if (q_row == nullptr && q_col == nullptr && rows != 0) return FP8G_ERR_INVALID_ARG;
    const fp8g_status st = check_quant(x, rows, cols, ld, in_dtype == FP8G_IN_BF16 ? 2 : 4, fmt);
    if (st != FP8G_OK) return st;
    if (!is_aligned(q_row, 16) || !is_aligned(s_row, 16) || !is_aligned(q_col, 16) || !is_aligned(s_col, 16))
        return FP8G_ERR_ALIGNMENT;
    const B128Quant a{x, ld, rows, cols, in_dtype, 0, nullptr, q_row, q_col, nullptr, s_row, s_col, nullptr};
    return run_quant(a, fmt, stream);
}

fp8g_status fp8g_quantize_tile128(const void *x, int32_t in_dtype, int64_t ld, int64_t rows, int64_t cols,
                                  int32_t fmt, uint8_t *q, float *s, cudaStream_t stream) {
    if (in_dtype != FP8G_IN_F32 && in_dtype != FP8G_IN_BF16) return FP8G_ERR_INVALID_ARG;
    if (rows != 0 && (q == nullptr || s == nullptr)) return FP8G_ERR_INVALID_ARG;
    const fp8g_status st = check_quant(x, rows, cols, ld, in_dtype == FP8G_IN_BF16 ? 2 : 4, fmt);
    if (st != FP8G_OK) return st;
    if (!is_aligned(q, 16) || !is_aligned(s, 16)) return FP8G_ERR_ALIGNMENT;
    const B128Quant a{x, ld, rows, cols, in_dtype, 0, nullptr, nullptr, nullptr, q, nullptr, nullptr, s};
    return run_quant(a, fmt, stream);
}

fp8g_status fp8g_requantize_block128(const uint8_t *q, int32_t q_fmt, const float *s, int64_t rows, int64_t cols,
                                     int32_t fmt, uint8_t *q_col, float *s_col, cudaStream_t stream) {
    if (!fp8_fmt(q_fmt)) return FP8G_ERR_INVALID_ARG;
    if (rows != 0 && (s == nullptr || q_col == nullptr || s_col == nullptr || q_col == q)) return FP8G_ERR_INVALID_ARG;
    const fp8g_status st = check_quant(q, rows, cols, cols, 1, fmt);
    if (st != FP8G_OK) return st;
    if (!is_aligned(s, 16) || !is_aligned(q_col, 16) || !is_aligned(s_col, 16)) return FP8G_ERR_ALIGNMENT;
    const B128Quant a{q, cols, rows, cols, kB128Codes, q_fmt, s, nullptr, q_col, nullptr, nullptr, s_col, nullptr};
    return run_quant(a, fmt, stream);
}

fp8g_status fp8_gemm_block128(int32_t form, const void *A, const float *sfa, int32_t a_fmt, const void *B,
                              const float *sfb, int32_t b_fmt, void *C, int out, int32_t add, int64_t M, int64_t N,
                              int64_t K, cudaStream_t stream) {
    if (form != FP8G_NT && form != FP8G_NN && form != FP8G_TN) return FP8G_ERR_INVALID_ARG;
    if (!fp8_fmt(a_fmt) || !fp8_fmt(b_fmt)) return FP8G_ERR_INVALID_ARG;
    if (out != FP8G_OUT_BF16 && out != FP8G_OUT_F32) return FP8G_ERR_INVALID_ARG;
    if (add != 0 && (add != 1 || out != FP8G_OUT_F32)) return FP8G_ERR_INVALID_ARG;
    const bool tn = form == FP8G_TN;
    if (M < 0 || N < 1 || K < 0 || (tn ? M < 1 : K < 1)) return FP8G_ERR_INVALID_ARG;
    if (M > 0 && C == nullptr) return FP8G_ERR_INVALID_ARG;
    if (M > 0 && K > 0 && (A == nullptr || sfa == nullptr || B == nullptr || sfb == nullptr))
        return FP8G_ERR_INVALID_ARG;
    if (M >= kMaxDim || N >= kMaxDim || K >= kMaxDim) return FP8G_ERR_UNSUPPORTED_SHAPE;
    const int64_t npm = (M + 2 * kBlk - 1) / (2 * kBlk), npn = (N + 2 * kBlk - 1) / (2 * kBlk);
    if (npm * npn >= kMaxDim / 2) return FP8G_ERR_UNSUPPORTED_SHAPE;
    const int64_t esz = out == FP8G_OUT_F32 ? 4 : 2;
    if ((!tn && K % 16 != 0) || (tn && M % 16 != 0) || (form != FP8G_NT && N % 16 != 0) || N * esz % 16 != 0)
        return FP8G_ERR_ALIGNMENT;
    if (!is_aligned(A, 16) || !is_aligned(B, 16) || !is_aligned(C, 16) || !is_aligned(sfa, 16) || !is_aligned(sfb, 16))
        return FP8G_ERR_ALIGNMENT;
    HostDevice d;
    fp8g_status st = host_device(d);
    if (st != FP8G_OK || M == 0) return st;
    if (K == 0) {  // no rows to sum over
        if (add) return FP8G_OK;
        return cudaMemsetAsync(C, 0, (size_t)(M * N * esz), stream) == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
    }
    B128Params p{};
    p.M = M;
    p.N = N;
    p.K = K;
    p.num_kb = (int32_t)blocks(K);
    p.sa = sfa;
    p.sb = sfb;
    p.n_blocks = (int32_t)blocks(N);
    p.sb_n = form == FP8G_NT ? p.num_kb : 1;
    p.sb_k = form == FP8G_NT ? 1 : p.n_blocks;
    p.a_mn = tn;
    p.b_mn = form != FP8G_NT;
    p.C = C;
    p.status = d.status;
    p.timeout_ns = d.timeout_ns;
    const int o = add ? kB128Add : out == FP8G_OUT_F32 ? kB128F32 : kB128Bf16;
    const uint32_t ta = host_mma_type(a_fmt), tb = host_mma_type(b_fmt);
    const Deal dl = deal(npm * npn, p.num_kb, d.num_sms / 2, true);
    const Plan pl = tn ? Plan{false, kBlk, 1} : plan(M, p.n_blocks, dl, p.num_kb, false, d.dev);
    B128Maps m{};
    st = tn ? map2(A, M, K, kBlk, d.dev, m.A) : map2(A, K, M, pl.nt, d.dev, m.A);
    if (st == FP8G_OK)
        st = p.b_mn ? map2(B, N, K, kBlk, d.dev, m.B) : map2(B, K, N, kBlk, d.dev, m.B);
    if (st == FP8G_OK && !pl.few) st = host_store_map(C, (int)esz, M, N, d.dev, m.C);
    if (st != FP8G_OK) return st;
    if (pl.few) {
        p.types = (tb << 7) | (ta << 10) | ((uint32_t)p.b_mn << 15);
        return launch_b128_few(m.A, m.B, p, o, pl.nt, pl.split, stream) == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
    } else {
        p.types = (ta << 7) | (tb << 10) | ((uint32_t)p.a_mn << 15) | ((uint32_t)p.b_mn << 16);
        p.npm = (int32_t)npm;
        p.npn = (int32_t)npn;
        p.T = (int32_t)(npm * npn);
        return run_pairs(m, p, dl, o, tn, d, stream);
    }
}

fp8g_status fp8_gated_block128(const void *x, const float *sfx, int32_t x_fmt, const void *W13, const float *sf13,
                               int32_t w_fmt, int32_t gate, uint8_t *h, float *sh, uint8_t *gu, float *sgu,
                               int64_t M, int64_t F, int64_t K, cudaStream_t stream) {
    if (!fp8_fmt(x_fmt) || !fp8_fmt(w_fmt)) return FP8G_ERR_INVALID_ARG;
    if (gate < FP8G_GATE_SILU || gate > FP8G_GATE_RELU) return FP8G_ERR_INVALID_ARG;
    if (M < 0 || F < 1 || K < 1) return FP8G_ERR_INVALID_ARG;
    if ((gu == nullptr) != (sgu == nullptr)) return FP8G_ERR_INVALID_ARG;
    if (M > 0 && (x == nullptr || sfx == nullptr || W13 == nullptr || sf13 == nullptr || h == nullptr || sh == nullptr))
        return FP8G_ERR_INVALID_ARG;
    if (F % kBlk != 0 || M >= kMaxDim || 2 * F >= kMaxDim || K >= kMaxDim) return FP8G_ERR_UNSUPPORTED_SHAPE;
    const int64_t npm = (M + 2 * kBlk - 1) / (2 * kBlk);
    if (npm * (F / kBlk) >= kMaxDim / 2) return FP8G_ERR_UNSUPPORTED_SHAPE;
    if (K % 16 != 0 || !is_aligned(x, 16) || !is_aligned(W13, 16) || !is_aligned(h, 16) || !is_aligned(gu, 16) ||
        !is_aligned(sfx, 16) || !is_aligned(sf13, 16) || !is_aligned(sh, 16) || !is_aligned(sgu, 16))
        return FP8G_ERR_ALIGNMENT;
    HostDevice d;
    fp8g_status st = host_device(d);
    if (st != FP8G_OK || M == 0) return st;
    B128Params p{};
    p.M = M;
    p.N = F;
    p.K = K;
    p.num_kb = (int32_t)blocks(K);
    p.sa = sfx;
    p.sb = sf13;
    p.n_blocks = (int32_t)(F / kBlk);
    p.sb_n = p.num_kb;
    p.sb_k = 1;
    p.h = h;
    p.sh = sh;
    p.gu = gu;
    p.sgu = sgu;
    p.status = d.status;
    p.timeout_ns = d.timeout_ns;
    const uint32_t tx = host_mma_type(x_fmt), tw = host_mma_type(w_fmt);
    const Deal dl = deal(npm * p.n_blocks, p.num_kb, d.num_sms / 2, false);
    const Plan pl = plan(M, p.n_blocks, dl, p.num_kb, true, d.dev);
    B128Maps m{};
    st = map2(x, K, M, pl.nt, d.dev, m.A);
    if (st == FP8G_OK) {
        const uint64_t dw[3] = {(uint64_t)K, (uint64_t)F, 2};
        const uint32_t bw[3] = {(uint32_t)kBlk, (uint32_t)kBlk, 1};
        st = host_operand_map(W13, FP8G_E4M3, 3, dw, bw, d.dev, m.B);
    }
    if (st == FP8G_OK && !pl.few) st = host_store_map(h, 1, M, F, d.dev, m.C);
    if (st == FP8G_OK && !pl.few && gu != nullptr) st = host_store_map(gu, 1, M, 2 * F, d.dev, m.gu);
    if (st != FP8G_OK) return st;
    if (pl.few) {
        p.types = (tw << 7) | (tx << 10);
        return launch_b128_few(m.A, m.B, p, kB128Gated + gate, pl.nt, pl.split, stream) == cudaSuccess ? FP8G_OK
                                                                                                    : FP8G_ERR_CUDA;
    } else {
        p.types = (tx << 7) | (tw << 10);
        p.npm = (int32_t)npm;
        p.npn = p.n_blocks;
        p.T = p.npm * p.npn;
        return run_pairs(m, p, dl, kB128Gated + gate, false, d, stream);
    }
}

fp8g_status fp8g_gated_block128_backward(const void *dh, int32_t dh_dtype, const uint8_t *gu, const float *sgu,
                                         int32_t gate, int32_t fmt, int64_t M, int64_t F, uint8_t *dgu_row,
                                         float *s_row, uint8_t *dgu_col, float *s_col, uint8_t *h_col, float *sh_col,
                                         cudaStream_t stream) {
    if (dh_dtype != FP8G_IN_F32 && dh_dtype != FP8G_IN_BF16) return FP8G_ERR_INVALID_ARG;
    if (gate < FP8G_GATE_SILU || gate > FP8G_GATE_RELU || !fp8_fmt(fmt)) return FP8G_ERR_INVALID_ARG;
    if (M < 0 || F < 1) return FP8G_ERR_INVALID_ARG;
    if (M > 0 && (dh == nullptr || gu == nullptr || sgu == nullptr || dgu_row == nullptr || s_row == nullptr ||
                  dgu_col == nullptr || s_col == nullptr || h_col == nullptr || sh_col == nullptr))
        return FP8G_ERR_INVALID_ARG;
    if (F % kBlk != 0 || M > kMaxQuantRows || 2 * F >= kMaxDim ||
        (M + kBlk - 1) / kBlk * (F / kBlk) >= kMaxDim / 2)
        return FP8G_ERR_UNSUPPORTED_SHAPE;
    const void *all[] = {dh, gu, sgu, dgu_row, s_row, dgu_col, s_col, h_col, sh_col};
    for (const void *ptr : all)
        if (!is_aligned(ptr, 16)) return FP8G_ERR_ALIGNMENT;
    HostDevice d;
    const fp8g_status st = host_device(d);
    if (st != FP8G_OK || M == 0) return st;
    const B128Backward a{dh, gu, sgu, M, F, dgu_row, dgu_col, h_col, s_row, s_col, sh_col, d.num_sms};
    return launch_b128_backward(a, dh_dtype == FP8G_IN_BF16, gate, fmt, stream) == cudaSuccess ? FP8G_OK
                                                                                               : FP8G_ERR_CUDA;
}

}  // extern "C"
