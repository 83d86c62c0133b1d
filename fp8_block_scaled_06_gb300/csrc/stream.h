// The streaming kernels (stream.cu): few tokens against block-scaled weights
// that are read once.  Declarations shared by their users (moe.cu, lora.cu).
#pragma once
#include "internal.h"

namespace fp8g {

constexpr int kStreamMaxTokens = 128;    // token rows of a group
constexpr int kStreamMaxGroups = 320;
constexpr int kStreamLoraRows = 512;     // token rows of a call with adapters
constexpr int kStreamLoraGroups = kStreamLoraRows / kStreamMaxTokens;
constexpr int kStreamSplitTiles = 128;   // a product with more tiles is not split (128 x 2 > 152 SMs)

// V = alpha A x of a slot (an adapter of a row tile) as bf16 pieces
// (lora_pieces.cuh): three where the output is fp32, else two.  In a row of 64
// values: three from columns 0, 16 and 32 on (rank up to 16), or two from columns
// 0 and 32 on (up to 32), a third one then in a row of its own: one 64-wide step a
// row.  Higher ranks: each piece in rows of its own, of r64 = rank rounded up to 64,
// r64 / 64 steps.  The first block of the tile's rows first, then the second, the third.
struct LoraV {
    int pieces, per, blocks, r64, kr;  // pieces in a row, blocks of rows, row length, steps per slot
    LoraV(int rank, bool out_f32)
        : pieces(out_f32 ? 3 : 2), per(rank > 32 ? 1 : rank > 16 ? 2 : pieces), blocks((pieces + per - 1) / per),
          r64(per > 1 ? 64 : (rank + 63) / 64 * 64), kr(r64 / 64) {}
};
// Where piece i of a value is from its first one on; block: values of a block of rows.
__host__ __device__ inline int64_t v_piece(int i, int per, int64_t block) {
    if (i == 0) return 0;
    if (i == 1) return per == 1 ? block : per == 2 ? 32 : 16;
    return per == 1 ? 2 * block : per == 2 ? block : 32;
}

// One product: weights [n_mat][rows][K] against a group's token rows.
struct StreamPhase {
    CUtensorMap W, X, X64; // weights (box 128 x 128 rows), token codes (boxes 128 x 16 and 64 rows)
    const uint8_t *sfw;    // packed weight scales [matrix][ks][n_rt][512]
    const uint8_t *sfx;    // packed token scales [group][ks][512]
    int32_t sub;           // 128-row weight tiles of a step: 2 or 1 (gated: gate and up rows)
    int32_t mt;            // tiles of sub * 128 rows (gated: of 128 features)
    int32_t ks;            // 128-wide K steps
    int32_t rows;          // rows of a weight matrix (gated: of each half)
    int32_t n_rt;          // 128-row tiles of packed scales per matrix
    float *part;           // partial tiles [tile][part][2][nb][128]
    int32_t *part_cnt;     // [kStreamSplitTiles] parts done of a tile (not of the down product: done_tile)
};

struct StreamParams {
    StreamPhase ph[2];     // MoE: gate/up and down products; adapters: ph[0]
    int32_t nb;            // token columns of an accumulator (a multiple of 16)
    int32_t nacc, chains, acc_cols;  // accumulators; chains of MMAs in one, its columns
    int32_t stages, stage_bytes, w_bytes, x_bytes;  // shared-memory ring: a stage, its weights, its tokens
    uint32_t w_fmt;        // weight format as MMA instruction-descriptor bits
    int32_t gap8;          // eighths of a weight tile a packed load does not deliver
    const void *x;         // tokens, fp32 or bf16
    int32_t x_bf16;
    int32_t T, K;          // token rows, their length
    int32_t first_row;     // of the call (adapters: it may be taken in shares)
    const int32_t *idx;    // MoE: expert of each pair [T][k]; adapters: adapter of each row [T]
    int32_t n_idx, n_mat;  // their number; experts / adapters
    uint8_t *xq, *xsf;     // token codes (MoE: expert order) and packed scales
    // counters, zeroed by the preparing kernel: [0] the next ticket, [1] the
    // next item of V, [2] items of V done, then (MoE) gated tiles done per group,
    // groups (of split tiles: parts) done per tile of the down product, and the
    // part counters of the first product
    int32_t *counters;
    int32_t n_counters;
    int32_t *done_group, *done_tile;
    void *out;
    int32_t out_f32;
    unsigned int *status;
    uint64_t timeout_ns;
    // MoE
    int32_t k, gate;
    const float *weights;  // [T][k]
    int32_t *pos;          // [T k] row of a pair in expert order, -1: none
    uint8_t *hq, *hsf;     // h: codes [T k][F] and packed scales
    float *y;              // [T k][H]
    // adapters
    CUtensorMap B, V, V32, V1;  // V: boxes of 16 and 32 rows of all blocks, of 16 rows of one
    const uint8_t *w;      // what B and ph[0].W map
    const void *b;
    int32_t fmt;           // of the weights
    const void *a;         // bf16 [L][rank][K]
    const float *alpha;    // [L] or null
    const float *bias;     // [N] or null
    void *v;               // bf16 [group][slot_cap][blocks][nb][r64]
    int32_t rank, kr, r64, pieces, per, blocks, slot_cap;  // LoraV; rank and kr 0: no adapters, idx is null
    int32_t v_cols;  // token columns whose pieces of V a stage takes
};

// Token columns for groups of up to n rows.
inline int stream_columns(int64_t n) { return n <= 64 ? (int)((n + 15) / 16 * 16) : kStreamMaxTokens; }
// Ring and accumulator sizes for nb token columns, sub weight tiles a stage.
void stream_sizes(StreamParams &p, int nb, int sub, bool lora, int v_blocks);
// Bytes of a product's partial tiles; SMs of the device.
size_t stream_part_bytes(const StreamParams &p, int num_sms);
// Prepares the tokens, then runs the products: two launches.
cudaError_t launch_stream(bool lora, const StreamParams &p, int num_sms, cudaStream_t s);

}  // namespace fp8g
