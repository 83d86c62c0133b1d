// The streaming GEMM kernel (stream.cu): few tokens against block-scaled
// weights that are read once.  Declarations shared by its users.
#pragma once
#include "internal.h"

namespace fp8g {

// One group: up to nb token rows against one weight matrix.
struct StreamGroup {
    int32_t mat;    // weight matrix (expert)
    int32_t row0;   // first token row of the operand
    int32_t n;      // token rows
    int32_t unit0;  // work units of the groups before it
};

constexpr int kStreamMaxGroups = 320;
constexpr int kStreamMaxLoraRows = 512;  // token rows of a call with low-rank steps
constexpr int kMaxAdapters = 1024;
constexpr int kStreamMaxTokens = 128;  // token rows of a group
constexpr int kStreamMinUnits = 4;     // work units a CTA takes at least

enum StreamEpi : int {
    kStreamGated = 0,  // act(gate) * up, quantised to E4M3 with 1x32 scales
    kStreamRows = 1,   // fp32 rows
    kStreamOut = 2,    // output rows with bias; low-rank steps
};

struct StreamParams {
    int32_t sub;     // 128-row weight tiles of a work unit (2, or 1; gated: 2)
    int32_t mt;      // weight-row tiles (of sub 128 rows; gated: 128 features) per group
    int32_t ks;      // 128-wide K steps
    int32_t rows;    // rows of a weight matrix (gated: of each half)
    int32_t n_rt;    // 128-row tiles of packed scales per matrix
    int32_t nb;      // token columns per accumulator (a multiple of 16)
    int32_t nacc;    // accumulators (2: a tile's epilogue overlaps the next tile)
    int32_t stages, stage_bytes, x_bytes;  // shared-memory ring
    uint32_t w_fmt;  // weight format as MMA instruction-descriptor bits
    int32_t gap8;    // eighths of a weight tile a packed load does not deliver
    const uint8_t *sfw;      // packed weight scales [matrix][ks][n_rt][512]
    const uint8_t *sfx;      // packed token scales [group][ks][512]
    // the groups, which every CTA derives from its call's routing: `n_idx`
    // indices idx[]: expert of each pair (negative or >= n_mat: none), or
    // (kStreamOut) adapter of each token row
    const int32_t *idx;
    int32_t n_idx, n_mat;
    int32_t *tile_cnt;       // [group][mt] units done of split tiles, zero at the start
    float *part;             // partial tiles [2 grid][2][nb][128]
    unsigned int *status;
    uint64_t timeout_ns;
    // gated
    int32_t gate;
    uint8_t *hq;             // codes [rows of tokens][rows]
    uint8_t *hsf;            // packed scales [group][mt][512]
    // rows
    float *y;                // [rows of tokens][rows]
    // out
    void *c;                 // [tokens][rows]
    int32_t out_f32;
    const float *bias;
    // low-rank: rank, steps per slot (0: none), slots per group, rows of V a
    // slot has (LoraV); n_mat adapters
    int32_t rank, kr, slot_cap, v_rows;
};

// V of a slot.  Rank up to 32: a row of 64 values holds both halves, hi in
// columns 0-31 and lo in 32-63, one 64-wide step.  More: rows of r64 = rank
// rounded up to 64, the hi rows first, then the lo rows, r64 / 64 steps.
struct LoraV {
    bool wide;  // halves in rows of their own
    int r64, kr, halves;  // row length, steps per slot, blocks of rows
    explicit LoraV(int rank)
        : wide(rank > 32), r64(wide ? (rank + 63) / 64 * 64 : 64), kr(r64 / 64), halves(wide ? 2 : 1) {}
};

// Ring and accumulator sizes for nb token columns; v_halves 2: V's two halves
// share the token region of a stage.
void stream_sizes(StreamParams &p, int nb, int v_halves);
size_t stream_part_bytes(const StreamParams &p, int grid);
cudaError_t launch_stream(int epi, const CUtensorMap &w, const CUtensorMap &x, const CUtensorMap &lb,
                          const CUtensorMap &v, const StreamParams &p, int grid, cudaStream_t s);

}  // namespace fp8g
