// Declarations of the block-scaled 8-bit operators and the scored router
// (quant.cu, blocks.cu, route_scored.cu), shared with the host layer.
#pragma once

#include "internal.h"

namespace moe {

constexpr int BLK = 128;             // columns (and weight rows) that share a scale
constexpr int SE_MAX = 512;          // experts
constexpr int ST_MAX = 65536;        // tokens
constexpr int SD_MIN = 16, SD_MAX = 16384;

inline int blocks_of(int n) { return (n + BLK - 1) / BLK; }
// floats between the scales of two rows in the library's own buffers: whole
// 16-byte pieces, which one copy each moves
inline int scale_pitch(int cols) { return (blocks_of(cols) + 3) / 4 * 4; }

// Control segment at the start of every workspace of these operators: the
// error word first (moe_check_error), then what a call counts in.  The layer
// path's Counters start at the same place: all four words are zero between
// calls there too, so one workspace may serve both in turn, as long as
// nothing else is kept in, or written to, the first
// MOE_GEMM_WORKSPACE_BYTES.
struct BlocksControl {
    int32_t error;
    int32_t next_tile, exits;  // product kernel: tiles claimed, CTAs finished (zero between calls)
    uint32_t ticket;           // router: blocks finished (zero between calls)
    int32_t pad[60];
};
static_assert(sizeof(BlocksControl) <= MOE_GEMM_WORKSPACE_BYTES, "control segment does not fit");

struct BlocksWs {
    size_t xq, xs, hq, hs, yp, counts, inv, total;
    size_t n_counts;  // cnt [B], then done [m-tiles]
};
BlocksWs blocks_ws(const moe_dims_t &d);
size_t route_ws_bytes(const moe_dims_t &d);

// TMA descriptors of a product's phases: activation rows as boxes of one row
// (gathered four at a time) and of product_box_rows rows, and two weight maps
// [E][rows][K] with boxes of 128 rows x 128 bytes (the same matrix twice for
// a plain product).
struct PhaseMaps {
    CUtensorMap a, ab, b0, b1;
};
struct ProductMaps {
    PhaseMaps phase[2];
};
int product_box_rows(const moe_dims_t &d);
int product_tile_entries(const moe_dims_t &d);  // list entries per tile
// Whether the expert FFN copies each entry's activation row to its place in
// the lists (else the rows are gathered by token).
bool product_dispatch(const moe_dims_t &d);
bool encode_phase_maps(PhaseMaps *m, const void *a, uint64_t a_rows, int box_rows, const void *b0, const void *b1,
                       uint64_t E, uint64_t rows, uint64_t K);

enum ProductKind : int { PRODUCT_OUT = 0, PRODUCT_SWIGLU = 1 };

struct ProductPhase {
    int kind;             // ProductKind
    int K, rows;          // columns of a weight row; rows of one weight matrix
    int by_pair;          // activation row of list entry p: p itself, else tok[p]
    const float *as;      // activation scales: row r, block j at as[r * as_pitch + j]
    int as_pitch;
    const float *bs0, *bs1;  // weight scales [E][blocks of rows][blocks of K]
    void *out;            // PRODUCT_OUT: [entries][rows] fp32 or bf16
    int out_bf16;
    uint8_t *hq;          // PRODUCT_SWIGLU: [entries][rows] e4m3
    float *hs;            // and its scales, row p's block j at hs[p * hs_pitch + j]
    int hs_pitch;
};
struct ProductArgs {
    ProductPhase phase[2];
    int phases;
    int tile_entries;     // product_tile_entries
    int B, E, k;          // dims of the lists
    const int32_t *n_active, *active, *offsets, *tok;
    int32_t *done;        // two phases: gate/up tiles done per m-tile
    int32_t *cnt, *inv;   // two phases: entries of each token: counts [B], entry indices [B][k]
    int32_t *error, *next_tile, *exits;
    unsigned long long wait_ns;
};
cudaError_t launch_product(const ProductMaps &maps, const ProductArgs &a, cudaStream_t s);

// e4m3 values and power-of-two scales of [batch][rows][cols] (block_rows 1
// or 128).
cudaError_t launch_quantize(const void *x, int type, int64_t batch, int64_t rows, int64_t cols, int block_rows,
                            uint8_t *q, float *scale, cudaStream_t s);
// Rows of x [n_src][cols] (row src[r] when src is given; negative: skipped)
// -> q [rows][cols], scales [rows][scale_pitch(cols)]; zero[0 .. n_zero) = 0.
cudaError_t launch_quantize_dispatch(const void *x, int type, int64_t rows, int cols, const int32_t *src, int n_src,
                                     uint8_t *q, float *scale, int32_t *zero, int n_zero, cudaStream_t s);
// y[t] = sum over the token's entries p, ascending, of w[p] * yp[p]
cudaError_t launch_combine(const float *yp, const float *w, const int32_t *cnt, const int32_t *inv, int B, int d,
                           int k, void *y, int y_bf16, cudaStream_t s);

cudaError_t launch_route_scored(const float *logits, const float *bias, const moe_dims_t &d,
                                const moe_scoring_t &r, int32_t *sel_idx, float *sel_w, const moe_lists_t &l,
                                void *ws, cudaStream_t s);

}  // namespace moe
