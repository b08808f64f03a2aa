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

// Control segment at the start of every workspace of these operators: the
// error word first (moe_check_error), then what a call counts in.
struct BlocksControl {
    int32_t error;
    int32_t pad[63];
};
static_assert(sizeof(BlocksControl) <= MOE_GEMM_WORKSPACE_BYTES, "control segment does not fit");

struct BlocksWs {
    size_t xq, xs, hq, hs, yp, cnt, inv, total;
};
BlocksWs blocks_ws(const moe_dims_t &d);
size_t route_ws_bytes(const moe_dims_t &d);

// TMA descriptors of one grouped product: activation rows (gathered four at
// a time) and two weight maps [E][rows][K] with boxes of 128 rows x 128
// bytes (the same matrix twice for a plain product).
struct ProductMaps {
    CUtensorMap a, b0, b1;
};
bool encode_product_maps(ProductMaps *m, const void *a, uint64_t a_rows, const void *b0, const void *b1,
                         uint64_t E, uint64_t rows, uint64_t K);

enum ProductKind : int { PRODUCT_OUT = 0, PRODUCT_SWIGLU = 1 };

struct ProductArgs {
    int kind;             // ProductKind
    int B, E, k;          // dims of the lists
    int K, rows;          // columns of a weight row; rows of one weight matrix
    int by_pair;          // activation row of list entry p: p itself, else tok[p]
    const float *as;      // activation scales [rows of a][blocks of K]
    const float *bs0, *bs1;  // weight scales [E][blocks of rows][blocks of K]
    const int32_t *n_active, *active, *offsets, *tok;
    void *out;            // PRODUCT_OUT: [entries][rows] fp32 or bf16
    int out_bf16;
    uint8_t *hq;          // PRODUCT_SWIGLU: [entries][rows] e4m3
    float *hs;            // and its scales [entries][blocks of rows]
    int32_t *cnt, *inv;   // entries of each token (or null): counts [B], entry indices [B][k]
    int32_t *error;
    unsigned long long wait_ns;
};
cudaError_t launch_product(const ProductMaps &maps, const ProductArgs &a, cudaStream_t s);

// e4m3 values and power-of-two scales of [batch][rows][cols] (block_rows 1
// or 128); cnt (or null): B counters set to zero.
cudaError_t launch_quantize(const void *x, int type, int64_t batch, int64_t rows, int64_t cols, int block_rows,
                            uint8_t *q, float *scale, int32_t *cnt, int n_cnt, cudaStream_t s);
// y[t] = sum over the token's entries p, ascending, of w[p] * yp[p]
cudaError_t launch_combine(const float *yp, const float *w, const int32_t *cnt, const int32_t *inv, int B, int d,
                           int k, void *y, int y_bf16, cudaStream_t s);

cudaError_t launch_route_scored(const float *logits, const float *bias, const moe_dims_t &d,
                                const moe_scoring_t &r, int32_t *sel_idx, float *sel_w, const moe_lists_t &l,
                                void *ws, cudaStream_t s);

}  // namespace moe
