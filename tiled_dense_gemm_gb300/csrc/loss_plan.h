// Host planning of the losses over a vocabulary (pure host code): pieces of
// the vocabulary, tile shapes, shares of the reductions, workspace.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "gemm_relu.h"

namespace gr {
namespace ls {

// One product's tiles.
struct TilePlan {
    int32_t pair;     // CTA pairs
    int32_t width;    // columns of a tile
    int32_t bk;       // k per stage
    int32_t m_tiles, n_tiles, splits, group_m;
    int32_t a_rows;   // rows of A's box (k-major)
    int32_t a_bytes, stage_bytes, num_stages, smem_bytes, tmem_cols, grid;
};

// Shares of exact logits of a call (eight warps on each of 152 SMs).
constexpr int64_t kMostShares = 1216;

struct LossPlan {
    int32_t status;
    int64_t rows;        // forward: rows of a block; backward: all
    int64_t piece;       // backward: words of a piece, a multiple of 256 (the last one may be shorter)
    int32_t pieces;
    int32_t gather;      // the rows in use are counted, and gathered if some are not
    int32_t masked;      // backward, up to 128 rows: a copy of X with zeros for those that are not
    int32_t low;         // backward, up to 32 rows: > 0: G's rows from here on hold what rounding left of the first
    int64_t g_rows;      // rows of G
    int32_t sum_splits;  // backward: shares of dX's reduction,
    int32_t sum_width;   // ... and its tiles' columns
    int64_t pitch;       // of the rows' copy
    // workspace, in bytes from its start
    int64_t header, index, flags, entropy, sorted, weights, gathered, stats, exact, main_weight, grad, sums, bytes;
};

// The logits (T x N, reduction K): `stats` of the forward pass, else G.  b_mn: B
// comes in chunks of 64 columns.
TilePlan plan_logits(int64_t T, int64_t N, int64_t K, bool b_mn, bool stats, int num_sms, int max_pairs);
// Sums of dX (T x N) in `splits` shares, tiles of `width`.
TilePlan plan_sum(int64_t T, int64_t N, int splits, int width, bool b_mn, int num_sms, int max_pairs);
// dW (M x N).
TilePlan plan_weight(int64_t M, int64_t N, int num_sms, int max_pairs);

// k: words of a teacher per row, 0: targets.
LossPlan plan_loss(int64_t T, int64_t V, int64_t D, int64_t k, bool gradient);

}  // namespace ls
}  // namespace gr
