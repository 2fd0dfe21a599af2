// Host planning of the ragged products (pure host code): tile shape, ring
// depth, grid and limits from the sizes the host knows.
#pragma once

#include <stdint.h>

#include "gemm_relu.h"

namespace gr {
namespace rg {

struct RaggedPlan {
    int32_t status;
    int32_t pair;        // CTA pairs (256 columns per tile) instead of single CTAs (128)
    int32_t cap;         // most rows of a tile
    int32_t row_tiles;   // adapters: row tiles,
    int32_t row_width;   // ... and rows of each
    int32_t cluster;     // single CTAs: CTAs (a cluster) that share each item's k-blocks
    int32_t num_kb, n_tiles;
    int32_t stage_bytes, num_stages, smem_bytes, tmem_cols;
    int32_t grid;        // CTAs
    int32_t rank_box, rank_pad;
    int32_t low_grid;    // adapters: > 0: the low-rank products come from a launch of tensor-core tiles, its CTAs
};

struct DwPlan {
    int32_t status;
    int32_t pair, cluster, p_tiles, q_tiles, num_stages, smem_bytes, grid;
};

// R == 0: experts' products over G groups; else adapters (G is 1).
RaggedPlan plan_rows(int64_t T, int64_t G, int64_t N, int64_t K, int64_t R, int64_t rank, int num_sms, int max_pairs);
DwPlan plan_dw(int64_t T, int64_t G, int64_t P, int64_t Q, int num_sms, int max_pairs);

}  // namespace rg
}  // namespace gr
