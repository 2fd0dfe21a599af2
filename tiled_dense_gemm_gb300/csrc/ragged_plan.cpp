#include "ragged_plan.h"

#include <algorithm>

namespace gr {
namespace rg {

namespace {
constexpr int64_t kSmem = 227 * 1024;  // per CTA
constexpr int64_t kCtrl = 1024;
constexpr int64_t kStageK = 128;       // k-rows per ring stage
constexpr int64_t kTurn = 128 * 80;    // the epilogue's transposition, four warps
// Adapters of pairs: up to this many rows the low-rank products come from the
// warp-level kernel beside the main one, beyond from a launch of tensor-core
// tiles.  The first reads a row block's own adapters only, the second every
// adapter of a row tile for all its rows, so which is faster goes by how the
// rows mix, which the host does not know (times so / with tiles).  Twenty
// requests in runs: 1024 x 1024, 16 adapters of rank 16, 1000 rows 15.4 / 19.5 us,
// 3000 rows 19.3 / 26.3; 4096 x 4096, 32 of rank 64, 300 rows 43.7 / 42.4, 1000
// 51.0 / 47.0, 2000 73.8 / 78.6, 3000 101.8 / 101.0.  Another adapter from row to
// row, same sizes: 1000 rows 25.4 / 24.9, 3000 38.6 / 30.8; 300 rows 100 / 93, 1000
// 147 / 105, 3000 386 / 265.
constexpr int64_t kLowRows = 1024;
constexpr int64_t kLowSmem = 6 * 1024;
constexpr int64_t kIndexMax = 0x7fffffff;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }
}  // namespace

// T rows in tiles of at most `width`, of equal widths in steps of `step` (the
// kernel finds the same width from their number): the number of tiles.
static int64_t equal_tiles(int64_t T, int64_t width, int64_t step, int64_t* w) {
    int64_t n = ceil_div(T, width);
    while (true) {
        *w = round_up(ceil_div(T, n), step);
        const int64_t fewer = ceil_div(T, *w);
        if (fewer == n) return n;
        n = fewer;
    }
}

RaggedPlan plan_rows(int64_t T, int64_t G, int64_t N, int64_t K, int64_t R, int64_t rank, int num_sms,
                     int max_pairs) {
    RaggedPlan p = {};
    const int64_t avg = ceil_div(T, G);
    const int pairs = max_pairs < 0 ? 0 : std::min(max_pairs ? max_pairs : num_sms / 2, num_sms / 2);
    // Up to 64 rows per group the weights' way from DRAM is what counts, and
    // single CTAs and pairs take the same time (64 groups of 4096 x 2048, 64
    // rows each: 163 us both; 4 rows: 153 and 154); above, pairs move fewer
    // bytes per operation into the multiprocessors (128 rows each: 171 us
    // against 266).  Tiles of at most 128 rows where groups have up to 96 on
    // average, else of 256: equal groups gain 2% by the first as long as they fit
    // (times with at most 128 / 256: 80 rows each 166 / 170 us, 96 168 / 172, 128
    // 172 / 176) and lose 27% once they do not (160 rows: 229 / 180), and groups
    // of more than 96 on average are seldom all below 128.
    // But a few pairs' tiles leave most multiprocessors idle, each with all of a
    // long reduction: up to two tiles for every five pairs, single CTAs, whose
    // clusters share the reduction, are faster (one group of 4096 x 1024, 512
    // rows, 8 tiles: 14.5 us against 24.2; 1024 rows, 16: 19.4 and 24.1; 2048
    // rows, 32: 33.7 and 24.4; 8 groups of 4096 x 512, 256 rows each, 30: 19.7
    // and 25.5).
    const int64_t pair_tiles = (std::min(G, T) + (T - std::min(G, T)) / 256) * ceil_div(N, 256);
    p.pair = avg > (R > 0 ? 128 : 64) && pairs > 0 && (R > 0 || pair_tiles * 5 > (int64_t)pairs * 2);
    int64_t cap;
    if (p.pair)
        cap = avg <= 96 ? 128 : 256;
    else
        cap = std::min<int64_t>(R > 0 ? 128 : 64, round_up(T, 16));
    p.cap = (int32_t)cap;
    p.num_kb = (int32_t)ceil_div(K, kStageK);
    p.n_tiles = (int32_t)ceil_div(N, p.pair ? 256 : 128);
    p.stage_bytes = (int32_t)(128 * kStageK * 2 + cap / (p.pair ? 2 : 1) * kStageK * 2);
    if (R > 0 && !p.pair && T > cap) {  // single CTAs list the adapters of one row tile
        p.status = GEMM_ERR_UNSUPPORTED_DEVICE;
        return p;
    }
    const bool low_tiles = R > 0 && p.pair && T > kLowRows;
    if (R > 0) {
        // As the kernel does for groups: tiles of the width whose waves take the
        // shortest time, if that is 5% less than with up to 256 rows (1500 rows,
        // 4096 x 4096, rank 32: 81.8 us with tiles of 256, 74.0; 2827 rows, 576 x
        // 320, rank 16: 24.2 and 18.8; 255 rows, 1728 x 360, rank 4: 19.8 and 17.3).
        int64_t width = 0;
        p.row_tiles = (int32_t)equal_tiles(T, cap, p.pair ? 32 : 16, &width);
        p.row_width = (int32_t)width;
        double least = 0;
        for (int64_t most = 256; p.pair && most >= 128; most -= 32) {
            const int64_t n = equal_tiles(T, most, 32, &width);
            const double cost = (double)ceil_div(n * p.n_tiles, pairs) * (128.0 + 0.5 * (double)width);
            if (most == 256 || (cost < 0.95 * least && n <= GEMM_RELU_MAX_GROUPS)) {
                least = cost;
                p.row_tiles = (int32_t)n;
                p.row_width = (int32_t)width;
            }
        }
    }
    const int64_t table = (R > 0 && !low_tiles ? 1 : 2) * kTurn +
                          round_up((2 * (G + 1) + (R == 0 ? 0 : p.pair ? p.row_tiles + 1 : 389)) * 4, 16);
    // (adapters: room beside it for a block of the kernel that computes low)
    const int64_t room = kSmem - kCtrl - table - (R > 0 && !low_tiles ? kLowSmem : 0);
    p.num_stages = (int32_t)std::min<int64_t>(8, room / p.stage_bytes);
    p.smem_bytes = (int32_t)(kCtrl + (int64_t)p.num_stages * p.stage_bytes + table);
    // accumulators are read 32 columns at a time; allocations are powers of two
    int64_t cols = 2 * round_up(cap, 32), alloc = 32;
    while (alloc < cols) alloc *= 2;
    p.tmem_cols = (int32_t)alloc;
    // at most this many row tiles, whatever the groups' sizes are: one row
    // in each of as many groups as can have one, the rest in full tiles
    const int64_t used = std::min(G, T);
    const int64_t tiles = R > 0 ? p.row_tiles : used + (T - used) / cap;
    const int64_t items = tiles * p.n_tiles;
    if (R > 0) {
        p.rank_box = 8;
        while (p.rank_box < 64 && p.rank_box < rank) p.rank_box *= 2;
        p.rank_pad = (int32_t)round_up(rank, p.rank_box);
    }
    if (low_tiles) {
        // (pairs have no more to do than every row tile with an adapter per row)
        const int64_t boxes = std::min<int64_t>(p.row_width, R) * (p.rank_pad / p.rank_box);
        const int64_t most = p.rank_box == 64 ? ceil_div(boxes, 2) : ceil_div(boxes * p.rank_box, 256);
        p.low_grid = 2 * (int32_t)std::min<int64_t>(pairs, p.row_tiles * most);
    }
    // (the kernel may cut pairs' groups into tiles of half that)
    if (items > kIndexMax / 2) {
        p.status = GEMM_ERR_TOO_LARGE;
        return p;
    }
    // Fewer tiles than half the multiprocessors: clusters share each tile's
    // k-blocks and add up on chip (one group of 4096 x 4096, 2 rows: 13.2
    // us against 18.7 without).
    p.cluster = 1;
    while (!p.pair && p.cluster < 8 && items * p.cluster * 2 <= num_sms && p.cluster * 4 <= p.num_kb) p.cluster *= 2;
    p.grid = p.pair ? 2 * (int32_t)std::min<int64_t>(pairs, items)
                    : (int32_t)std::min<int64_t>(num_sms, items) * p.cluster;
    return p;
}

DwPlan plan_dw(int64_t T, int64_t G, int64_t P, int64_t Q, int num_sms, int max_pairs) {
    DwPlan p = {};
    const int pairs = max_pairs < 0 ? 0 : std::min(max_pairs ? max_pairs : num_sms / 2, num_sms / 2);
    // Pairs from one tile for each of them on (single CTAs read an operand twice
    // as often): with little more than a wave, 13129 rows, 704 x 6408, 78 tiles for
    // 76 pairs, 133 us and 165 with single CTAs; 4000 rows, 4096 x 4864, 304 tiles, 85
    // and 127; 4 groups of 2000, 2048 x 1280, 160 tiles, 38 and 47; 24 groups of
    // 42, 1032 x 520, 15.6 and 17.7.
    p.pair = pairs > 0 && G * ceil_div(P, 256) * ceil_div(Q, 256) >= pairs;
    const int64_t tile = p.pair ? 256 : 128;
    p.p_tiles = (int32_t)ceil_div(P, tile);
    p.q_tiles = (int32_t)ceil_div(Q, tile);
    const int64_t stage = 2 * 128 * kStageK * 2;
    p.num_stages = 3;
    p.smem_bytes = (int32_t)(kCtrl + 3 * stage + 32 * 1024);
    const int64_t items = G * p.p_tiles * p.q_tiles;
    if (items > kIndexMax) {
        p.status = GEMM_ERR_TOO_LARGE;
        return p;
    }
    // Few tiles of long groups: clusters share each tile's rows and
    // add up on chip (one group of 7433 rows, 1472 x 376, 36 tiles: 37.5 us
    // without, 18.4 with; two of 3000 rows, 512 x 512: 15.6 and 11.9).
    p.cluster = 1;
    const int64_t blocks = ceil_div(T, G * kStageK);  // of an average group
    while (!p.pair && p.cluster < 8 && items * p.cluster * 2 <= num_sms && p.cluster * 4 <= blocks) p.cluster *= 2;
    p.grid = p.pair ? 2 * (int32_t)std::min<int64_t>(pairs, items)
                    : (int32_t)std::min<int64_t>(num_sms, items) * p.cluster;
    return p;
}

}  // namespace rg
}  // namespace gr
