// Host planning of the losses over a vocabulary: see loss_plan.h.
#include "loss_plan.h"

#include <algorithm>

namespace gr {
namespace ls {

namespace {
constexpr int64_t kSmem = 227 * 1024;
constexpr int64_t kCtrl = 2048;  // control block and alignment
constexpr int64_t kStagingBytes = 8 * 4096;
constexpr int kMaxRing = 8;
constexpr int64_t kStatBytes = 384ll << 20;   // of a forward call's statistics: its rows go in blocks,
constexpr int64_t kLeastRows = 2048;          // ... of at least so many and
constexpr int64_t kMostRows = 16384;          // at most so many rows
constexpr int64_t kGradBytes = 512ll << 20;   // of G
constexpr int64_t kPlanSms = 152;             // the device's (plans fix the workspace before one is asked)

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

int pairs_of(int num_sms, int max_pairs) {
    return max_pairs < 0 ? 0 : std::min(max_pairs ? max_pairs : num_sms / 2, num_sms / 2);
}

// Clocks that a tile of `w` columns takes per 64 k.  A pair: the tensor core's,
// but no less than its commands take (about 300 in stages of 128 k).  A single
// CTA streams B from memory at its share of it, 24 bytes a clock, and takes in
// `rows` rows of A besides, at most 41 bytes a clock in all.
double block_clocks(int64_t w, int64_t rows, bool pair) {
    if (pair) return std::max(2.0 * (double)w, 300.0);
    return std::max(128.0 * (double)w / 24, 128.0 * (double)(w + rows) / 41);
}

// not staged: statistics (the epilogue's halves hand over a few numbers)
void finish_plan(TilePlan& p, int64_t M, int64_t N, bool a_mn, bool b_mn, bool staged, bool logits, int num_sms, int max_pairs) {
    const int64_t tile_m = p.pair ? 256 : 128, per_cta = p.width / (p.pair ? 2 : 1);
    p.m_tiles = (int32_t)ceil_div(M, tile_m);
    p.n_tiles = (int32_t)ceil_div(N, p.width);
    // (rows of A that the batch does not have are not copied: what the MMA then
    // reads there ends in lanes that nothing looks at)
    p.a_rows = (int32_t)(a_mn ? 128 : std::min<int64_t>(128, round_up(M, 8)));
    const int64_t blocks = p.bk / 64;
    p.a_bytes = (int32_t)(a_mn ? 2 * 128 * p.bk : p.a_rows * 128 * blocks);
    p.stage_bytes = (int32_t)(p.a_bytes + (b_mn ? per_cta / 64 * 128 * p.bk : per_cta * 128 * blocks));
    const int64_t staging = staged ? kStagingBytes : 4096;
    // (the MMA reads 128 rows of A's last 64 k, from the last stage's start on)
    const int64_t tail = std::max<int64_t>(0, p.a_bytes / blocks * (blocks - 1) + 128 * 128 - p.stage_bytes - staging);
    p.num_stages = (int32_t)std::min<int64_t>(kMaxRing, (kSmem - kCtrl - staging - tail) / p.stage_bytes);
    p.smem_bytes = (int32_t)(kCtrl + (int64_t)p.num_stages * p.stage_bytes + staging + tail);
    int32_t cols = 64;
    while (cols < p.width) cols *= 2;
    p.tmem_cols = 2 * cols;
    const int64_t items = (int64_t)p.m_tiles * p.n_tiles * p.splits;
    p.grid = p.pair ? 2 * (int32_t)std::min<int64_t>(pairs_of(num_sms, max_pairs), items)
                    : (int32_t)std::min<int64_t>(num_sms, items);
    // Row tiles walked together, column tile by column tile.  Logits: their rows of
    // X stay in L2 while the weights pass, so the more the fewer passes (8192 rows,
    // 131072 words of 4096: 4 together 5.53 ms, 8 5.32, 16 5.19, 32 5.48; 4096
    // rows, 65536 of 2048: 702, 685, 665, 664 us).  Elsewhere both operands of a
    // group are long: 8 (the gradients of 4096 rows, 131072 words of 4096, with 8 for
    // all products 7.97 ms, with 16 8.10).
    p.group_m = (int32_t)std::min<int64_t>(p.m_tiles, logits ? 16 : 8);
}
}  // namespace

TilePlan plan_logits(int64_t T, int64_t N, int64_t K, bool b_mn, bool stats, int num_sms, int max_pairs) {
    TilePlan p = {};
    const int pairs = pairs_of(num_sms, max_pairs);
    p.pair = T > 128 && pairs > 0;
    p.splits = 1;
    // The width whose waves take the shortest time, the widest of equals, in the
    // MMA's steps; in whole chunks of 64 columns where B comes in such.  A pair's CTAs
    // take half each.
    const int64_t m_tiles = ceil_div(T, p.pair ? 256 : 128), workers = p.pair ? pairs : num_sms;
    const int32_t step = (b_mn ? 64 : 16) * (p.pair ? 2 : 1);
    const int64_t rows = std::min<int64_t>(128, T);
    double least = 0;
    for (int32_t w = 256; w >= 64; w -= step) {
        const double tile = block_clocks(w, rows, p.pair != 0) * (double)ceil_div(K, 64) + 400;
        const double cost = (double)ceil_div(m_tiles * ceil_div(N, w), workers) * tile;
        if (w == 256 || cost < least * 0.98) {
            p.width = w;
            least = cost;
        }
    }
    p.bk = p.pair ? (p.width > 192 ? 64 : 128) : (rows <= 64 ? 128 : 64);
    finish_plan(p, T, N, false, b_mn, !stats, true, num_sms, max_pairs);
    return p;
}

TilePlan plan_sum(int64_t T, int64_t N, int splits, int width, bool b_mn, int num_sms, int max_pairs) {
    TilePlan p = {};
    p.pair = T > 128 && pairs_of(num_sms, max_pairs) > 0;
    p.splits = splits;
    p.width = width;
    p.bk = p.pair && width > 192 ? 64 : 128;
    finish_plan(p, T, N, false, b_mn, true, false, num_sms, max_pairs);
    return p;
}

TilePlan plan_weight(int64_t M, int64_t N, int num_sms, int max_pairs) {
    TilePlan p = {};
    p.pair = pairs_of(num_sms, max_pairs) > 0;
    p.splits = 1;
    p.width = N > 128 ? 256 : 128;
    p.bk = 64;
    finish_plan(p, M, N, true, true, true, false, num_sms, max_pairs);
    return p;
}

LossPlan plan_loss(int64_t T, int64_t V, int64_t D, int64_t k, bool gradient) {
    LossPlan p = {};
    // (statistics of the narrowest tiles)
    const int64_t parts = ceil_div(V, 64);
    const int64_t most_rows = std::max(kLeastRows, std::min(kMostRows, kStatBytes / (12 * parts) / 256 * 256));
    p.rows = gradient || T <= most_rows ? T : round_up(ceil_div(T, ceil_div(T, most_rows)), 256);
    // forward: rows in use are gathered where that saves tiles
    p.gather = T > 128;
    p.masked = gradient && !p.gather;
    // Up to 32 rows G has two parts, the rounded values and what that left, in rows
    // of their own: a tile of 128 rows holds both, and dX and dW are as exact as their
    // own rounding.  (One rounding of G, which averages out over many rows, made up to
    // 1.5 times that.  16 rows, 65536 words of 2048: 128.6 us in one part, 130.8 in
    // two; 32 rows, 32768 of 1024: 42.6 and 46.7.)
    p.low = p.masked && T <= 32 ? (int32_t)round_up(T, 8) : 0;
    p.g_rows = p.low ? 2 * p.low : T;
    const int64_t rows = p.rows;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += round_up(bytes, 1024);
        return here;
    };
    p.header = take(64);
    p.index = take(4 * rows);
    if (k > 0) {
        p.flags = take(4 * rows);
        p.entropy = take(4 * rows);
        p.sorted = take(4 * rows * k);
        p.weights = take(4 * rows * k);
    }
    // The copy's rows start at multiples of 128 bytes, so that a box row lies in one
    // line (1800 of 3000 rows, 50021 words of 2056: 280 us at X's pitch, 266 so; the
    // gradients 930 and 892).
    p.pitch = round_up(D, 64);
    if (p.gather || p.masked) p.gathered = take(2 * std::max(rows, p.masked ? p.g_rows : 0) * p.pitch);
    if (!gradient) {
        if (parts * ceil_div(rows, 128) > 2000000000ll) p.status = GEMM_ERR_TOO_LARGE;
        p.stats = take(12 * round_up(rows, 32) * parts);
        if (!p.gather) {
            p.exact = take(8 * kMostShares);
            p.main_weight = take(4 * rows);
        }
    } else {
        const int64_t most = std::max<int64_t>(256, kGradBytes / (2 * p.g_rows) / 256 * 256);
        p.piece = round_up(ceil_div(V, ceil_div(V, most)), 256);
        p.pieces = (int32_t)ceil_div(V, p.piece);
        // Tiles and shares of dX's reduction by the time of their waves, their start
        // and end (3000 clocks) and the shares' way to memory and back.
        const bool pair = rows > 128;
        const int64_t workers = pair ? kPlanSms / 2 : kPlanSms, m_tiles = ceil_div(rows, pair ? 256 : 128);
        const int64_t blocks = ceil_div(std::min(p.piece, V), 64);
        double least = 0;
        for (int32_t w : {256, 128}) {
            if (w == 256 && D <= 128) continue;
            const double clocks = block_clocks(w, std::min<int64_t>(128, p.g_rows), pair);
            const int64_t tiles = m_tiles * ceil_div(D, w);
            for (int32_t s = 1; s <= 64; ++s) {
                if (s > 1 && blocks / s < 8) break;
                const double cost = (double)ceil_div(tiles * s, workers) * (clocks * (double)ceil_div(blocks, s) + 3000) +
                                    8.0 * (double)s * (double)p.g_rows * (double)D / 2600;
                if (p.sum_splits == 0 || cost < least * 0.98) {
                    least = cost;
                    p.sum_splits = s;
                    p.sum_width = w;
                }
            }
        }
        p.grad = take(2 * p.g_rows * p.piece);
        p.sums = take(4 * p.g_rows * D * p.sum_splits);
        if (m_tiles * ceil_div(p.piece, 64) > 2000000000ll || ceil_div(p.piece, 128) * ceil_div(D, 64) > 2000000000ll ||
            m_tiles * ceil_div(D, 64) * p.sum_splits > 2000000000ll)
            p.status = GEMM_ERR_TOO_LARGE;
    }
    p.bytes = at;
    return p;
}

}  // namespace ls
}  // namespace gr
