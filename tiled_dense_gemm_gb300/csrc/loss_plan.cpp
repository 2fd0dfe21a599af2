// Host planning of the losses over a vocabulary: see loss_plan.h.
#include "loss_plan.h"

#include <algorithm>

namespace gr {
namespace ls {

namespace {
constexpr int64_t kBlockK = 64;
constexpr int64_t kSmem = 227 * 1024;
constexpr int64_t kCtrl = 2048;  // control block and alignment
constexpr int64_t kStagingBytes = 8 * 4096;
constexpr int kMaxRing = 8;
constexpr int64_t kBlockRows = 16384;         // of a forward call's block
constexpr int64_t kGradBytes = 512ll << 20;   // of G
constexpr int64_t kPlanSms = 152;             // the device's (plans fix the workspace before one is asked)

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

int pairs_of(int num_sms, int max_pairs) {
    return max_pairs < 0 ? 0 : std::min(max_pairs ? max_pairs : num_sms / 2, num_sms / 2);
}

void finish_plan(TilePlan& p, int64_t M, int64_t N, bool a_mn, bool staged, int num_sms, int max_pairs) {
    const int64_t tile_m = p.pair ? 256 : 128, per_cta = p.width / (p.pair ? 2 : 1);
    p.m_tiles = (int32_t)ceil_div(M, tile_m);
    p.n_tiles = (int32_t)ceil_div(N, p.width);
    // (rows of A that the batch does not have are not copied: what the MMA then
    // reads there ends in lanes that nothing looks at)
    p.a_rows = (int32_t)(a_mn ? 128 : std::min<int64_t>(128, round_up(M, 8)));
    p.a_bytes = p.a_rows * 128;
    p.stage_bytes = (int32_t)(p.a_bytes + per_cta * 128);
    const int64_t staging = staged ? kStagingBytes : 0;
    // (the MMA reads 128 rows of A from the last stage's start)
    const int64_t tail = std::max<int64_t>(0, 128 * 128 - p.stage_bytes - staging);
    p.num_stages = (int32_t)std::min<int64_t>(kMaxRing, (kSmem - kCtrl - staging - tail) / p.stage_bytes);
    p.smem_bytes = (int32_t)(kCtrl + (int64_t)p.num_stages * p.stage_bytes + staging + tail);
    int32_t cols = 32;
    while (cols < p.width) cols *= 2;
    p.tmem_cols = 2 * cols;
    const int64_t items = (int64_t)p.m_tiles * p.n_tiles * p.splits;
    p.grid = p.pair ? 2 * (int32_t)std::min<int64_t>(pairs_of(num_sms, max_pairs), items)
                    : (int32_t)std::min<int64_t>(num_sms, items);
    p.group_m = (int32_t)std::min<int64_t>(p.m_tiles, 8);
}

// The width whose waves take the shortest time.
int32_t best_width(int64_t m_tiles, int64_t N, bool pair, bool b_mn, int64_t workers) {
    int32_t best = 256;
    double least = 0;
    for (int32_t w : {256, 192, 128, 64}) {
        if (pair && (w == 64 || (w == 192 && b_mn))) continue;  // (whole chunks per CTA)
        const double cost = (double)ceil_div(m_tiles * ceil_div(N, w), workers) * (w + 24);
        if (w == 256 || cost < least * 0.98) {
            best = w;
            least = cost;
        }
    }
    return best;
}
}  // namespace

TilePlan plan_logits(int64_t T, int64_t N, int64_t K, bool b_mn, bool staged, int num_sms, int max_pairs) {
    (void)K;
    TilePlan p = {};
    const int pairs = pairs_of(num_sms, max_pairs);
    p.pair = T > 128 && pairs > 0;
    p.splits = 1;
    p.width = best_width(ceil_div(T, p.pair ? 256 : 128), N, p.pair != 0, b_mn, p.pair ? pairs : num_sms);
    finish_plan(p, T, N, false, staged, num_sms, max_pairs);
    return p;
}

TilePlan plan_sum(int64_t T, int64_t N, int64_t K, int splits, bool b_mn, int num_sms, int max_pairs) {
    (void)K;
    (void)b_mn;
    TilePlan p = {};
    p.pair = T > 128 && pairs_of(num_sms, max_pairs) > 0;
    p.splits = splits;
    p.width = N > 128 ? 256 : 128;
    finish_plan(p, T, N, false, true, num_sms, max_pairs);
    return p;
}

TilePlan plan_weight(int64_t M, int64_t N, int64_t K, int num_sms, int max_pairs) {
    (void)K;
    TilePlan p = {};
    p.pair = pairs_of(num_sms, max_pairs) > 0;
    p.splits = 1;
    p.width = N > 128 ? 256 : 128;
    finish_plan(p, M, N, true, true, num_sms, max_pairs);
    return p;
}

LossPlan plan_loss(int64_t T, int64_t V, int64_t D, int64_t k, bool gradient) {
    LossPlan p = {};
    p.rows = gradient ? T : std::min(T, kBlockRows);
    // forward: rows in use are gathered where that saves tiles
    p.gather = gradient || T > 128;
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
    if (p.gather) p.gathered = take(2 * rows * D);
    if (!gradient) {
        // (one or two parts per tile, whatever its width)
        p.parts = (int32_t)(2 * ceil_div(V, 128));
        if (ceil_div(V, 64) * ceil_div(rows, 128) > 2000000000ll) p.status = GEMM_ERR_TOO_LARGE;
        p.stats = take(4 * 3 * round_up(rows, 32) * p.parts);
    } else {
        int64_t piece = round_up(V, 256);
        const int64_t most = std::max<int64_t>(256, kGradBytes / (2 * rows) / 256 * 256);
        p.pieces = (int32_t)ceil_div(piece, most);
        p.piece = round_up(ceil_div(piece, p.pieces), 256);
        p.pieces = (int32_t)ceil_div(V, p.piece);
        // Shares of dX's reduction: as many as fill the last wave best, of at least 16 k-blocks.
        const bool pair = rows > 128;
        const int64_t workers = pair ? kPlanSms / 2 : kPlanSms;
        const int64_t tiles = ceil_div(rows, pair ? 256 : 128) * ceil_div(D, D > 128 ? 256 : 128);
        const int64_t blocks = ceil_div(std::min(p.piece, V), kBlockK);
        double least = 0;
        for (int32_t s = 1; s <= 16; ++s) {
            if (s > 1 && blocks / s < 16) break;
            // waves of k-blocks, plus the tile's start and end, plus the shares' way to memory and back
            const double cost = (double)ceil_div(tiles * s, workers) * ((double)blocks / s + 6) + 0.5 * s;
            if (s == 1 || cost < least * 0.97) {
                least = cost;
                p.sum_splits = s;
            }
        }
        p.grad = take(2 * rows * p.piece);
        p.sums = take(4 * rows * D * p.sum_splits);
        if (ceil_div(rows, 128) * ceil_div(p.piece, 64) > 2000000000ll || ceil_div(p.piece, 128) * ceil_div(D, 64) > 2000000000ll ||
            tiles * p.sum_splits > 2000000000ll)
            p.status = GEMM_ERR_TOO_LARGE;
    }
    p.bytes = at;
    return p;
}

}  // namespace ls
}  // namespace gr
