// Products of ragged rows with several weights, for sm_103a:
//
//   Y[t, :] = epilogue( sum_k X[t, k] W[g(t)][k, :] )
//
// where the rows t are sorted by group and only the device knows how many
// rows each group has (experts' products, forward and data gradient), or
// where every row shares one W and adds a low-rank part of its own adapter
// (kAdapters).
//
// Operand roles.  The weights are the MMA's M side (128 output columns per
// CTA, 256 per CTA pair) and the rows its N side: tcgen05's N goes in steps
// of 16 at run time, so a group of any size costs its rows rounded up to 16
// (32 for a pair), not to a 128- or 256-row tile, and a group of a few rows
// streams its weights with next to no MMA work.  D^T sits in tensor memory
// with an output column per lane and a row per TMEM column, so masking the
// rows past a group's end is a uniform branch per store.
//
// Work list.  Each CTA reads the G + 1 row offsets once and builds two
// prefix arrays in shared memory (first row, row tiles before the group);
// item i is then (group, row tile, column tile) by binary search, with no
// host round trip and no launch of its own.  A group's rows are cut into
// tiles of equal width, so a pair's 260 rows are 160 + 100 and not 256 + 4.
//
// Column tiles that are few (short calls) are computed by clusters: each CTA
// takes a share of the tile's k-blocks and the cluster adds the shares up
// through distributed shared memory.
//
// Roles (352 threads; 224 with adapters, but 352 where warps 7-10 help; one CTA
// per SM): warp 0 copies row tiles, warp 6 the weights, warp 1 issues the MMAs,
// warps 2-5 and 7-10 (2-5) drain the accumulators; shared-memory ring of 128-k stages, two TMEM accumulators.  Every wait is
// bounded.  The epilogue turns D^T round in shared memory (each warp its own
// 32 x 32 blocks), applies the ReLU or the gate in 32 bits or on the rounded
// value, and rounds once, to the output's type.
//
// What bounds it, and what it measured (bfloat16 or binary16; the GPU's time
// alone, of calls in a CUDA graph whose inputs rotate beyond L2.  Long runs of
// single calls settle at a lower clock: the large cases take 10-15% more there):
//   few rows per group: the weights' way from DRAM.  64 groups of 4096 x
//     2048, 256 rows: 152-154 us, 7.0 TB/s.
//   many: bytes into the multiprocessors.  A pair takes 256 x (rows of the
//     tile) products per k from L2, and tiles of ragged groups are narrower
//     than 256: 32 groups of 2048 x 4096, 16384 rows: 184-189 us,
//     1480 TFLOP/s, with 13.2 TB/s from L2 (159 us with the weights' copies left
//     out, 157 us with the MMAs left out: neither hides the other wholly).
//     Stages of 64 k (six of them) instead of 128 (three): 197 us.
//   row pitches that are not multiples of 128 bytes cost a second copy per
//     stage and operand and a second line per row: 5000 rows, 12 groups of
//     2056 x 3000, 65 us.
//   rows with adapters: as above, and the second factors and the low-rank
//     products in extra k-blocks at the end of each tile, ~0.9 us each
//     (64 rows, 48 adapters of rank 32, 8192 x 8192: 48-49 us, of which DRAM
//     takes 32; 8192 rows, 24 adapters of rank 64, 4096 x 4096: 202 us, of
//     which ~150 us are the shared product's and ~35 the launch of low before).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "ptx.cuh"
#include "ragged_ptx.cuh"

namespace gr {
namespace rg {

constexpr int kHelped = 352;  // threads of the adapters' pair kernel with four more warps for its main tiles' epilogue

// Epilogue warps: eight, each half of a quarter's 32-row chunks (one warp per
// scheduler takes 0.7 us per chunk, which shows where the last tile's epilogue
// has nothing to hide behind: 3000 rows, 8 groups, 4096 -> 1024: 32.9 us with
// four warps, 30.0 with eight); four in the adapters' kernels, which share the
// registers with the low-rank kernel, and where there is none four more, which
// drain the main tiles while the first four fill the next one's extra k-blocks
// (12153 rows, 296 x 6608, rank 8: 152 us without, 120 with; 8192 rows of 4096 x
// 4096, whose main k-blocks are longer than both: the same).
constexpr uint32_t kEpiThreads = 128;
__host__ __device__ constexpr uint32_t epi_threads(bool adapters) { return adapters ? kEpiThreads : 2 * kEpiThreads; }
__host__ __device__ constexpr int row_threads(bool adapters) { return 96 + (int)epi_threads(adapters); }
constexpr uint32_t kEpiBarrier = 1;
constexpr int kBK = 128;       // k-rows per ring stage: eight MMAs per wait and commit
constexpr int kMaxStages = 8;
constexpr int kMaxBoxes = 2048;  // adapters: boxes of rank_box rows of a row tile's second factors (256 x 512 / 64)
constexpr int kTokBoxes = 8;   // row-tile boxes of 16, 32, ..., 128 rows per CTA
constexpr int kXK = 64;        // adapters: products of the rank per extra k-block, each in two parts
constexpr int kRaster = 8;     // row tiles of one group walked together, column tile by column tile
constexpr uint32_t kTurnPitch = 80;  // bytes per row of the transposition: 64, + 16 against bank conflicts
constexpr uint32_t kWBytes = 128 * kBK * 2;  // weights per stage and CTA

enum : int32_t {
    kErrTokens = 0x61,
    kErrWeights = 0x62,
    kErrStage = 0x63,
    kErrAccum = 0x64,
    kErrEpi = 0x65,
    kErrFinal = 0x66,
};
// codes of the second error word (bad values in an index array)
enum : int32_t { kBadOffsets = 1, kBadIds = 2 };

struct Maps {
    CUtensorMap w;             // weights
    CUtensorMap x[kTokBoxes];  // rows, boxes of 16 (i + 1) rows
    CUtensorMap b;             // adapters' second factors
    CUtensorMap a, a4;         // ... and first ones: boxes of rank_box rows x 64 k; a4: x 2 x 64 k
};

struct Params {
    int32_t T, G;        // rows of X; groups (1: all rows)
    int32_t N, K;        // output columns, reduction length
    int32_t num_kb;      // ceil(K / kBK)
    int32_t n_tiles;     // column tiles (128, or 256 for a pair)
    int32_t cap;         // most rows of a tile
    int32_t cluster;     // single CTAs: > 1: each item's k-blocks shared by the CTAs of a cluster
    int32_t num_stages;
    int32_t stage_bytes; // stride of a ring stage
    int32_t turn_off;    // shared-memory offsets from the ring's start: the epilogue's transposition,
    int32_t table_off;   // the prefix arrays
    uint32_t tmem_cols;  // allocated; half of them per accumulator
    int32_t w_kmajor;    // weights stored with the reduction contiguous
    int32_t w4d;         // one copy per stage and CTA of the weights
    int32_t x3d;         // one copy per stage of a row tile
    int32_t apply_relu, bf16;
    const int32_t* offsets;  // G + 1, or null: one group of all rows
    uint16_t* Y;
    int64_t ldy;
    const uint16_t* act;     // gate: outputs where act <= 0 are set to +0 (null: none)
    int64_t ld_act;
    int32_t* err;            // err[0] timed-out waits, err[1] bad index arrays
    uint64_t timeout_ns;
    // test hook of the bounded waits, 0 in every normal call: k + 1 leaves the
    // row copy of k-block k of each CTA's first item undone (its stage is
    // still armed for the bytes); the host pairs it with a short timeout_ns
    // and plans of single CTAs
    int32_t test_drop_kb;
    // adapters
    int32_t row_tiles;       // of equal widths
    const int32_t* ids;      // adapter of each row, -1 none
    const uint16_t* low;     // (T, 2, rank_pad): scale * x A^T, in two parts of the element type
    const int32_t* nslots;   // distinct adapters of each row tile; null: single CTAs, which list them themselves
    const int32_t* slots;    // [tile][cap] their indexes
    const uint16_t* B;       // second factors (R, rank, N)
    int32_t rank, rank_pad, rank_box, b4d, a4d;  // rank_box: 8, 16, 32 or 64; rank_pad a multiple of it
    int32_t box_shift;       // rank_box = 1 << box_shift
    int32_t per_slot;        // rank_pad / rank_box
    int32_t R;
    const float* scale;      // of each adapter, or null: 1
    uint16_t* low_out;       // pairs: this launch's items are the low-rank products (null: columns of Y)
};

struct __align__(8) Ctrl {
    uint64_t full[kMaxStages];
    uint64_t empty[kMaxStages];
    uint64_t tmem_full[2];
    uint64_t tmem_empty[2];
    uint64_t final_bar;
    uint64_t extra[kMaxStages];  // adapters: the stage is free for an extra k-block
    uint64_t peer[kMaxStages];   // ... and, of a pair's leader, filled by the peer
    uint32_t sick[kMaxBoxes / 32];  // adapters: boxes of the item's second factors that are not finite
    uint64_t boxes[kMaxStages];     // ... landed in a stage
    int32_t helped;                 // ... items that the helping warps have drained, times their number
    int32_t sick_item;              // ... 1 + the CTA's item some of whose boxes are kept out
    uint32_t tmem_addr;
    int32_t abort_flag;
    int32_t ring_s, ring_ph, ring_lap;
};
static_assert(sizeof(Ctrl) <= 1024, "control block exceeds its reserved 1 KiB");

__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, Ctrl* ctrl, const Params& p, int32_t site) {
    if (mbar_try_wait(bar, parity)) return true;
    volatile int32_t* abort_flag = &ctrl->abort_flag;
    const uint64_t t0 = globaltimer_ns();
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (globaltimer_ns() - t0 > p.timeout_ns) {
            *abort_flag = 1;
            atomicCAS(p.err, 0, site);
            return false;
        }
    }
}

// The same for arrivals from the other CTA of a pair.
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity, Ctrl* ctrl, const Params& p) {
    volatile int32_t* abort_flag = &ctrl->abort_flag;
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait_acq_cluster(bar, parity))
        if (*abort_flag || globaltimer_ns() - t0 > p.timeout_ns) {
            *abort_flag = 1;
            atomicCAS(p.err, 0, (int32_t)kErrEpi);
            return false;
        }
    return true;
}

// The same until a counter in shared memory has reached a value.
__device__ __forceinline__ bool wait_counter(int32_t* counter, int32_t value, Ctrl* ctrl, const Params& p) {
    volatile int32_t* const c = counter;
    volatile int32_t* abort_flag = &ctrl->abort_flag;
    const uint64_t t0 = globaltimer_ns();
    while (*c < value)
        if (*abort_flag || globaltimer_ns() - t0 > p.timeout_ns) {
            *abort_flag = 1;
            atomicCAS(p.err, 0, (int32_t)kErrEpi);
            return false;
        }
    __threadfence_block();
    return true;
}

// Bounded wait (100 us in all) for the copies that an aborting CTA has in
// flight, before its shared memory is released.
__device__ __forceinline__ void drain_ring(Ctrl* ctrl, uint32_t full0, uint32_t S) {
    const uint64_t t0 = globaltimer_ns();
    const uint32_t ring_s = (uint32_t)ctrl->ring_s, ring_ph = (uint32_t)ctrl->ring_ph;
    for (uint32_t i = 0; i < S; ++i) {
        if (i >= ring_s && !ctrl->ring_lap) continue;  // never armed
        const uint32_t parity = i < ring_s ? ring_ph : ring_ph ^ 1u;
        while (!mbar_try_wait(full0 + 8u * i, parity))
            if (globaltimer_ns() - t0 > 100000ull) return;
    }
}

// ------------------------------------------------------------------ work list

// Prefix arrays of the groups, by one warp: start[g] = first row of group g
// (start[G]: end of the last), tiles[g] = row tiles before it.  Offsets are
// clamped to [0, T] and to be non-decreasing, so no later index can leave the
// tensors; if that changed any, bad index arrays are reported.
__device__ __forceinline__ void build_table(const Params& p, int32_t* start, int32_t* tiles, uint32_t lane, uint32_t workers) {
    if (!p.offsets) {
        if (lane == 0) {
            start[0] = 0;
            start[1] = p.T;
            tiles[0] = 0;
            tiles[1] = p.row_tiles;
        }
        return;
    }
    bool bad = false;
    int32_t top = 0, count = 0;  // running maximum and tile count before this round
    for (int32_t g0 = 0; g0 < p.G; g0 += 32) {
        const int32_t g = g0 + (int32_t)lane;
        int32_t lo = 0, hi = 0;
        if (g < p.G) {
            const int32_t a = __ldcg(p.offsets + g), b = __ldcg(p.offsets + g + 1);
            lo = min(max(a, 0), p.T);
            hi = min(max(b, 0), p.T);
            bad |= a != lo || b != hi || hi < lo;
        }
        // inclusive maximum of lo over the lanes, and of every offset before
        int32_t m = max(lo, top);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t o = __shfl_up_sync(0xffffffffu, m, d);
            if ((int)lane >= d) m = max(m, o);
        }
        const int32_t end = max(m, hi);
        int32_t n = g < p.G ? (end - m + p.cap - 1) / p.cap : 0;
        const int32_t mine = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t o = __shfl_up_sync(0xffffffffu, n, d);
            if ((int)lane >= d) n += o;
        }
        if (g < p.G) {
            start[g] = m;
            tiles[g] = count + n - mine;
            if (g == p.G - 1) {
                start[p.G] = end;
                tiles[p.G] = count + n;
            }
        }
        const int32_t last = min(31, p.G - 1 - g0);
        top = __shfl_sync(0xffffffffu, end, last);
        count += __shfl_sync(0xffffffffu, n, last);
    }
    if (bad) atomicCAS(p.err + 1, 0, (int32_t)kBadOffsets);
    if (p.cap != 256) return;
    // Pairs with tiles of up to 256 rows: the last of few waves may be nearly
    // empty.  A wave takes about as long as its copies, 128 weights and half a
    // tile's rows per k and CTA; of tiles of up to 256, 224, ..., 128 rows the
    // ones whose waves take the shortest time, if that is 5% less (4 groups of
    // 2583 rows, 5440 x 512: 61.1 us with tiles of 240, 54.1 with 160; 4 of 1030,
    // 4096 x 1024: 41.4 and 38.4).
    __syncwarp();
    int32_t rows = 0, cnt[5] = {0, 0, 0, 0, 0};  // in steps of 32 rows; tiles for each width
    for (int32_t g = (int32_t)lane; g < p.G; g += 32) {
        const int32_t units = (start[g + 1] - start[g] + 31) >> 5;
        rows += units;
        cnt[0] += (units + 7) / 8;
        cnt[1] += (units + 6) / 7;
        cnt[2] += (units + 5) / 6;
        cnt[3] += (units + 4) / 5;
        cnt[4] += (units + 3) / 4;
    }
    rows = __reduce_add_sync(0xffffffffu, rows);
    int32_t n_here = 1;  // lane k: the k-th width's tiles
#pragma unroll
    for (int k = 0; k < 5; ++k) {
        cnt[k] = __reduce_add_sync(0xffffffffu, cnt[k]);
        if ((int)lane == k) n_here = max(cnt[k], 1);
    }
    const uint32_t waves = ((uint32_t)n_here * (uint32_t)p.n_tiles + workers - 1u) / workers;
    const float cost = (float)waves * (128.0f + __fdividef(16.0f * (float)rows, (float)n_here));
    int32_t best = 8;
    float least = __shfl_sync(0xffffffffu, cost, 0);
#pragma unroll
    for (int k = 1; k < 5; ++k) {
        const float c = __shfl_sync(0xffffffffu, cost, k);
        if (c < 0.95f * least) {
            least = c;
            best = 8 - k;
        }
    }
    if (best == 8) return;
    count = 0;
    for (int32_t g0 = 0; g0 < p.G; g0 += 32) {
        const int32_t g = g0 + (int32_t)lane;
        const int32_t mine = g < p.G ? (((start[g + 1] - start[g] + 31) >> 5) + best - 1) / best : 0;
        int32_t n = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t o = __shfl_up_sync(0xffffffffu, n, d);
            if ((int)lane >= d) n += o;
        }
        if (g < p.G) tiles[g] = count + n - mine;
        count += __shfl_sync(0xffffffffu, n, 31);
    }
    if (lane == 0) tiles[p.G] = count;
}

struct Item {
    int32_t g;          // group
    int32_t tile;       // row tile (over all groups)
    int32_t row0;       // first row
    int32_t valid;      // rows of this tile
    int32_t w;          // rows rounded up to the MMA's granularity
    int32_t n;          // column tile
    int32_t kb0, kb1;   // this CTA's k-blocks [kb0, kb1)
    int32_t x0, x1;     // ... and extra ones (adapters)
    bool low;           // low-rank products of the row tile (n: which of them), not columns of Y
};

// The slot (position among a row tile's adapters) that box `box` of its
// ranks belongs to.  (Divisions cost the single-thread roles ~100 cycles
// each; ranks up to 64 need none.)
__device__ __forceinline__ int32_t slot_of(const Params& p, int32_t box) {
    return p.per_slot == 1 ? box : box / p.per_slot;
}

// Low items compute the low-rank products of a row tile, boxes of rank_box of
// them at a time: one box per CTA of the pair where the tile has at most two,
// or boxes are large (64), which takes one copy per stage; else as many as
// the MMA's 128 rows hold, at two copies per box.  (Copies issue one after
// another, ~450 cycles each: with four per stage an item of 32 stages took
// 33 us, most of it waiting for them.)
__device__ __forceinline__ int32_t low_boxes(const Params& p, int32_t slots) {
    return p.rank_box == 64 || slots * p.per_slot <= 2 ? 1 : 128 >> p.box_shift;
}

__device__ __forceinline__ int32_t low_items(const Params& p, int32_t slots) {
    const int32_t boxes = slots * p.per_slot;
    return p.rank_box == 64 || boxes <= 2 ? (boxes + 1) / 2 : (boxes + (256 >> p.box_shift) - 1) >> (8 - p.box_shift);
}

// Extra k-blocks of a row tile: its distinct adapters' ranks side by side.
__device__ __forceinline__ int32_t extra_blocks(const Params& p, int32_t slots) {
    return (slots * p.rank_pad + kXK - 1) / kXK;
}

// The distinct adapters of one row tile of at most 128 rows, in order of
// first appearance, by 128 threads (i = 0 .. 127); of each also the 16-row
// window that holds its rows, lo | hi << 16.  Leaves the rows' ids in shared
// memory and reports indexes outside [-1, R).
__device__ __forceinline__ void list_slots(const Params& p, int32_t* ids, int32_t* slots, int32_t* windows,
                                           int32_t* count, int32_t* nslots, int32_t i) {
    int32_t mine = i < p.T ? __ldcg(p.ids + i) : -1;
    if (mine < -1 || mine >= p.R) {
        atomicCAS(p.err + 1, 0, (int32_t)kBadIds);
        mine = -1;
    }
    ids[i] = mine;
    named_bar_sync(kEpiBarrier, kEpiThreads);
    // the rows of the same adapter, warp by warp (ids is 16-byte aligned)
    const int32_t lane = i % 32;
    const uint32_t own = __match_any_sync(0xffffffffu, mine);
    bool first = mine >= 0 && (own & ((1u << lane) - 1u)) == 0;
    int32_t last = i / 32 * 32 + 31 - __clz((int)own);
    for (int32_t w = 0; w < (min(128, p.T) + 31) / 32; ++w) {
        if (w == i / 32) continue;
        uint32_t same = 0;
#pragma unroll
        for (int32_t j = 0; j < 8; ++j) {
            const int4 q = reinterpret_cast<const int4*>(ids)[8 * w + j];
            same |= ((uint32_t)(q.x == mine) | (uint32_t)(q.y == mine) << 1 | (uint32_t)(q.z == mine) << 2 |
                     (uint32_t)(q.w == mine) << 3) << (4 * j);
        }
        if (same && w < i / 32) first = false;
        if (same) last = max(last, 32 * w + 31 - __clz((int)same));
    }
    const uint32_t votes = __ballot_sync(0xffffffffu, first);
    if (lane == 0) count[i / 32] = __popc(votes);
    named_bar_sync(kEpiBarrier, kEpiThreads);
    int32_t at = __popc(votes & ((1u << lane) - 1u));
    for (int32_t w = 0; w < i / 32; ++w) at += count[w];
    if (first) {
        slots[at] = mine;
        windows[at] = (i & ~15) | ((last | 15) + 1) << 16;
    }
    if (i == 0) *nslots = count[0] + count[1] + count[2] + count[3];
}

template <bool kPair, bool kAdapters>
struct Iter {
    const Params& p;
    const int32_t* start;
    const int32_t* tiles;
    const int32_t* nslots;
    const int32_t* lows;  // a launch of low items: those before each row tile
    uint32_t u, u1, step;
    int32_t share;      // this CTA's rank in its cluster
    int32_t max_extra;  // single CTAs of adapters: the one row tile's extra k-blocks

    __device__ __forceinline__ Iter(const Params& p_, const int32_t* start_, const int32_t* tiles_,
                                    const int32_t* nslots_, const int32_t* lows_, uint32_t worker, uint32_t workers,
                                    int32_t max_extra_, int32_t share_)
        : p(p_), start(start_), tiles(tiles_), nslots(nslots_), lows(lows_), share(share_), max_extra(max_extra_) {
        u = worker;
        u1 = kPair && kAdapters && p.low_out ? (uint32_t)lows[tiles[p.G]] : (uint32_t)tiles[p.G] * (uint32_t)p.n_tiles;
        step = workers;
    }

    // rows of tile j of the cnt of group g: equal widths, in the MMA's steps,
    // but the last only as wide as what is left for it (32 groups of 512 rows
    // on average: 4% fewer columns of MMA work than with all equal)
    __device__ __forceinline__ void row_tile(Item& it, int32_t g, int32_t cnt, int32_t j) {
        const int32_t s0 = start[g], len = start[g + 1] - s0;
        constexpr int32_t kGran = kPair ? 32 : 16;
        it.w = ((len + cnt - 1) / cnt + kGran - 1) / kGran * kGran;
        it.row0 = s0 + j * it.w;
        it.valid = min(it.w, len - j * it.w);
        it.w = (it.valid + kGran - 1) / kGran * kGran;
    }

    __device__ __forceinline__ bool next(Item& it) {
        if (u >= u1) return false;
        const uint32_t item = u;
        u += step;
        it.kb0 = it.x0 = it.x1 = 0;
        it.kb1 = p.num_kb;
        if (!kPair && p.cluster > 1) {
            // an even share of the main k-blocks (DRAM) and of the extra ones
            // (latency) for each CTA of the cluster
            it.kb0 = share * p.num_kb / p.cluster;
            it.kb1 = (share + 1) * p.num_kb / p.cluster;
            it.x0 = share * max_extra / p.cluster;
            it.x1 = (share + 1) * max_extra / p.cluster;
        } else if (kAdapters) {
            it.x1 = kPair ? -1 : max_extra;  // (-1: the row tile's, below)
        }
        it.low = false;
        if constexpr (kPair && kAdapters) {
            if (p.low_out) {
                int32_t lo = 0, hi = tiles[p.G];  // largest row tile with lows[tile] <= item
                while (hi - lo > 1) {
                    const int32_t mid = (lo + hi) >> 1;
                    if (lows[mid] <= (int32_t)item) lo = mid; else hi = mid;
                }
                it.low = true;
                it.g = 0;
                it.tile = lo;
                it.n = (int32_t)item - lows[lo];
                row_tile(it, 0, tiles[p.G], lo);
                it.x1 = 0;
                return true;
            }
        }
        const uint32_t nt = (uint32_t)p.n_tiles;
        const int32_t rt = (int32_t)(item / nt);
        int32_t lo = 0, hi = p.G;  // largest g with tiles[g] <= rt
        while (hi - lo > 1) {
            const int32_t mid = (lo + hi) >> 1;
            if (tiles[mid] <= rt) lo = mid; else hi = mid;
        }
        it.g = lo;
        const int32_t first = tiles[lo], cnt = tiles[lo + 1] - first;
        const uint32_t l = item - (uint32_t)first * nt;
        const uint32_t band = l / (kRaster * nt);
        const uint32_t r = l - band * (kRaster * nt);
        const uint32_t rows = min((uint32_t)kRaster, (uint32_t)cnt - band * kRaster);
        it.n = (int32_t)(r / rows);
        const int32_t j = (int32_t)(band * kRaster + r - (uint32_t)it.n * rows);
        it.tile = first + j;
        row_tile(it, lo, cnt, j);
        if (kAdapters && it.x1 < 0) it.x1 = extra_blocks(p, nslots[it.tile]);
        return true;
    }
};

// ------------------------------------------------------------------ numbers

__device__ __forceinline__ uint16_t round16(float x, int32_t bf16) {
    if (bf16) return __bfloat16_as_ushort(__float2bfloat16_rn(x));
    return __half_as_ushort(__float2half_rn(x));
}

// Two values rounded to nearest-even 16-bit floats, a in the low half.
__device__ __forceinline__ uint32_t pack16(float a, float b, int32_t bf16) {
    if (bf16) {
        __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t*>(&h);
    }
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ float2 unpack16(uint32_t x, int32_t bf16) {
    if (bf16) return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&x));
}

// What rounding x and y to the pair `hi` left out, rounded (nothing where hi
// is not finite).
__device__ __forceinline__ uint32_t rest16x2(float x, float y, uint32_t hi, int32_t bf16) {
    const float2 back = unpack16(hi, bf16);
    return pack16(isfinite(back.x) ? x - back.x : 0.0f, isfinite(back.y) ? y - back.y : 0.0f, bf16);
}

// v[at] += x for an index that is not a constant (the array stays in registers).
__device__ __forceinline__ void add_at(float (&v)[32], int at, float x) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] += j == at ? x : 0.0f;
}

// A pair of 16-bit floats, each +0 where its gate is not positive (sign set,
// zero or NaN), as unsigned compares of the gate's words.
__device__ __forceinline__ uint32_t gate16(uint32_t x, uint32_t gate, int32_t bf16) {
    const uint32_t inf = bf16 ? 0x7F80u : 0x7C00u;
    const uint32_t lo = (gate & 0xFFFFu) - 1u < inf ? 0x0000FFFFu : 0u;
    const uint32_t hi = (gate >> 16) - 1u < inf ? 0xFFFF0000u : 0u;
    return x & (lo | hi);
}

// ------------------------------------------------------------------ kernel

template <bool kPair, bool kAdapters>
__global__ void __maxnreg__(128)  // (adapters: leaves room for a block of the low kernel)
    ragged_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
    constexpr int kCG = kPair ? 2 : 1;
    constexpr uint32_t kEpi = epi_threads(kAdapters);
    using It = Iter<kPair, kAdapters>;
    extern __shared__ __align__(1024) uint8_t smem[];
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem);
    const uint32_t ring = (smem_u32(smem) + (uint32_t)sizeof(Ctrl) + 1023u) & ~1023u;
    int32_t* const start = reinterpret_cast<int32_t*>(smem + (ring - smem_u32(smem)) + p.table_off);
    int32_t* const tiles = start + p.G + 1;
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = kPair ? cluster_ctarank() : 0u;
    const bool clustered = !kPair && p.cluster > 1;
    // A launch of low items has no helping warps.  They wait on an
    // accumulator's phase parity, so they have to be the ones that release
    // every accumulator they pass: were one released by other warps, two more
    // items could end before they look, and the parity would be that of a later one.
    const bool helpers = kPair && kAdapters && blockDim.x == kHelped;
    const uint32_t share = clustered ? cluster_ctarank() : 0u;
    const uint32_t worker = kPair ? blockIdx.x / 2 : clustered ? blockIdx.x / (uint32_t)p.cluster : blockIdx.x;
    const uint32_t workers = kPair ? gridDim.x / 2 : clustered ? gridDim.x / (uint32_t)p.cluster : gridDim.x;

    if (warp == 2 && lane == 0) {
        for (int s = 0; s < p.num_stages; ++s) {
            mbar_init(smem_u32(&ctrl->full[s]), 1);
            mbar_init(smem_u32(&ctrl->empty[s]), 1);
            mbar_init(smem_u32(&ctrl->extra[s]), 1);
            mbar_init(smem_u32(&ctrl->peer[s]), 1);
            mbar_init(smem_u32(&ctrl->boxes[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&ctrl->tmem_full[b]), 1);
            mbar_init(smem_u32(&ctrl->tmem_empty[b]), (kPair ? 2u : 1u) * (kEpi / 32));
        }
        mbar_init(smem_u32(&ctrl->final_bar), 1);
        ctrl->helped = ctrl->sick_item = 0;
        ctrl->abort_flag = 0;
        ctrl->ring_s = ctrl->ring_ph = ctrl->ring_lap = 0;
        for (int i = 0; i < kMaxBoxes / 32; ++i) ctrl->sick[i] = 0u;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc<kCG>(smem_u32(&ctrl->tmem_addr), p.tmem_cols);
        tmem_relinquish<kCG>();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&maps.w);
        tma_prefetch_desc(&maps.x[0]);
    }
    // Nothing before this reads or writes global memory.  The adapters' main
    // launch goes on: the one before it in the stream computes low and
    // nothing else, and lets this one start only after it has itself waited
    // for all that came before, so X, W, ids, the slot lists and the
    // workspace are ready and Y is free; low alone is waited for where it is
    // read, after the main k-blocks.  (So a launch of low items waits first.
    // The main one starts only once all its CTAs have, that is, are resident
    // or done: what the main CTAs wait for never waits for a place of theirs.)
    const bool lows_only = kPair && kAdapters && p.low_out;
    if (lows_only) grid_dependency_wait();
    grid_launch_dependents();
    if (!kAdapters) grid_dependency_wait();
    int32_t* const lows = tiles + p.G + 1;
    if (warp == 6) {
        build_table(p, start, tiles, lane, workers);
        if (lows_only) {
            __syncwarp();
            int32_t before = 0;
            for (int32_t t0 = 0; t0 < tiles[1]; t0 += 32) {
                const int32_t t = t0 + (int32_t)lane;
                int32_t n = t < tiles[1] ? low_items(p, __ldcg(p.nslots + t)) : 0;
                const int32_t mine = n;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int32_t o = __shfl_up_sync(0xffffffffu, n, d);
                    if ((int)lane >= d) n += o;
                }
                if (t < tiles[1]) lows[t] = before + n - mine;
                before += __shfl_sync(0xffffffffu, n, 31);
            }
            if (lane == 0) lows[tiles[1]] = before;
        }
    }
    __syncwarp();
    tc_fence_before();
    if (kPair)
        cluster_sync();
    else
        cta_barrier_sync();
    tc_fence_after();
    const int32_t* nslots = p.nslots;
    const int32_t* slot_list = p.slots;
    int32_t* const row_ids = tiles + p.G + 1;  // single CTAs of adapters: one row tile, listed by each
    int32_t* const windows = row_ids + 256;
    if constexpr (kAdapters) {
        if (!kPair) {
            if (warp >= 2 && warp <= 5)
                list_slots(p, row_ids, row_ids + 128, windows, row_ids + 384, row_ids + 388, (int32_t)threadIdx.x - 64);
            slot_list = row_ids + 128;
            nslots = row_ids + 388;
            __syncwarp();
            cta_barrier_sync();
        }
    }
    // (single CTAs: every item has the one row tile's extra k-blocks)
    const int32_t max_extra = kAdapters && !kPair ? extra_blocks(p, *nslots) : 0;
    // rows [lo, hi) that the 16 products from column `col` of the extra
    // k-blocks reach (two adapters of 8 products: both)
    auto window = [&](int32_t slots, int32_t col, uint32_t& lo, uint32_t& hi) {
        const int32_t a = slot_of(p, col >> p.box_shift), b = slot_of(p, (col + 8) >> p.box_shift);
        const uint32_t wa = (uint32_t)windows[a];
        lo = wa & 0xFFFFu;
        hi = wa >> 16;
        if (b != a && b < slots) {
            const uint32_t wb = (uint32_t)windows[b];
            lo = min(lo, wb & 0xFFFFu);
            hi = max(hi, wb >> 16);
        }
    };
    const uint32_t tmem_base = ctrl->tmem_addr;
    const uint32_t S = (uint32_t)p.num_stages, stride = (uint32_t)p.stage_bytes;
    const uint32_t full0 = smem_u32(&ctrl->full[0]), empty0 = smem_u32(&ctrl->empty[0]);
    It iter(p, start, tiles, nslots, lows, worker, workers, max_extra, (int32_t)share);
    Item it;

    // pieces (boxes of rank_box rows of an adapter's second factor) of extra
    // k-block e of a tile with `slots` adapters; a box of 8 rows is half of
    // an MMA's 16, so their number is made even with one of zeros
    auto pieces_of = [&](int32_t slots, int32_t e) {
        const int32_t per = kXK >> p.box_shift;
        int32_t n = min(per, slots * p.per_slot - e * per);
        if (p.rank_box == 8) n = (n + 1) & ~1;
        return n;
    };

    // boxes of rank_box products of a low item that CTA r of the pair holds
    auto low_pieces = [&](const Item& i, int32_t slots, uint32_t r) {
        const int32_t per = low_boxes(p, slots);
        return max(0, min(per, slots * p.per_slot - (2 * i.n + (int32_t)r) * per));
    };
    // expect a stage's bytes (of both CTAs of a pair) on its barrier
    auto arm = [&](uint32_t full, uint32_t bytes) {
        if (!kPair || rank == 0) mbar_arrive_expect_tx(full, bytes);
    };

    if (warp == 0) {
        // ---------------------------------------------------------- row tiles
        if (lane == 0) {
            uint32_t s = 0, ph = 0;
            uint32_t pos = 0;  // stages passed
            bool ok = true;
            while (ok && iter.next(it)) {
                const uint32_t rows = (uint32_t)it.w / (kPair ? 2u : 1u);
                const int32_t y = it.row0 + (int32_t)(rank * rows);
                uint32_t bytes = (kPair ? 2u : 1u) * (kWBytes + rows * (uint32_t)(kBK * 2));
                if constexpr (kPair && kAdapters) {
                    if (it.low)
                        bytes = (uint32_t)((low_pieces(it, nslots[it.tile], 0) + low_pieces(it, nslots[it.tile], 1)) *
                                           p.rank_box) * 256u + 2u * rows * (uint32_t)(kBK * 2);
                }
                const CUtensorMap* m = &maps.x[rows / 16 - 1];
                for (int32_t kb = it.kb0; kb < it.kb1; ++kb) {
                    if (!wait_phase(empty0 + 8u * s, ph ^ 1u, ctrl, p, kErrTokens)) {
                        ok = false;
                        break;
                    }
                    const uint32_t full = full0 + 8u * s;
                    arm(full, bytes);
                    const uint32_t dst = ring + s * stride + kWBytes;
                    const uint32_t bar = kPair ? mapa_shared(full, 0) : full;
                    if (!kPair && kb == p.test_drop_kb - 1 && pos == (uint32_t)(kb - it.kb0)) {
                        // (test hook: not copied)
                    } else if (p.x3d) {
                        load_3d<kPair>(dst, m, bar, 0, y, kb * (kBK / 64));
                    } else {
                        load_2d<kPair>(dst, m, bar, kb * kBK, y);
                        load_2d<kPair>(dst + rows * 128u, m, bar, kb * kBK + 64, y);
                    }
                    ++pos;
                    if (++s == S) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if constexpr (kAdapters) {
                    // the epilogue's warps fill and arm the extra k-blocks;
                    // this thread, which is never more than a lap ahead of
                    // the MMAs, tells them when a stage is free
                    for (int32_t e = it.x0; ok && e < it.x1; ++e) {
                        ok = wait_phase(empty0 + 8u * s, ph ^ 1u, ctrl, p, kErrTokens);
                        if (!ok) break;
                        mbar_arrive(smem_u32(&ctrl->extra[s]));
                        ++pos;
                        if (++s == S) {
                            s = 0;
                            ph ^= 1u;
                        }
                    }
                }
            }
            if (!kPair || rank == 0) {
                // what an aborting CTA waits for before its shared memory is released
                ctrl->ring_s = (int32_t)(pos % S);
                ctrl->ring_ph = (int32_t)((pos / S) & 1u);
                ctrl->ring_lap = pos >= S ? 1 : 0;
            }
        }
        __syncwarp();
    } else if (warp == 6) {
        // ------------------------------------------------------------ weights
        uint32_t s = 0, ph = 0;
        bool ok = true;
        while (ok && iter.next(it)) {
            const int32_t n0 = it.n * (kPair ? 256 : 128) + 128 * (int32_t)rank;
            const int32_t n_main = it.kb1 - it.kb0;
            if (kPair && kAdapters && it.low) {
                // first factors of the tile's adapters, 128 rows per CTA; a
                // lane per box of rank_box rows x 64 k
                const int32_t slots = nslots[it.tile], mine = low_pieces(it, slots, rank);
                const int32_t per = low_boxes(p, slots);
                const int32_t piece = (2 * it.n + (int32_t)rank) * per + (int32_t)(lane >> 1);
                const int32_t slot = slot_of(p, piece);
                const bool one = per == 1 && p.a4d;  // both 64-k boxes in one copy
                const bool has = (int32_t)(lane >> 1) < mine && !(one && (lane & 1u));
                const uint32_t sub = (per == 1 ? (uint32_t)p.rank_box : 128u) * 128u;  // from one 64 k to the next
                const int32_t id = has ? slot_list[(int64_t)it.tile * p.cap + slot] : 0;
                uint32_t ls = s, lph = ph;
                for (int32_t kb = 0; kb < it.kb1; ++kb) {
                    ok = wait_phase(empty0 + 8u * ls, lph ^ 1u, ctrl, p, kErrWeights);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const int32_t row = (piece - slot * p.per_slot) * p.rank_box;
                    if (has && one)
                        load_4d<kPair>(ring + ls * stride, &maps.a4, mapa_shared(full0 + 8u * ls, 0), 0, row,
                                       kb * (kBK / 64), id);
                    else if (has)
                        load_3d<kPair>(ring + ls * stride + (lane & 1u) * sub + (lane >> 1) * (uint32_t)p.rank_box * 128u,
                                       &maps.a, mapa_shared(full0 + 8u * ls, 0), kb * kBK + 64 * (int32_t)(lane & 1u),
                                       row, id);
                    __syncwarp();
                    if (++ls == S) {
                        ls = 0;
                        lph ^= 1u;
                    }
                }
            } else if (lane == 0) {
                uint32_t ls = s, lph = ph;
                for (int32_t kb = it.kb0; kb < it.kb1; ++kb) {
                    if (!wait_phase(empty0 + 8u * ls, lph ^ 1u, ctrl, p, kErrWeights)) {
                        ok = false;
                        break;
                    }
                    const uint32_t full = full0 + 8u * ls;
                    const uint32_t bar = kPair ? mapa_shared(full, 0) : full;
                    const uint32_t dst = ring + ls * stride;
                    const int32_t k0 = kb * kBK;
                    if constexpr (!kPair && kAdapters) {
                        // read once: not to push the factors out of L2
                        const uint64_t once = l2_policy_evict_first();
                        if (p.w4d) {
                            load_4d_hint(dst, &maps.w, bar, 0, p.w_kmajor ? n0 : k0, (p.w_kmajor ? k0 : n0) / 64, it.g, once);
                        } else if (p.w_kmajor) {
                            load_3d_hint(dst, &maps.w, bar, k0, n0, it.g, once);
                            load_3d_hint(dst + 128u * 128u, &maps.w, bar, k0 + 64, n0, it.g, once);
                        } else {
                            load_3d_hint(dst, &maps.w, bar, n0, k0, it.g, once);
                            load_3d_hint(dst + (uint32_t)kBK * 128u, &maps.w, bar, n0 + 64, k0, it.g, once);
                        }
                    } else if (p.w4d) {
                        if (p.w_kmajor)
                            load_4d<kPair>(dst, &maps.w, bar, 0, n0, k0 / 64, it.g);
                        else
                            load_4d<kPair>(dst, &maps.w, bar, 0, k0, n0 / 64, it.g);
                    } else if (p.w_kmajor) {
                        load_3d<kPair>(dst, &maps.w, bar, k0, n0, it.g);
                        load_3d<kPair>(dst + 128u * 128u, &maps.w, bar, k0 + 64, n0, it.g);
                    } else {
                        load_3d<kPair>(dst, &maps.w, bar, n0, k0, it.g);
                        load_3d<kPair>(dst + (uint32_t)kBK * 128u, &maps.w, bar, n0 + 64, k0, it.g);
                    }
                    if (++ls == S) {
                        ls = 0;
                        lph ^= 1u;
                    }
                }
            }
            ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
            const uint32_t adv = s + (uint32_t)n_main;
            ph ^= (adv / S) & 1u;
            s = adv % S;
            if constexpr (kAdapters) {
                const int32_t slots = nslots[it.tile];
                const int32_t per = kXK >> p.box_shift;
                for (int32_t e = it.x0; ok && e < it.x1; ++e) {
                    ok = wait_phase(empty0 + 8u * s, ph ^ 1u, ctrl, p, kErrWeights);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const uint32_t bar = smem_u32(&ctrl->boxes[s]);  // (this CTA's own, of a pair too)
                    const int32_t pieces = pieces_of(slots, e);
                    if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(pieces * p.rank_box) * 256u);
                    __syncwarp();
                    if ((int32_t)lane < pieces) {
                        const int32_t piece = e * per + (int32_t)lane;
                        const int32_t slot = slot_of(p, piece);
                        // (past the last adapter a box of zeros, beyond the tensor)
                        const int32_t id = slot < slots ? slot_list[(int64_t)it.tile * p.cap + slot] : p.R;
                        const int32_t row = (piece - slot * p.per_slot) * p.rank_box;
                        const uint32_t dst = ring + s * stride + lane * (uint32_t)p.rank_box * 256u;
                        if (p.b4d) {
                            load_4d<false>(dst, &maps.b, bar, 0, row, n0 / 64, id);
                        } else {
                            load_3d<false>(dst, &maps.b, bar, n0, row, id);
                            load_3d<false>(dst + (uint32_t)p.rank_box * 128u, &maps.b, bar, n0 + 64, row, id);
                        }
                    }
                    __syncwarp();
                    if (++s == S) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA
        if (lane == 0 && (!kPair || rank == 0)) {
            const uint32_t tfull0 = smem_u32(&ctrl->tmem_full[0]), tempty0 = smem_u32(&ctrl->tmem_empty[0]);
            const uint32_t cols = p.tmem_cols / 2;
            const uint32_t idesc0 = make_idesc_f16_f32(kPair ? 256 : 128, 0, !p.w_kmajor, false, p.bf16 != 0);
            const uint32_t idesc_k = make_idesc_f16_f32(kPair ? 256 : 128, 0, false, false, p.bf16 != 0);
            const uint32_t idesc1 = make_idesc_f16_f32(kPair ? 256 : 128, 0, true, false, p.bf16 != 0);
            constexpr uint32_t kK = kBK / 16;
            // weights: MN-major, 64-column chunks of kBK k-rows (16 k-rows =
            // two 1024-byte atoms per MMA), or K-major, 128 rows per 64 k
            const uint64_t a_desc0 = p.w_kmajor ? make_sw128_desc(ring, 16, 1024)
                                                : make_sw128_desc(ring, (uint32_t)kBK * 128u, 1024);
            const uint64_t a_desc_k = make_sw128_desc(ring, 16, 1024);
            const uint64_t b_desc0 = make_sw128_desc(ring + kWBytes, 16, 1024);
            uint32_t a_off[kK];
#pragma unroll
            for (uint32_t k = 0; k < kK; ++k)
                a_off[k] = p.w_kmajor ? (k / 4) * (128u * 128u >> 4) + (k % 4) * 2u : k * (2048u >> 4);
            const uint32_t stride16 = stride >> 4;
            uint32_t s = 0, ph = 0, local = 0;
            bool ok = true;
            while (ok && iter.next(it)) {
                const uint32_t buf = local & 1u, bph = (local >> 1) & 1u;
                if (!wait_phase(tempty0 + 8u * buf, bph ^ 1u, ctrl, p, kErrAccum)) break;
                tc_fence_after();
                const uint32_t d = tmem_base + buf * cols;
                const uint32_t nbits = ((uint32_t)it.w >> 3) << 17;
                const uint32_t half16 = ((uint32_t)it.w / (kPair ? 2u : 1u)) * 128u >> 4;  // second 64 k of the rows
                uint32_t acc = 0;
                // the k-blocks; weights from `a_first`, k-step k at offset(k)
                auto main_blocks = [&](uint64_t a_first, uint32_t idesc, auto offset) {
                    for (int32_t kb = it.kb0; kb < it.kb1; ++kb) {
                        if (!wait_phase(full0 + 8u * s, ph, ctrl, p, kErrStage)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t a_desc = a_first + (uint64_t)(s * stride16);
                        const uint64_t b_desc = b_desc0 + (uint64_t)(s * stride16);
#pragma unroll
                        for (uint32_t k = 0; k < kK; ++k)
                            mma_f16_ss<kCG>(d, a_desc + offset(k), b_desc + (k / 4) * half16 + (k % 4) * 2u, idesc,
                                            k > 0 ? 1u : acc);
                        acc = 1;
                        mma_commit<kCG>(empty0 + 8u * s, 0x3);
                        if (++s == S) {
                            s = 0;
                            ph ^= 1u;
                        }
                    }
                };
                if (kPair && kAdapters && it.low) {
                    // (one box: the MMA's rows past it read what lies there, into lanes that nothing reads)
                    const uint32_t sub16 =
                        (low_boxes(p, nslots[it.tile]) == 1 ? (uint32_t)p.rank_box : 128u) * 128u >> 4;
                    main_blocks(a_desc_k, idesc_k | nbits, [=](uint32_t k) { return (k / 4) * sub16 + (k % 4) * 2u; });
                } else {
                    main_blocks(a_desc0, idesc0 | nbits, [&](uint32_t k) { return a_off[k]; });
                }
                if constexpr (kAdapters) {
                    const int32_t slots = nslots[it.tile];
                    const uint32_t box = (uint32_t)p.rank_box;
                    // second factors: boxes of `box` k-rows x two 64-column
                    // chunks; boxes of 8 rows pair up to an MMA's 16
                    const uint64_t x_desc0 = box == 8 ? make_sw128_desc(ring, 1024, 2048)
                                                      : make_sw128_desc(ring, box * 128u, 1024);
                    for (int32_t e = it.x0; ok && e < it.x1; ++e) {
                        if (!wait_phase(full0 + 8u * s, ph, ctrl, p, kErrStage)) {
                            ok = false;
                            break;
                        }
                        if (kPair) fence_acq_rel_cluster();  // the peer wrote its rows itself
                        tc_fence_after();
                        const uint64_t a_desc = x_desc0 + (uint64_t)(s * stride16);
                        const uint64_t b_desc = b_desc0 + (uint64_t)(s * stride16);
                        const uint32_t nk = (uint32_t)pieces_of(slots, e) << p.box_shift >> 4;
                        // hi's columns, then lo's, with the same rows of the factors
#pragma unroll
                        for (uint32_t k = 0; k < kXK / 16; ++k) {
                            if (k >= nk) break;
                            const uint32_t r = 16u * k;
                            const uint32_t off = box == 8 ? k * 4096u : (r & ~(box - 1u)) * 256u + (r & (box - 1u)) * 128u;
                            uint32_t lo = 0, hi = (uint32_t)it.w;
                            if (!kPair && (e > it.x0 || it.kb0 < it.kb1))
                                window(slots, e * kXK + (int32_t)r, lo, hi);
                            const uint32_t idesc_x = idesc1 | (((hi - lo) >> 3) << 17);
                            const uint64_t bd = b_desc + (lo * 128u >> 4) + k * 2u;
                            mma_f16_ss<kCG>(d + lo, a_desc + (off >> 4), bd, idesc_x, acc);
                            mma_f16_ss<kCG>(d + lo, a_desc + (off >> 4), bd + half16, idesc_x, 1u);
                            acc = 1;
                        }
                        mma_commit<kCG>(empty0 + 8u * s, 0x3);
                        if (++s == S) {
                            s = 0;
                            ph ^= 1u;
                        }
                    }
                }
                if (!ok) break;
                mma_commit<kCG>(tfull0 + 8u * buf, 0x3);
                ++local;
            }
            mma_commit<kCG>(smem_u32(&ctrl->final_bar), 0x1);
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(smem_u32(&ctrl->final_bar), 0))
                if (globaltimer_ns() - t0 > p.timeout_ns) {
                    atomicCAS(p.err, 0, (int32_t)kErrFinal);
                    break;
                }
        }
        __syncwarp();
    } else {
        // ----------------------------------------------------------- epilogue
        const uint32_t quarter = warp & 3u, half = warp > 6 ? 1u : 0u;
        constexpr int32_t kChunkStep = (int32_t)kEpi / 4;  // from one of a warp's chunks of 32 rows to its next
        const int32_t chunk0 = kAdapters ? 0 : 32 * (int32_t)half;
        const uint32_t group_barrier = kEpiBarrier + (kAdapters ? half : 0u);
        const uint32_t lane_row = quarter * 32 + lane;
        const uint32_t cols = p.tmem_cols / 2;
        uint32_t local = 0;
        float v[32];
        const uint32_t turn = ring + (uint32_t)p.turn_off + (quarter + 4u * half) * (32u * kTurnPitch);
        const uint32_t turn_st = turn + (lane & 7u) * kTurnPitch + (lane >> 3) * 16u;
        const uint32_t turn_ld = turn + (lane >> 2) * kTurnPitch + (lane & 3u) * 16u;
        const uint32_t et = threadIdx.x - 64 - (kAdapters ? 160 : 32) * half;  // (warp 6 has another role)
        uint32_t pos = 0;  // adapters: ring stages before the item's extra ones
        uint32_t extra_ph = 0;  // ... and the phase of each stage's `extra` barrier
        bool any_sick = false;  // ... and whether any of the item's boxes is kept out of the MMAs
        // Adapters, few rows: the item's second factors to L2 before the main
        // k-blocks' copies fill DRAM's queues (a thread per row, two lines).
        auto ask_for_boxes = [&]() {
            const int32_t slots = nslots[it.tile], per = kXK >> p.box_shift;
            const int32_t b0 = it.x0 * per, rows = (min(it.x1 * per, slots * p.per_slot) - b0) << p.box_shift;
            for (int32_t r = (int32_t)et; r < rows; r += (int32_t)kEpi) {
                const int32_t box = b0 + (r >> p.box_shift), slot = slot_of(p, box);
                const int32_t j = ((box - slot * p.per_slot) << p.box_shift) + (r & (p.rank_box - 1));
                if (j >= p.rank) continue;
                const int64_t row = (int64_t)slot_list[(int64_t)it.tile * p.cap + slot] * p.rank + j;
                for (int32_t n = it.n * 128; n < min(it.n * 128 + 128, p.N); n += 64) prefetch_line(p.B + row * p.N + n);
            }
        };
        // The second factors of an extra k-block, once they have landed: a
        // row's columns of other adapters are zeros in its low-rank part, and
        // zero times an infinity or NaN is not zero, so a box that is not
        // finite is made zeros here and its own rows get its products from the
        // epilogue: one adapter's broken weights stay in its rows.  Looked at
        // in shared memory: a read of them in global memory, ahead of the copies,
        // stood in DRAM's queues behind the weights (64 rows, 48 adapters of
        // rank 32, 8192 x 8192: 56.5 us, so 47.3).
        // (exponent all ones: adding its lowest bit carries into the sign's place)
        const uint32_t inf = p.bf16 ? 0x7F807F80u : 0x7C007C00u, low_bit = p.bf16 ? 0x00800080u : 0x04000400u;
        auto carries = [&](const uint4& q) {
            return ((q.x & inf) + low_bit) | ((q.y & inf) + low_bit) | ((q.z & inf) + low_bit) | ((q.w & inf) + low_bit);
        };
        auto vec_finite = [&](const uint4& q) { return (carries(q) & 0x80008000u) == 0u; };
        auto boxes_finite = [&](uint32_t at, int32_t vecs) {
            constexpr int32_t kEach = kXK * 16 / (int32_t)kEpi;  // vectors of a thread
            uint32_t bad = 0;
#pragma unroll
            for (int32_t i0 = 0; i0 < kEach; i0 += 4) {
                uint4 q[4];
#pragma unroll
                for (int32_t i = 0; i < 4; ++i) {
                    const int32_t v = (int32_t)et + (i0 + i) * (int32_t)kEpi;
                    q[i] = ld_shared_v4(at + 16u * (uint32_t)min(v, vecs - 1));
                }
#pragma unroll
                for (int32_t i = 0; i < 4; ++i) bad |= carries(q[i]);
            }
            return (bad & 0x80008000u) == 0u;
        };
        // ... and the boxes of block e that are not finite to zeros (all threads)
        auto clear_boxes = [&](uint32_t at, int32_t vecs, int32_t e) {
            const int32_t b0 = e * (kXK >> p.box_shift), shift = p.box_shift + 4;  // vectors of a box, as a power of two
            for (int32_t v = (int32_t)et; v < vecs; v += (int32_t)kEpi)
                if (!vec_finite(ld_shared_v4(at + 16u * (uint32_t)v))) {
                    const int32_t box = b0 + (v >> shift);
                    atomicOr(&ctrl->sick[box >> 5], 1u << (box & 31));
                }
            named_bar_sync(kEpiBarrier, kEpi);
            for (int32_t v = (int32_t)et; v < vecs; v += (int32_t)kEpi) {
                const int32_t box = b0 + (v >> shift);
                if ((ctrl->sick[box >> 5] >> (box & 31)) & 1u) st_shared_v4(at + 16u * (uint32_t)v, make_uint4(0, 0, 0, 0));
            }
            fence_proxy_async_smem();
            named_bar_sync(kEpiBarrier, kEpi);
        };
        // The products of the boxes kept out, for one of their own rows: what
        // row t's low-rank part is to have in column n besides.
        auto sick_part = [&](int32_t t, int32_t n) {
            float sum = 0.0f;
            const int32_t his = t < it.row0 + it.valid && n < p.N ? __ldcg(p.ids + t) : -1, per = kXK >> p.box_shift;
            for (int32_t box = it.x0 * per; his >= 0 && box < min(it.x1 * per, nslots[it.tile] * p.per_slot); ++box) {
                if (((ctrl->sick[box >> 5] >> (box & 31)) & 1u) == 0) continue;
                const int32_t slot = slot_of(p, box), j0 = (box - slot * p.per_slot) * p.rank_box;
                if (slot_list[(int64_t)it.tile * p.cap + slot] != his) continue;
                const uint16_t* low = p.low + (int64_t)t * 2 * p.rank_pad;
                for (int32_t j = j0; j < min(j0 + p.rank_box, p.rank); ++j) {
                    const float2 b = unpack16(p.B[((int64_t)his * p.rank + j) * p.N + n], p.bf16);
                    const float2 hi = unpack16(__ldcg(low + j), p.bf16), rest = unpack16(__ldcg(low + p.rank_pad + j), p.bf16);
                    sum = fmaf(hi.x, b.x, sum);
                    if (rest.x != 0.0f) sum = fmaf(rest.x, b.x, sum);  // (0 x inf would be NaN)
                }
            }
            return sum;
        };
        // Adapters: fill and arm an item's extra k-blocks.  A row tile's
        // low-rank products, each row only in its own adapter's columns: 64
        // columns of hi, then of lo.  Thread = 16-byte vector (8 columns) of
        // one of eight rows at a time, copied (or zeros) to the 128-byte
        // swizzle's place; one block's copies fly while the next one's are
        // issued.
        auto fill_extras = [&]() {
            const int32_t slots = nslots[it.tile];
            const int32_t e0 = it.x0, e1 = it.x1;
            pos += (uint32_t)(it.kb1 - it.kb0);
            if (e0 >= e1) return true;
            const uint32_t rows = (uint32_t)it.w / (kPair ? 2u : 1u);
            const int32_t y = it.row0 + (int32_t)(rank * rows);
            bool ok = true;     // (alike in all threads)
            bool armed = true;  // of the thread that arms
            grid_dependency_wait();  // low is complete
            const uint32_t v = et & 15u, r0 = et >> 4;
            int32_t who[kPair ? 16 : 1];  // adapters of rows r0, r0 + 8, ...
            if constexpr (kPair) {
#pragma unroll
                for (uint32_t j = 0; j < 16; ++j) {
                    const int32_t t = y + (int32_t)(r0 + 8u * j);
                    who[j] = r0 + 8u * j < rows && t < it.row0 + it.valid ? __ldcg(p.ids + t) : -1;
                }
            }
            // Blocks in flight: stage e + S - 2 is free while the MMAs work
            // on block e - 1, in time for e.
            const int32_t ahead = max(0, min(3, (int32_t)S - 2));
            int32_t issued = e0;
            for (int32_t e = e0; ok && e < e1; ++e) {
                for (; issued < e1 && issued <= e + ahead; ++issued) {
                    const uint32_t st = (pos + (uint32_t)(issued - e0)) % S;
                    ok = wait_phase(smem_u32(&ctrl->extra[st]), (extra_ph >> st) & 1u, ctrl, p, kErrTokens);
                    extra_ph ^= 1u << st;
                    ok = named_bar_and(kEpiBarrier, kEpi, ok);
                    if (!ok) break;
                    const int32_t col = issued * kXK + 8 * (int32_t)(v & 7u);
                    const int32_t slot = slot_of(p, col >> p.box_shift);
                    // (no row's where no adapter's: rows' ids, as they are, may be anything)
                    const bool real = slot < slots;
                    const int32_t id = real ? slot_list[(int64_t)it.tile * p.cap + slot] : -1;
                    const uint16_t* src = p.low + (int64_t)y * 2 * p.rank_pad + (col - slot * p.rank_pad) +
                                          (int32_t)(v >> 3) * p.rank_pad;
                    const uint32_t dst = ring + st * stride + kWBytes + (v >> 3) * rows * 128u;
                    auto put = [&](uint32_t i, bool his) {
                        copy_async_16(dst + i * 128u + (((v & 7u) ^ (i & 7u)) << 4),
                                      his ? src + (int64_t)i * 2 * p.rank_pad : p.low, his ? 16u : 0u);
                    };
                    if constexpr (kPair) {
#pragma unroll
                        for (uint32_t j = 0; j < 16; ++j)
                            if (r0 + 8u * j < rows) put(r0 + 8u * j, real && who[j] == id);
                    } else if ((col & ~15) < slots * p.rank_pad) {
                        // only the rows that the MMAs of these columns read
                        // (all where they begin an accumulator)
                        uint32_t lo = 0, hi = rows;
                        if (issued > e0 || it.kb0 < it.kb1) window(slots, col & ~15, lo, hi);
                        for (uint32_t i = lo + r0; i < hi; i += 8) put(i, real && row_ids[i] == id);
                    }
                    copy_async_commit();
                }
                if (!ok) break;
                switch (issued - e) {
                    case 1: copy_async_wait<0>(); break;
                    case 2: copy_async_wait<1>(); break;
                    case 3: copy_async_wait<2>(); break;
                    default: copy_async_wait<3>(); break;
                }
                fence_proxy_async_smem();
                // (extra_ph has moved on once since this block, the last use of its stage)
                const uint32_t st = (pos + (uint32_t)(e - e0)) % S, phase = ((extra_ph >> st) & 1u) ^ 1u;
                const uint32_t at = ring + st * stride;
                const int32_t vecs = pieces_of(slots, e) * p.rank_box * 16;
                const bool landed = wait_phase(smem_u32(&ctrl->boxes[st]), phase, ctrl, p, kErrEpi);
                if (!named_bar_and(kEpiBarrier, kEpi, landed && boxes_finite(at, vecs))) {
                    ok = named_bar_and(kEpiBarrier, kEpi, landed);
                    if (!ok) break;
                    clear_boxes(at, vecs, e);
                    any_sick = true;
                    if (et == 0) *(volatile int32_t*)&ctrl->sick_item = (int32_t)local + 1;
                }
                if (et == 0) {
                    if (kPair && rank != 0) {
                        mbar_arrive_cluster(mapa_shared(smem_u32(&ctrl->peer[st]), 0));
                    } else {
                        if (kPair && armed) armed = wait_cluster(smem_u32(&ctrl->peer[st]), phase, ctrl, p);
                        if (armed) mbar_arrive(full0 + 8u * st);
                    }
                }
            }
            pos += (uint32_t)(e1 - e0);
            return named_bar_and(kEpiBarrier, kEpi, ok && armed);
        };
        // the item whose accumulator is the CTA's `local`-th; false: aborting
        auto drain = [&](const Item& it, uint32_t local) {
            const uint32_t buf = local & 1u, bph = (local >> 1) & 1u;
            auto ready = [&]() {
                bool ok = wait_phase(smem_u32(&ctrl->tmem_full[buf]), bph, ctrl, p, kErrEpi);
                ok = named_bar_and(group_barrier, kEpi, ok);
                tc_fence_after();
                if (kAdapters && half) any_sick = *(volatile int32_t*)&ctrl->sick_item == (int32_t)local + 1;
                return ok;
            };
            const uint32_t taddr = tmem_base + ((quarter * 32u) << 16) + buf * cols;
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (kPair)
                        mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&ctrl->tmem_empty[buf]), 0));
                    else
                        mbar_arrive(smem_u32(&ctrl->tmem_empty[buf]));
                }
            };
            if constexpr (kPair && kAdapters) {
                if (it.low) {
                    const int32_t slots = nslots[it.tile];
                    const int32_t held = low_boxes(p, slots) * p.rank_box;  // products of each CTA
                    const int32_t r0 = (2 * it.n + (int32_t)rank) * held;   // its first
                    // scale of this thread's fragment rows; columns past the
                    // rank are zeros whatever the scale is
                    float scale[4];
                    bool keep[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int32_t r = r0 + 32 * (int32_t)quarter + 8 * k + (int32_t)(lane >> 2);
                        const int32_t slot = slot_of(p, r >> p.box_shift);
                        keep[k] = slot < slots && r - slot * p.rank_pad < p.rank;
                        scale[k] = keep[k] && p.scale ? __ldcg(p.scale + slot_list[(int64_t)it.tile * p.cap + slot])
                                                      : 1.0f;
                    }
                    // after the transposition: eight products of adapter id, from number j
                    const int32_t col = 32 * (int32_t)quarter + 8 * (int32_t)(lane & 3u);
                    const int32_t slot = slot_of(p, (r0 + col) >> p.box_shift), j = r0 + col - slot * p.rank_pad;
                    // (no row's where this thread holds no adapter's products:
                    // rows' ids, as they are, may be anything)
                    const bool real = col < held && slot < slots;
                    const int32_t id = real ? slot_list[(int64_t)it.tile * p.cap + slot] : -1;
                    // adapter of row c + lane, asked for a chunk ahead
                    auto who_at = [&](int32_t r) { return r < it.valid ? __ldcg(p.ids + it.row0 + r) : -1; };
                    int32_t who = who_at((int32_t)lane);
                    if (!ready()) return false;
                    // (not unrolled: it runs once per item, and the code of all
                    // chunks came from memory, 16 us for eight of them)
#pragma unroll 1
                    for (int32_t c = 0; c < it.w; c += 32) {
                        const int32_t coming = who_at(c + 32 + (int32_t)lane);
                        int32_t his[4];  // adapters of rows c + lane / 4, + 8, ...
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            his[i] = __shfl_sync(0xffffffffu, who, 8 * i + (int)(lane >> 2));
                        who = coming;
                        __syncwarp();
                        tmem_load_fragments(taddr + c, v);
                        uint32_t hi[16], rest[16];
#pragma unroll
                        for (int k = 0; k < 4; ++k)  // row of the fragments: 8 k + lane / 4
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int at = 16 * (k >> 1) + 4 * i + 2 * (k & 1);
                                const float x = keep[k] ? v[at] * scale[k] : 0.0f;
                                const float y = keep[k] ? v[at + 1] * scale[k] : 0.0f;
                                hi[4 * i + k] = pack16(x, y, p.bf16);
                                rest[4 * i + k] = rest16x2(x, y, hi[4 * i + k], p.bf16);
                            }
#pragma unroll
                        for (int part = 0; part < 2; ++part) {
                            __syncwarp();
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t* q = (part ? rest : hi) + 4 * i;
                                st_matrix_trans(turn_st + (uint32_t)i * 8u * kTurnPitch, q[0], q[1], q[2], q[3]);
                            }
                            __syncwarp();
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (real && his[i] == id)
                                    *reinterpret_cast<uint4*>(
                                        p.low_out + (int64_t)(it.row0 + c + 8 * i + (int32_t)(lane >> 2)) * 2 * p.rank_pad +
                                        part * p.rank_pad + j) = ld_shared_v4(turn_ld + (uint32_t)i * 8u * kTurnPitch);
                        }
                    }
                    release();
                    return true;
                }
            }
            if (!ready()) return false;
            if (clustered) {
                // this CTA's share, fp32, into its ring (idle by now): rows of
                // Y x 128 columns; the cluster adds them up below
                for (int32_t c = chunk0; c < it.w; c += kChunkStep) {
                    __syncwarp();
                    tmem_load_32cols(taddr + c, v);
                    if (kAdapters && any_sick)
#pragma unroll 1
                        for (int j = 0; j < 32; ++j) add_at(v, j, sick_part(it.row0 + c + j, it.n * 128 + (int32_t)lane_row));
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (c + j < it.w) st_shared_f32(ring + (uint32_t)((c + j) * 128 + (int32_t)lane_row) * 4u, v[j]);
                }
                release();
                return true;
            }
            // this thread's 8 columns of Y (of rows lane / 4, + 8, ...)
            const int32_t n = it.n * (kPair ? 256 : 128) + 128 * (int32_t)rank + 32 * (int32_t)quarter + 8 * (int32_t)(lane & 3u);
            const bool in_n = n < p.N;
            for (int32_t c = chunk0; c < it.w; c += kChunkStep) {
                uint4 gate[4];
                if (p.act) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int32_t r = c + 8 * i + (int32_t)(lane >> 2);
                        if (in_n && r < it.valid)
                            gate[i] = __ldcg(reinterpret_cast<const uint4*>(
                                p.act + (int64_t)(it.row0 + r) * p.ld_act + n));
                    }
                }
                __syncwarp();  // (also: the last chunk's shared-memory reads are done)
                tmem_load_fragments(taddr + c, v);
                if (kAdapters && any_sick)
#pragma unroll 1
                    for (int j = 0; j < 32; ++j)
                        add_at(v, j, sick_part(it.row0 + c + 8 * ((j >> 2) & 3) + 2 * (int32_t)(lane & 3u) + (j & 1),
                                               n - 8 * (int32_t)(lane & 3u) + 16 * (j >> 4) + 8 * ((j >> 1) & 1) +
                                                   (int32_t)(lane >> 2)));
                if (p.apply_relu) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = v[j] > 0.0f ? v[j] : 0.0f;  // -0 and NaN become +0
                }
                // transposed through shared memory: 32 rows of Y x this
                // warp's 32 columns, 64 bytes at a pitch of 80
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    st_matrix_trans(turn_st + (uint32_t)i * 8u * kTurnPitch,
                                    pack16(v[4 * i], v[4 * i + 1], p.bf16), pack16(v[4 * i + 2], v[4 * i + 3], p.bf16),
                                    pack16(v[16 + 4 * i], v[17 + 4 * i], p.bf16),
                                    pack16(v[18 + 4 * i], v[19 + 4 * i], p.bf16));
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int32_t r = c + 8 * i + (int32_t)(lane >> 2);
                    uint4 q = ld_shared_v4(turn_ld + (uint32_t)i * 8u * kTurnPitch);
                    if (in_n && r < it.valid) {
                        if (p.act) {
                            q.x = gate16(q.x, gate[i].x, p.bf16);
                            q.y = gate16(q.y, gate[i].y, p.bf16);
                            q.z = gate16(q.z, gate[i].z, p.bf16);
                            q.w = gate16(q.w, gate[i].w, p.bf16);
                        }
                        *reinterpret_cast<uint4*>(p.Y + (int64_t)(it.row0 + r) * p.ldy + n) = q;
                    }
                }
            }
            release();
            return true;
        };
        for (bool ok = true; ok && iter.next(it); ++local) {
            if (kAdapters && !half) {
                if (!kPair) ask_for_boxes();
                ok = fill_extras();
            }
            // with helping warps these fill the next item's extra k-blocks while
            // those drain this one
            if (ok && (!helpers || half)) ok = drain(it, local);
            if (kAdapters && half) {
                __threadfence_block();
                __syncwarp();
                if (lane == 0) atomicAdd(&ctrl->helped, 1);
            } else if (kAdapters && any_sick) {
                // (all have drained it)
                if (helpers) ok = ok && wait_counter(&ctrl->helped, 4 * ((int32_t)local + 1), ctrl, p);
                ok = named_bar_and(kEpiBarrier, kEpi, ok);
                for (int32_t i = (int32_t)et; i < kMaxBoxes / 32; i += (int32_t)kEpi) ctrl->sick[i] = 0u;
                if (et == 0) ctrl->sick_item = 0;
                any_sick = false;
            }
        }
        // rows of no group: before the first group and past the last one
        const int32_t head = start[0], tail = start[p.G];
        const int32_t outside = head + (p.T - tail);
        const int32_t vecs = p.N / 8;  // 16-byte vectors of an output row
        for (int32_t r = (int32_t)blockIdx.x; r < outside; r += (int32_t)gridDim.x) {
            const int32_t t = r < head ? r : tail + (r - head);
            uint4* y = reinterpret_cast<uint4*>(p.Y + (int64_t)t * p.ldy);
            for (int32_t i = (int32_t)et; i < vecs; i += (int32_t)kEpi) y[i] = make_uint4(0, 0, 0, 0);
        }
    }

    if (clustered) {
        // every CTA of the cluster adds its part of the rows up, the shares
        // in their order, and writes them: 16 threads per row
        __syncwarp();
        cluster_sync();
        It again(p, start, tiles, nslots, lows, worker, workers, max_extra, 0);
        if (again.next(it) && warp >= 2 && warp <= 5) {
            const uint32_t c = (uint32_t)p.cluster;
            const int32_t r1 = min(it.valid, (int32_t)((share + 1) * (uint32_t)it.w / c));
            const uint32_t col = ((threadIdx.x - 64) & 15u) * 8u;
            const int32_t n = it.n * 128 + (int32_t)col;
            if (n < p.N) {
                for (int32_t r = (int32_t)(share * (uint32_t)it.w / c + ((threadIdx.x - 64) >> 4)); r < r1; r += 8) {
                    float x[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = 0.0f;
                    for (uint32_t q = 0; q < c; ++q) {
                        const uint32_t from = mapa_shared(ring + ((uint32_t)r * 128u + col) * 4u, q);
                        const float4 a = ld_shared_cluster_f4(from), b = ld_shared_cluster_f4(from + 16u);
                        x[0] += a.x;
                        x[1] += a.y;
                        x[2] += a.z;
                        x[3] += a.w;
                        x[4] += b.x;
                        x[5] += b.y;
                        x[6] += b.z;
                        x[7] += b.w;
                    }
                    if (p.apply_relu) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] = x[j] > 0.0f ? x[j] : 0.0f;
                    }
                    uint4 q = make_uint4(pack16(x[0], x[1], p.bf16), pack16(x[2], x[3], p.bf16),
                                         pack16(x[4], x[5], p.bf16), pack16(x[6], x[7], p.bf16));
                    if (p.act) {
                        const uint4 gate = __ldcg(
                            reinterpret_cast<const uint4*>(p.act + (int64_t)(it.row0 + r) * p.ld_act + n));
                        q.x = gate16(q.x, gate.x, p.bf16);
                        q.y = gate16(q.y, gate.y, p.bf16);
                        q.z = gate16(q.z, gate.z, p.bf16);
                        q.w = gate16(q.w, gate.w, p.bf16);
                    }
                    *reinterpret_cast<uint4*>(p.Y + (int64_t)(it.row0 + r) * p.ldy + n) = q;
                }
            }
        }
    }
    // (a later kernel's wait covers this one only: it must not end first)
    if (kAdapters && !lows_only) grid_dependency_wait();
    __syncthreads();
    if (threadIdx.x == 0 && *(volatile int32_t*)&ctrl->abort_flag) drain_ring(ctrl, full0, S);
    tc_fence_before();
    if (kPair || clustered)
        cluster_sync_relaxed();  // the other CTAs' accesses to this one's shared memory are done
    else
        __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<kCG>(tmem_base, p.tmem_cols);
    }
}

}  // namespace rg
}  // namespace gr
