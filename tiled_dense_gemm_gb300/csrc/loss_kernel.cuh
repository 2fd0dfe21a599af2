// The products behind the losses over a vocabulary, for sm_103a.  With z[t, v]
// = sum_d X[t, d] W[v, d] the logits of T rows over V words, c = log2(e) / tau,
// and the wanted words of a row (a target of weight 1, or a teacher's best
// words with weights q):
//
//   kStats   per row and tile: m = max z, s = sum 2^(c (z - m)),
//            t = sum of q z over the wanted words among them        (no z is kept)
//   kGrad    G[t, v] = a_t (2^(c (z - tau lse_t)) - sum of q of the wanted word v)
//            over a piece of the vocabulary, rounded to the 16-bit type; kGradLow, up to
//            32 rows: in two parts, the rounded value and the rounded rest
//   kSum     dX += G W over the piece, in 32 bits, split along the piece
//   kWeight  dW[piece] = G^T X
//
// One kernel, five epilogues: D = A B^T in tiles of 128 rows x `width` columns
// per CTA, or 256 x `width` per CTA pair, over k-blocks of 64 or 128.  An operand's
// reduction index is contiguous ("k-major": boxes of 64 k x rows) or its rows'
// index is ("mn-major": chunks of 64 rows x the k-block), as the matrices are
// stored; nothing is transposed in memory.  Rows of X are A's rows in kStats, kGrad
// and kSum, so that a row's logits sit in one lane of tensor memory: the running
// maximum and sum of the softmax never leave a thread.
//
// The rows in use (those with a wanted word) may have been gathered to the
// front of a copy of X; only the device knows how many there are.  The row
// tiles, the reduction of kWeight and the choice between X and its copy go by
// that count.
//
// Roles (352 threads, one CTA per SM): warp 0 copies A's tiles and arms the
// stages, warp 6 B's, warp 1 issues the MMAs, warps 2-5 and 7-10 drain the two
// accumulators (a quarter of the rows each, every other chunk of 64 columns).
// Every wait is bounded.
//
// What bounds it, and what it measured (the GPU's time alone, in a CUDA graph
// whose inputs rotate beyond L2):
//   up to 128 rows: the weights' way from memory.  64 rows, 131072 words of 4096:
//     158-162 us, 6.6-6.8 TB/s of weights; 16 rows, 65536 of 2048: 45 us; one row, 32000
//     of 1024: 16.1 us, of which 6.4 are left with next to no words.  (Boxes of 256
//     k: 5-15% slower; tiles of 64 to 112 words 5-60%.)  The gradients pass the
//     weights three times (G, dX, dW): 16 rows, 65536 of 2048: 137 us, 5.9 TB/s of
//     those; 128 rows, 131072 of 4096: 525 us, 6.1 TB/s.
//   many rows, alone: bytes from L2 into the multiprocessors, 12.7-15.6 TB/s in
//     every product (a pair takes in 64 KB per 512 clocks of the tensor core, which
//     at 1.8 GHz would be 17.5 TB/s): the tensor pipe is active 65-87% of the time.
//   many rows, back to back: the power cap.  8192 rows, 131072 words of 4096: 5.1-
//     5.3 ms, 1660-1730 TFLOP/s at 1.5 GHz, what the library product sustains; the
//     gradients of 4096 rows 7.8-8.3 ms.
//   rows whose pitch is not a multiple of 128 bytes cost a second line per box
//     row: 50021 words of 2056, 1800 of 3000 rows in use, 266-290 us.
#pragma once

#include "ragged_kernel.cuh"

namespace gr {
namespace ls {

using rg::Ctrl;
using rg::pack16;
using rg::wait_phase;

enum Mode : int { kStats = 0, kGrad = 1, kSum = 2, kWeight = 3, kGradLow = 4 };  // (kGradLow: G in two parts)

constexpr int kThreads = 352;
constexpr uint32_t kStaging = 4096;  // bytes per epilogue warp
constexpr int32_t kRowPad = 128;     // rows in use, and G's, end in zeros up to a multiple of this
constexpr int32_t kNone = 0x7fffffff;
constexpr int32_t kAhead = 8;        // k-blocks of B asked for in L2 ahead of a launch's turn

// What the device knows of the rows.
struct RowsHeader {
    int32_t valid;    // rows in use
    int32_t compact;  // 1: they are gathered in the copy of X
    float scale;      // of G, and its inverse: brings the largest |a_t| to the top of a binade
    float unscale;
};

struct LossMaps {
    CUtensorMap a[2], b[2];  // (the second: where the rows are gathered)
    CUtensorMap edge[2];     // of an mn-major operand, chunk by chunk, where its rows' end cuts through one
    CUtensorMap d, low;      // (low: of G's second part)
};

// dX from its sums.
struct FinishParams {
    const float* sums;       // [splits][rows][D]
    int32_t splits, T, D, bf16;
    int32_t rows_of, low;    // rows of a plane; > 0: those from here on are added to the first
    const RowsHeader* rows;
    const int32_t* index;    // null: all rows in their places,
    const int32_t* flags;    // ... in use where in [0, limit)
    int32_t limit;
    uint16_t* dX;
    int64_t ld_dx;
};

// What the logit of a single word is summed from, by so many threads.
struct WordSums {
    const uint16_t* X;
    int64_t ldx;
    const uint16_t* W;
    int64_t w_word, w_depth;  // from one word to the next, and from one k: one of them 1
    const int32_t* targets;   // a row's word, or
    const int32_t* ids;       // a teacher's (T, k), sorted, with weights: its main word
    const float* weights;
    int32_t k, D, bf16;
};
constexpr int32_t kSumThreads = 256;

struct LossParams {
    int32_t M, N, K;       // D is M x N, K the reduction (bounds, where the rows' count replaces them)
    int32_t rows_m;        // M is the rows' count
    int32_t rows_k;        // K is the rows' count
    int32_t width;         // columns of a tile
    int32_t bk;            // k per ring stage: 64 or 128
    int32_t n_tiles;
    int32_t group_m;       // row tiles walked together
    int32_t splits;        // kSum: shares of the reduction, each summed apart
    int32_t a_mn, b_mn;    // operand is mn-major
    int32_t a_3d, b_3d;    // a stage's boxes or chunks come in one copy
    int32_t a_blocks, b_blocks;  // ... up to this many chunks of the operand, beyond through `edge`
    uint32_t a_bytes;      // of a stage (the box's)
    uint32_t stage_bytes;
    int32_t num_stages;
    // This launch goes by its predecessor's wait: it reads nothing of what that
    // one writes, and that one lets it start only once it has itself waited for all
    // before.  It waits for its predecessor before it ends, so that its end says
    // that all before it is done.
    int32_t late;
    // kGrad: only the epilogue waits for the predecessor, which lets this launch start
    // once it has itself waited for all before: the rest reads nothing of what that
    // one writes (100 rows with a teacher, 32768 words of 1024: 76 us without, 71 with;
    // kStats is better started before that one's wait, with its first words on their
    // way into L2: 16 rows, 32000 of 1024, 20.4 and 21.7).
    int32_t early;
    int32_t once;          // the weights' lines (B; kWeight: its output's) leave L2 first
    uint32_t tmem_cols;    // allocated; half per accumulator
    int32_t bf16;
    int32_t w_row, w_k;    // first word of the piece, added to B's row or to its k
    int32_t d_row, d_col;  // ... or to the output's row or column
    int32_t first;         // kSum: 1: set, 0: add
    const RowsHeader* rows;  // the rows' count; null: all rows, as given
    const RowsHeader* scale;  // kGrad: null: to be found from `top` (up to 128 rows)
    float top;
    const int32_t* flags;    // kGrad, rows null: a row is in use if its flag is in [0, limit)
    int32_t limit;
    const int32_t* index;    // row of the batch of each gathered row
    // the wanted words: a target per row, or (ids != null) k sorted ones with weights
    const int32_t* targets;
    const int32_t* ids;
    const float* weights;
    int32_t k, V;
    float log2_scale;        // c
    float* stats;            // kStats: [tile][3][stats_pitch]
    int64_t stats_pitch;
    WordSums sums;
    int32_t shares;          // kStats, up to 128 rows: so many shares of each row's
    double* exact;           // ... main word's logit,
    float* main_weight;      // ... and that word's weight
    const float* lse;        // kGrad
    const float* dloss;
    int64_t dloss_stride;    // 0 or 1
    float grad_scale;        // tau
    uint16_t* grad;          // G, for tiles that end inside a chunk
    int64_t grad_pitch;
    int32_t low;             // > 0: G's rows from here on take what rounding left of the first
    FinishParams finish;     // kWeight: dX != null: to be done at the end
    int32_t* err;
    uint64_t timeout_ns;
    int32_t test_drop_kb;    // as of the ragged kernels: a block of A's rows (single CTAs)
};

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// (a - b) c for two a at once (one at a time 4096 rows with a teacher, 65536 words of
// 2048, took 650 us, 640 so; 8192 rows, 131072 of 4096, 5107 and 5070).
struct Shifted {
    uint64_t b, c;
    __device__ __forceinline__ Shifted(float by, float scale) {
        asm("mov.b64 %0, {%1, %1};" : "=l"(b) : "f"(-by));
        asm("mov.b64 %0, {%1, %1};" : "=l"(c) : "f"(scale));
    }
    __device__ __forceinline__ void operator()(float& x, float& y) const {
        asm("{\n\t.reg .b64 t;\n\tmov.b64 t, {%0, %1};\n\tadd.rn.f32x2 t, t, %2;\n\tmul.rn.f32x2 t, t, %3;\n\tmov.b64 {%0, %1}, t;\n\t}"
            : "+f"(x), "+f"(y)
            : "l"(b), "l"(c));
    }
};

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
    return x;
}

// The largest |dloss| of the rows in use, by one warp (few rows).
__device__ __forceinline__ float largest_dloss(const int32_t* flags, int32_t limit, const float* dloss, int64_t stride, int32_t T) {
    float top = 0.0f;
    for (int32_t t = (int32_t)threadIdx.x % 32; t < T; t += 32) {
        const int32_t y = __ldcg(flags + t);
        const float d = dloss[(int64_t)t * stride];
        if (y >= 0 && y < limit) top = fmaxf(top, fabsf(d));
    }
    return warp_max(top);
}

// The scale of G that brings the largest |dloss grad_scale| to `top`.
__device__ __forceinline__ float scale_of(float top, float grad_scale, float largest) {
    largest *= grad_scale;
    return largest > 1e-30f && largest < 1e30f ? top / largest : 1.0f;
}

__device__ __forceinline__ void st_shared_u16(uint32_t addr, uint16_t x) {
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(x) : "memory");
}

// Tensor copies global -> shared with an L2 policy; of a pair's, `bar` is the leader's.
template <bool kPair>
__device__ __forceinline__ void load_2d_hint(uint32_t dst, const CUtensorMap* m, uint32_t bar, int32_t x, int32_t y,
                                             uint64_t policy) {
    if constexpr (kPair)
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
            " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y),
            "l"(policy)
            : "memory");
    else
        tma_load_2d_hint(dst, m, bar, x, y, policy);
}

template <bool kPair>
__device__ __forceinline__ void load_3d_hint(uint32_t dst, const CUtensorMap* m, uint32_t bar, int32_t x, int32_t y,
                                             int32_t z, uint64_t policy) {
    if constexpr (kPair)
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
            " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x),
            "r"(y), "r"(z), "l"(policy)
            : "memory");
    else
        rg::load_3d_hint(dst, m, bar, x, y, z, policy);
}

__device__ __forceinline__ void store_2d_hint(const CUtensorMap* m, uint32_t src, int32_t x, int32_t y, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group.L2::cache_hint [%0, {%2, %3}], [%1], %4;" ::"l"(
            reinterpret_cast<uint64_t>(m)),
        "r"(src), "r"(x), "r"(y), "l"(policy)
        : "memory");
}

// 64 numbers of 32 bits per lane into tensor memory.
__device__ __forceinline__ void tmem_store_64cols(uint32_t taddr, const float (&v)[64]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x64.b32 [%0],"
        " {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16,"
        " %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32,"
        " %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48,"
        " %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63, %64};\n\t"
        "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
        "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
        "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
        "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])), "r"(__float_as_uint(v[8])),
        "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
        "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])),
        "r"(__float_as_uint(v[15])), "r"(__float_as_uint(v[16])), "r"(__float_as_uint(v[17])),
        "r"(__float_as_uint(v[18])), "r"(__float_as_uint(v[19])), "r"(__float_as_uint(v[20])),
        "r"(__float_as_uint(v[21])), "r"(__float_as_uint(v[22])), "r"(__float_as_uint(v[23])),
        "r"(__float_as_uint(v[24])), "r"(__float_as_uint(v[25])), "r"(__float_as_uint(v[26])),
        "r"(__float_as_uint(v[27])), "r"(__float_as_uint(v[28])), "r"(__float_as_uint(v[29])),
        "r"(__float_as_uint(v[30])), "r"(__float_as_uint(v[31])), "r"(__float_as_uint(v[32])),
        "r"(__float_as_uint(v[33])), "r"(__float_as_uint(v[34])), "r"(__float_as_uint(v[35])),
        "r"(__float_as_uint(v[36])), "r"(__float_as_uint(v[37])), "r"(__float_as_uint(v[38])),
        "r"(__float_as_uint(v[39])), "r"(__float_as_uint(v[40])), "r"(__float_as_uint(v[41])),
        "r"(__float_as_uint(v[42])), "r"(__float_as_uint(v[43])), "r"(__float_as_uint(v[44])),
        "r"(__float_as_uint(v[45])), "r"(__float_as_uint(v[46])), "r"(__float_as_uint(v[47])),
        "r"(__float_as_uint(v[48])), "r"(__float_as_uint(v[49])), "r"(__float_as_uint(v[50])),
        "r"(__float_as_uint(v[51])), "r"(__float_as_uint(v[52])), "r"(__float_as_uint(v[53])),
        "r"(__float_as_uint(v[54])), "r"(__float_as_uint(v[55])), "r"(__float_as_uint(v[56])),
        "r"(__float_as_uint(v[57])), "r"(__float_as_uint(v[58])), "r"(__float_as_uint(v[59])),
        "r"(__float_as_uint(v[60])), "r"(__float_as_uint(v[61])), "r"(__float_as_uint(v[62])),
        "r"(__float_as_uint(v[63]))
        : "memory");
}

// 3-D tiled add shared -> global (bulk-group completion).
__device__ __forceinline__ void reduce_add_3d(const CUtensorMap* m, uint32_t src, int32_t x, int32_t y, int32_t z) {
    asm volatile(
        "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
            reinterpret_cast<uint64_t>(m)),
        "r"(src), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// A row's wanted words in rising order, from the first at or behind some column.
// Frequent words come close together, so the word after the next one is on its
// way while that is dealt with, and they are read through L1: the first tiles hold
// tens of a row's words, one after another (100 rows, 64 words each, 32768 words of
// 1024: 34 us from L2, 29 so, the gradients 70 and 61; 4096 rows of 65536 of 2048:
// 645 and 632).
struct Wanted {
    int32_t row, at;  // row of the lists, place of the word after `next2` in it
    int32_t next;     // word, kNone: no more
    float weight;     // its
    int32_t next2;
    float weight2;

    // `y`: the row's target where there is no teacher
    __device__ __forceinline__ void start(const LossParams& q, int32_t t, int32_t y, bool live, int32_t col) {
        row = t;
        at = q.k;
        next = next2 = kNone;
        weight = weight2 = 1.0f;
        if (!live) return;
        if (!q.ids) {
            if (y >= col && y < q.V) next = y;
            return;
        }
        const int32_t* const ids = q.ids + (int64_t)row * q.k;
        int32_t lo = 0, hi = q.k;
        while (lo < hi) {
            const int32_t mid = (lo + hi) >> 1;
            if (ids[mid] < col)
                lo = mid + 1;
            else
                hi = mid;
        }
        at = lo;
        fetch(q, next, weight);
        fetch(q, next2, weight2);
    }

    __device__ __forceinline__ void fetch(const LossParams& q, int32_t& id, float& w) {
        id = kNone;
        if (at < q.k) {
            const int64_t i = (int64_t)row * q.k + at;
            id = q.ids[i];
            w = q.weights[i];
            ++at;
        }
    }

    __device__ __forceinline__ void advance(const LossParams& q) {
        next = next2;
        weight = weight2;
        fetch(q, next2, weight2);
    }
};

// A row's main word, the wanted one that weighs most, and its weight, by one warp.  A
// word that comes several times weighs as all of its entries: the sorted list goes
// by in 32 entries at once, each with the sum of its word's entries so far, whose
// maximum is that of the whole sums.
__device__ __forceinline__ int32_t main_word(const WordSums& p, int32_t t, float& weight) {
    weight = 1.0f;
    if (!p.ids) return __ldcg(p.targets + t);
    const int32_t lane = (int32_t)threadIdx.x % 32;
    const int32_t* const ids = p.ids + (int64_t)t * p.k;
    const float* const weights = p.weights + (int64_t)t * p.k;
    float most = 0.0f, carry = 0.0f;
    int32_t word = kNone, before = kNone;  // (carry: the last word's sum before this entry)
#pragma unroll 2
    for (int32_t j0 = 0; j0 < p.k; j0 += 32) {
        const int32_t id = j0 + lane < p.k ? __ldcg(ids + j0 + lane) : kNone;
        float all = j0 + lane < p.k ? __ldcg(weights + j0 + lane) : 0.0f;
        if (lane == 0 && id == before) all += carry;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const float x = __shfl_up_sync(0xffffffffu, all, d);
            const int32_t y = __shfl_up_sync(0xffffffffu, id, d);
            if (lane >= d && y == id) all += x;
        }
        carry = __shfl_sync(0xffffffffu, all, 31);
        before = __shfl_sync(0xffffffffu, id, 31);
        if (id != kNone && all > most) {  // (of equal ones the first, which is the lowest)
            most = all;
            word = id;
        }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const float x = __shfl_xor_sync(0xffffffffu, most, d);
        const int32_t y = __shfl_xor_sync(0xffffffffu, word, d);
        if (x > most || (x == most && y < word)) {
            most = x;
            word = y;
        }
    }
    weight = most;
    return word;
}

// Eight of the products of X's row with a word's weights, from k = d on (D is a
// multiple of 8); each is exact in 32 bits.
__device__ __forceinline__ void products_8(const WordSums& p, const uint16_t* x, const uint16_t* w, int32_t d, float (&o)[8]) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(x + d));
    uint4 b;
    if (p.w_depth == 1) {
        b = __ldg(reinterpret_cast<const uint4*>(w + d));
    } else {
        uint32_t e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = __ldg(w + (int64_t)(d + j) * p.w_depth);
        b = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
    }
    const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 m = rg::unpack16(av[j], p.bf16), n = rg::unpack16(bv[j], p.bf16);
        o[2 * j] = m.x * n.x;
        o[2 * j + 1] = m.y * n.y;
    }
}

// A sum in two numbers of 32 bits, the second what rounding left of the first (Knuth's
// exact sum of two): as exact as 64 bits here, whose additions take the GPU 64 clocks a
// warp.
struct Wide {
    float hi, lo;

    __device__ __forceinline__ void add(float b) {
        const float s = __fadd_rn(hi, b), t = __fsub_rn(s, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, t)), __fsub_rn(b, t)));
        hi = s;
    }
    __device__ __forceinline__ void add_lane(int d) {  // another lane's
        const float h = __shfl_xor_sync(0xffffffffu, hi, d), l = __shfl_xor_sync(0xffffffffu, lo, d);
        add(h);
        lo = __fadd_rn(lo, l);
    }
};

// Eight products more.
__device__ __forceinline__ void add_8(Wide (&z)[2], const float (&o)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j & 1].add(o[j]);
}

// Thread i's of kSumThreads' products of that logit.
__device__ __forceinline__ double some_products(const WordSums& p, int32_t t, int32_t word, int32_t i) {
    const uint16_t *const x = p.X + (int64_t)t * p.ldx, *const w = p.W + (int64_t)word * p.w_word;
    Wide z[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
    for (int32_t d = 8 * i; d < p.D; d += 8 * kSumThreads) {
        float o[8];
        products_8(p, x, w, d, o);
        add_8(z, o);
    }
    z[0].add(z[1].hi);
    return (double)z[0].hi + (double)__fadd_rn(z[0].lo, z[1].lo);
}

// One of `shares` shares of that logit by one warp.
__device__ __forceinline__ Wide exact_share(const WordSums& p, int32_t t, int32_t word, int32_t share, int32_t shares) {
    const uint16_t *const x = p.X + (int64_t)t * p.ldx, *const w = p.W + (int64_t)word * p.w_word;
    const int64_t vecs = p.D / 8;
    const int32_t end = 8 * (int32_t)((share + 1) * vecs / shares);
    Wide z[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
#pragma unroll 2
    for (int32_t d = 8 * ((int32_t)(share * vecs / shares) + (int32_t)threadIdx.x % 32); d < end; d += 256) {
        float o[8];
        products_8(p, x, w, d, o);
        add_8(z, o);
    }
    z[0].add(z[1].hi);
    z[0].lo = __fadd_rn(z[0].lo, z[1].lo);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) z[0].add_lane(d);
    return z[0];
}

// v[at], halving.
template <int kFrom, int kCount, int kSize>
__device__ __forceinline__ float pick(const float (&v)[kSize], int32_t at) {
    if constexpr (kCount == 1) {
        return v[kFrom];
    } else {
        const float low = pick<kFrom, kCount / 2>(v, at), high = pick<kFrom + kCount / 2, kCount / 2>(v, at);
        return at & (kCount / 2) ? high : low;
    }
}

// The logits' reduction in parts of at most this many k, each in an accumulator of
// its own, added up in registers.  The tensor core truncates its sums in 32 bits, 16
// products at a time, always towards zero: over 4096 that was 2.4e-6 of the losses
// (6e-7 for a sum that rounds).  Pairs: 5.4e-7 in parts of 1024, which cost
// nothing; parts of 512 3e-7, at 4096 rows, 65536 words of 2048 682 us for 645.
// Single CTAs, which wait for memory: 1.3e-7 in parts of 256 (64 rows, 131072 words
// of 4096: 162.1 -> 163.5 us), 9e-8 in parts of 128 (169.4).
//
// The gradients take the pairs' parts.  So beyond 128 rows what truncation leaves is the
// same in z and in the forward pass's lse, and drops out of their difference: at 1 - p =
// 1e-6 and z = 27, binary16, p - 1 is off by 1e-6, the rounding of lse; by 1.7e-4 from
// an exact lse.  Up to 128 rows words of p > 1/2 are summed exactly in both passes, and
// the other words' p is off by 1.7e-4 of itself at most there; parts of 256, as the
// forward pass's, cost 100 rows with a teacher, 32768 words of 1024, 69 -> 74 us (the
// product stops two parts ahead of the epilogue, which waits for the teacher).
constexpr int32_t kPartLogits = 1024, kPartFew = 256;
// dX's and dW's sums, whose terms may all have one sign: in one accumulator they lost
// 1.07% over 2^20 rows and 0.08% over 94000 words; in parts of 4096 4e-5, a tenth of
// binary16's rounding.
constexpr int32_t kPartSum = 4096;

// In steps of 128 k, whatever a stage holds.  kMany: there may be several.
template <bool kPair, int kMode, bool kMany>
struct Parts {
    static constexpr bool kLogits = kMode == kStats || kMode == kGrad || kMode == kGradLow;
    static constexpr int32_t kPart = !kMany ? 1 << 30 : !kLogits ? kPartSum : kMode == kStats && !kPair ? kPartFew : kPartLogits;
    int32_t first, last, steps, count, two;

    // blocks [kb0, kb1) of `bk` k
    __device__ __forceinline__ Parts(int32_t kb0, int32_t kb1, int32_t bk) : first(kb0), last(kb1), two(bk == 64 ? 1 : 0) {
        steps = (kb1 - kb0 + two) >> two;
        count = (steps + kPart / 128 - 1) / (kPart / 128);
    }
    // one behind the last block of part `part` - 1
    __device__ __forceinline__ int32_t end(int32_t part) const {
        return min(last, first + ((int32_t)((int64_t)part * steps / count) << two));
    }
};

// Division by a number that many items share.
struct Divider {
    uint32_t d, inverse;

    __device__ __forceinline__ explicit Divider(uint32_t by) : d(by), inverse(0xffffffffu / by) {}

    __device__ __forceinline__ uint32_t operator()(uint32_t x, uint32_t& rest) const {
        uint32_t q = __umulhi(x, inverse);  // at most one too small, for x below 2^31
        rest = x - q * d;
        if (rest >= d) {
            ++q;
            rest -= d;
        }
        return q;
    }
};

// 64 numbers times a factor, rounded to the 16-bit type.
__device__ __forceinline__ void pack_64(uint32_t (&x)[32], const float (&v)[64], float u, int32_t bf16) {
    if (bf16) {
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = pack16(u * v[2 * j], u * v[2 * j + 1], 1);
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = pack16(u * v[2 * j], u * v[2 * j + 1], 0);
    }
}

// What that rounding left of them, rounded.
__device__ __forceinline__ void rest_64(uint32_t (&x)[32], const float (&v)[64], int32_t bf16) {
    if (bf16) {
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = rg::rest16x2(v[2 * j], v[2 * j + 1], x[j], 1);
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = rg::rest16x2(v[2 * j], v[2 * j + 1], x[j], 0);
    }
}

// Two parts of a row's statistics as one.
__device__ __forceinline__ void merge_stats(float& m, float& s, float m1, float s1, float c) {
    const float top = fmaxf(m, m1);
    const float ref = fabsf(top) == INFINITY ? 0.0f : top;
    // (a sum taken at an infinite maximum is itself infinite or zero and needs no other reference)
    const float f0 = fabsf(m) == INFINITY ? 1.0f : exp2_fast((m - ref) * c);
    const float f1 = fabsf(m1) == INFINITY ? 1.0f : exp2_fast((m1 - ref) * c);
    s = s * f0 + s1 * f1;
    m = top;
}

// dX[row] from its shares, rounded once; +0 in the rows that are not in use.
// kLanes threads per eight columns take the shares in turn and are added up in a
// fixed order.  By all blocks of a launch, `threads` each.
template <int kLanes>
__device__ __forceinline__ void finish_lanes(const FinishParams& p, int32_t threads) {
    const int32_t valid = p.index ? __ldcg(&p.rows->valid) : p.T;
    const float u = __ldcg(&p.rows->unscale);
    const int32_t vecs = p.D / 8, lane = (int32_t)threadIdx.x % kLanes;
    const int64_t total = (int64_t)p.T * vecs, share = (int64_t)p.rows_of * p.D, low = (int64_t)p.low * p.D;
    const int64_t step = (int64_t)gridDim.x * (threads / kLanes), rounds = (total + step - 1) / step;
    int64_t i = (int64_t)blockIdx.x * (threads / kLanes) + threadIdx.x / kLanes;
    for (int64_t n = 0; n < rounds; ++n, i += step) {
        const int32_t r = i < total ? (int32_t)(i / vecs) : 0, c = (int32_t)(i - (int64_t)r * vecs);
        float4 a = make_float4(0, 0, 0, 0), b = a;
        if (i < total && r < valid) {
            const float4* const src = reinterpret_cast<const float4*>(p.sums + (int64_t)r * p.D) + 2 * c;
#pragma unroll 4
            for (int32_t k = lane; k < p.splits; k += kLanes) {
                const float4 x = __ldcs(src + k * (share / 4)), y = __ldcs(src + k * (share / 4) + 1);
                a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
                b.x += y.x, b.y += y.y, b.z += y.z, b.w += y.w;
                if (low) {
                    const float4 x2 = __ldcs(src + k * (share / 4) + low / 4), y2 = __ldcs(src + k * (share / 4) + low / 4 + 1);
                    a.x += x2.x, a.y += x2.y, a.z += x2.z, a.w += x2.w;
                    b.x += y2.x, b.y += y2.y, b.z += y2.z, b.w += y2.w;
                }
            }
        }
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) {
            a.x += __shfl_xor_sync(0xffffffffu, a.x, d), a.y += __shfl_xor_sync(0xffffffffu, a.y, d);
            a.z += __shfl_xor_sync(0xffffffffu, a.z, d), a.w += __shfl_xor_sync(0xffffffffu, a.w, d);
            b.x += __shfl_xor_sync(0xffffffffu, b.x, d), b.y += __shfl_xor_sync(0xffffffffu, b.y, d);
            b.z += __shfl_xor_sync(0xffffffffu, b.z, d), b.w += __shfl_xor_sync(0xffffffffu, b.w, d);
        }
        if (i < total && lane == 0) {
            uint4 o = make_uint4(0, 0, 0, 0);
            bool in = r < valid;
            if (!p.index) {
                const int32_t f = __ldcg(p.flags + r);
                in = f >= 0 && f < p.limit;
            }
            if (in)
                o = make_uint4(pack16(a.x * u, a.y * u, p.bf16), pack16(a.z * u, a.w * u, p.bf16),
                               pack16(b.x * u, b.y * u, p.bf16), pack16(b.z * u, b.w * u, p.bf16));
            reinterpret_cast<uint4*>(p.dX + (int64_t)(p.index ? __ldcg(p.index + r) : r) * p.ld_dx)[c] = o;
        }
    }
}

__device__ __forceinline__ void finish_dx(const FinishParams& p, int32_t threads) {
    if (p.splits >= 8)
        finish_lanes<4>(p, threads);
    else
        finish_lanes<1>(p, threads);
}

// kMany false: reductions of one part.  (The gradients with room for several parts in
// all three kernels: 64 rows, 65536 words of 2048, 140.4 us for 137.2, 300 rows, 32008 of
// 1000 by columns, 85.5 for 81.5.)
template <bool kPair, int kMode, bool kMany>
__global__ void __launch_bounds__(kThreads, 1)
    loss_kernel(const __grid_constant__ LossMaps maps, const __grid_constant__ LossParams q) {
    constexpr int kCG = kPair ? 2 : 1;
    constexpr int32_t kTileM = kPair ? 256 : 128;
    constexpr bool kLow = kMode == kGradLow, kAnyGrad = kMode == kGrad || kLow;
    extern __shared__ __align__(1024) uint8_t smem[];
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem);
    const uint32_t ring = (smem_u32(smem) + (uint32_t)sizeof(Ctrl) + 1023u) & ~1023u;
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = kPair ? cluster_ctarank() : 0u;
    const uint32_t worker = kPair ? blockIdx.x / 2 : blockIdx.x;
    const uint32_t workers = kPair ? gridDim.x / 2 : gridDim.x;
    rg::Params w;  // what wait_phase reads
    w.err = q.err;
    w.timeout_ns = q.timeout_ns;

    if (warp == 2 && lane == 0) {
        for (int s = 0; s < q.num_stages; ++s) {
            mbar_init(smem_u32(&ctrl->full[s]), 1);
            mbar_init(smem_u32(&ctrl->empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&ctrl->tmem_full[b]), 1);
            mbar_init(smem_u32(&ctrl->tmem_empty[b]), (kPair ? 2u : 1u) * 8u);
        }
        mbar_init(smem_u32(&ctrl->final_bar), 1);
        for (int b = 0; b < 8; ++b) {
            mbar_init(smem_u32(&ctrl->extra[b]), 1);
            mbar_init(smem_u32(&ctrl->peer[b]), 1);
        }
        ctrl->abort_flag = 0;
        ctrl->ring_s = ctrl->ring_ph = ctrl->ring_lap = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc<kCG>(smem_u32(&ctrl->tmem_addr), q.tmem_cols);
        tmem_relinquish<kCG>();
    }
    __syncwarp();
    tc_fence_before();
    if (kPair)
        cluster_sync();
    else
        cta_barrier_sync();
    tc_fence_after();
    if constexpr (!kPair && kMode != kWeight) {
        // Few rows: the weights' way from memory is all there is, so the first item's
        // are asked for in L2 before the kernel before is waited for (a line that it
        // still writes is current there): 1.4 us less for one row, 32000 words of 1024.
        if (warp == 6 && lane == 0) {
            const uint32_t split = worker / (uint32_t)q.n_tiles, nt = worker - split * (uint32_t)q.n_tiles;
            const int32_t blocks = (q.K + q.bk - 1) / q.bk;
            const int32_t r0 = (int32_t)nt * q.width + q.w_row, kb0 = (int32_t)((int64_t)split * blocks / q.splits);
            for (int32_t i = 0; i < kAhead && kb0 + i < blocks; ++i) {
                const int32_t k0 = (kb0 + i) * q.bk + q.w_k;
                if (q.b_3d) {
                    tma_prefetch_3d(&maps.b[0], 0, q.b_mn ? k0 : r0, (q.b_mn ? r0 : k0) / 64);
                } else {
                    for (int32_t j = 0; j < (q.b_mn ? q.width : q.bk) / 64; ++j)
                        tma_prefetch_2d(&maps.b[0], q.b_mn ? r0 + 64 * j : k0 + 64 * j, q.b_mn ? k0 : r0);
                }
            }
        }
        __syncwarp();
    }
    const Divider by_group((uint32_t)q.group_m * (uint32_t)q.n_tiles), by_rows((uint32_t)q.group_m);
    if (kMode == kStats) grid_launch_dependents();
    const bool early = kAnyGrad && q.early;
    if (!q.late && !early) grid_dependency_wait();
    if (kMode != kStats && !early) grid_launch_dependents();  // (behind the wait: what follows may go by it)
    const uint32_t tmem_base = ctrl->tmem_addr;
    const uint32_t S = (uint32_t)q.num_stages, stride = q.stage_bytes;
    const uint32_t full0 = smem_u32(&ctrl->full[0]), empty0 = smem_u32(&ctrl->empty[0]);
    const uint32_t buf_cols = q.tmem_cols / 2;
    const int32_t valid = q.rows ? __ldcg(&q.rows->valid) : 0;
    const int32_t gathered = q.rows ? __ldcg(&q.rows->compact) : 0;
    const int32_t M = q.rows_m && q.rows ? valid : q.M, K = q.rows_k ? valid : q.K;
    const int32_t m_tiles = (M + kTileM - 1) / kTileM, blocks = (K + q.bk - 1) / q.bk;
    const uint32_t tiles = (uint32_t)m_tiles * (uint32_t)q.n_tiles;
    const uint32_t items = tiles * (uint32_t)q.splits;

    // item -> share of the reduction, row tile, column tile
    struct Work {
        int32_t split, mt, nt, kb0, kb1;
    };
    // (three divisions per item cost 450 clocks in every role)
    uint32_t item = worker;
    const uint32_t whole = (uint32_t)m_tiles / (uint32_t)q.group_m;
    const Divider by_share(max(tiles, 1u)), by_last(max((uint32_t)m_tiles - whole * (uint32_t)q.group_m, 1u));
    auto next = [&](Work& k) {
        if (item >= items) return false;
        uint32_t l = item, r, m;
        k.split = 0;
        k.kb0 = 0;
        k.kb1 = blocks;
        if (q.splits > 1) {
            k.split = (int32_t)by_share(item, l);
            k.kb0 = (int32_t)((int64_t)k.split * blocks / q.splits);
            k.kb1 = (int32_t)((int64_t)(k.split + 1) * blocks / q.splits);
        }
        const uint32_t g = by_group(l, r);
        k.nt = (int32_t)(g < whole ? by_rows(r, m) : by_last(r, m));
        k.mt = (int32_t)(g * (uint32_t)q.group_m + m);
        item += workers;
        return true;
    };
    Work k;

    if (warp == 0 || warp == 6) {
        // warp 0 copies A's tiles and arms the stages, warp 6 B's
        if (lane == 0) {
            const bool is_a = warp == 0;
            const CUtensorMap* const maps_of = is_a ? &maps.a[gathered] : &maps.b[gathered];
            const int32_t width = q.width / kCG;
            uint32_t s = 0, ph = 0;
            int32_t issued = 0;
            bool ok = true;
            const bool once = kMode != kWeight && !is_a && q.once;
            const uint64_t policy = l2_policy_evict_first();
            const bool mn = is_a ? q.a_mn : q.b_mn, in_one = is_a ? q.a_3d : q.b_3d;
            // copies of a stage where it takes several, and the bytes of one: 64 k of
            // all rows, or 64 rows of all k
            const int32_t copies = mn ? (is_a ? 2 : width / 64) : q.bk / 64;
            const uint32_t piece = mn ? (uint32_t)q.bk * 128u : is_a ? q.a_bytes / (uint32_t)copies : (uint32_t)width * 128u;
            while (ok && next(k)) {
                const int32_t r0 = is_a ? k.mt * kTileM + 128 * (int32_t)rank : k.nt * q.width + width * (int32_t)rank + q.w_row;
                const bool inside = !mn || r0 / 64 + copies <= (is_a ? q.a_blocks : q.b_blocks);
                const bool one = in_one && inside;
                const CUtensorMap* const m = inside ? maps_of : &maps.edge[gathered];
                for (int32_t kb = k.kb0; kb < k.kb1; ++kb) {
                    if (!wait_phase(empty0 + 8u * s, ph ^ 1u, ctrl, w, is_a ? rg::kErrTokens : rg::kErrWeights)) {
                        ok = false;
                        break;
                    }
                    const uint32_t full = full0 + 8u * s;
                    if (is_a) {
                        if (!kPair || rank == 0) mbar_arrive_expect_tx(full, (kPair ? 2u : 1u) * stride);
                        ++issued;
                    }
                    const uint32_t bar = kPair ? mapa_shared(full, 0) : full;
                    const uint32_t dst = ring + s * stride + (is_a ? 0u : q.a_bytes);
                    const int32_t k0 = kb * q.bk + (is_a ? 0 : q.w_k);
                    if (!kPair && is_a && issued == q.test_drop_kb && q.test_drop_kb > 0) {
                        // (test hook: not copied)
                    } else if (one) {
                        if (once)
                            load_3d_hint<kPair>(dst, m, bar, 0, mn ? k0 : r0, (mn ? r0 : k0) / 64, policy);
                        else
                            rg::load_3d<kPair>(dst, m, bar, 0, mn ? k0 : r0, (mn ? r0 : k0) / 64);
                    } else {
                        for (int32_t j = 0; j < copies; ++j) {
                            const uint32_t to = dst + (uint32_t)j * piece;
                            const int32_t x = mn ? r0 + 64 * j : k0 + 64 * j, y = mn ? k0 : r0;
                            if (once)
                                load_2d_hint<kPair>(to, m, bar, x, y, policy);
                            else
                                rg::load_2d<kPair>(to, m, bar, x, y);
                        }
                    }
                    if (++s == S) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (is_a && (!kPair || rank == 0)) {
                ctrl->ring_s = (int32_t)s;
                ctrl->ring_ph = (int32_t)ph;
                ctrl->ring_lap = issued >= (int32_t)S ? 1 : 0;
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0 && (!kPair || rank == 0)) {
            const uint32_t tfull0 = smem_u32(&ctrl->tmem_full[0]), tempty0 = smem_u32(&ctrl->tmem_empty[0]);
            const uint32_t idesc = make_idesc_f16_f32((uint32_t)kTileM, (uint32_t)q.width, q.a_mn != 0, q.b_mn != 0, q.bf16 != 0);
            // k-major: 32 bytes per 16 k inside the swizzled rows, the next 64 k behind
            // all rows; mn-major: 16 rows of k, chunks of 64 rows apart by the k-block
            const uint32_t b_rows = (uint32_t)q.width / kCG;
            const uint64_t a_desc0 = make_sw128_desc(ring, q.a_mn ? (uint32_t)q.bk * 128u : 16u, 1024);
            const uint64_t b_desc0 = make_sw128_desc(ring + q.a_bytes, q.b_mn ? (uint32_t)q.bk * 128u : 16u, 1024);
            const uint64_t a_step = q.a_mn ? 128u : 2u, b_step = q.b_mn ? 128u : 2u;
            const uint64_t a_next = q.a_mn ? 512u : (q.a_bytes / 2) >> 4, b_next = q.b_mn ? 512u : (b_rows * 128u) >> 4;
            const bool two = q.bk == 128;
            uint32_t s = 0, ph = 0, local = 0;
            bool ok = true;
            while (ok && next(k)) {
                const Parts<kPair, kMode, kMany> parts(k.kb0, k.kb1, q.bk);
                int32_t kb = k.kb0;
                for (int32_t part = 1; ok && part <= parts.count; ++part) {
                    const int32_t begin = kb, end = parts.end(part);
                    const uint32_t buf = local & 1u, bph = (local >> 1) & 1u;
                    if (!wait_phase(tempty0 + 8u * buf, bph ^ 1u, ctrl, w, rg::kErrAccum)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem_base + buf * buf_cols;
                    for (; kb < end; ++kb) {
                        if (!wait_phase(full0 + 8u * s, ph, ctrl, w, rg::kErrStage)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t a_desc = a_desc0 + (uint64_t)(s * (stride >> 4));
                        const uint64_t b_desc = b_desc0 + (uint64_t)(s * (stride >> 4));
                        const uint32_t acc = kb > begin ? 1u : 0u;
#pragma unroll
                        for (uint32_t i = 0; i < 4; ++i)
                            mma_f16_ss<kCG>(d, a_desc + i * a_step, b_desc + i * b_step, idesc, i > 0 ? 1u : acc);
                        if (two) {
#pragma unroll
                            for (uint32_t i = 0; i < 4; ++i)
                                mma_f16_ss<kCG>(d, a_desc + a_next + i * a_step, b_desc + b_next + i * b_step, idesc, 1u);
                        }
                        mma_commit<kCG>(empty0 + 8u * s, 0x3);
                        if (++s == S) {
                            s = 0;
                            ph ^= 1u;
                        }
                    }
                    if (!ok) break;
                    mma_commit<kCG>(tfull0 + 8u * buf, 0x3);
                    ++local;
                }
            }
            mma_commit<kCG>(smem_u32(&ctrl->final_bar), 0x1);
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(smem_u32(&ctrl->final_bar), 0))
                if (globaltimer_ns() - t0 > q.timeout_ns) {
                    atomicCAS(q.err, 0, (int32_t)rg::kErrFinal);
                    break;
                }
        }
        __syncwarp();
    } else {
        const uint32_t quarter = warp & 3u, half = warp >= 7 ? 1u : 0u;
        const uint32_t staging = ring + S * stride + (quarter + 4u * half) * kStaging;
        const int32_t chunks = (q.width + 63) / 64;
        // (G's rows are kWeight's reduction: zeros up to the end of its last k-block)
        const int32_t row_end = !kAnyGrad ? M : kLow ? q.low : (M + kRowPad - 1) / kRowPad * kRowPad;
        uint32_t local = 0, tile = 0;
        if (early) {
            grid_dependency_wait();
            grid_launch_dependents();  // (behind the wait: the mask kernel goes by it)
        }
        float scale = 1.0f;
        if constexpr (kAnyGrad) scale = q.scale ? __ldcg(&q.scale->scale) : scale_of(q.top, q.grad_scale, largest_dloss(q.flags, q.limit, q.dloss, q.dloss_stride, q.M));
        if constexpr (kMode == kWeight) scale = __ldcg(&q.scale->unscale);
        if constexpr (!kPair && kMode == kStats) {
            // The exact logits of the rows' main words (see the joining kernel), while the
            // first tile's weights are on their way: a share of a row per warp, over all CTAs.
            // (A column of W by words is a line per k, and soon a page: with a row per CTA 8
            // rows, 128000 words of 8192 by columns, took 384 us, 313 so, 310 without these
            // sums; with a CTA beside the others for eight rows 430.)
            for (int32_t i = (int32_t)(blockIdx.x + gridDim.x * (quarter + 4u * half)); i < q.M * q.shares; i += 8 * (int32_t)gridDim.x) {
                const int32_t t = i / q.shares, share = i - t * q.shares;
                float weight;
                const int32_t word = main_word(q.sums, t, weight);
                const bool is = word >= 0 && word < q.V;
                const Wide y = is ? exact_share(q.sums, t, word, share, q.shares) : Wide{-INFINITY, 0.0f};
                if (lane == 0) q.exact[i] = (double)y.hi + (double)y.lo;
                if (lane == 0 && share == 0 && q.ids) q.main_weight[t] = weight;
            }
        }
        // the copy issued from the staging buffer before must have read it
        auto turn = [&]() {
            if (lane == 0) bulk_wait_group_read<0>();
            __syncwarp();
        };
        while (next(k)) {
            const int32_t row0 = k.mt * kTileM + 128 * (int32_t)rank + 32 * (int32_t)quarter;
            const int32_t r = row0 + (int32_t)lane, n0 = k.nt * q.width;
            bool live = r < M;
            // what the row's epilogue reads, before the accumulator is waited for
            int32_t t = 0, y = kNone;
            float coef = 0.0f, shift = 0.0f;
            if constexpr (kMode == kStats || kAnyGrad) {
                t = live && gathered ? __ldcg(q.index + r) : r;
                if (kAnyGrad && live && q.flags) {
                    const int32_t f = __ldcg(q.flags + t);
                    live = f >= 0 && f < q.limit;
                }
                if (live && !q.ids) y = __ldcg(q.targets + t);
                if constexpr (kAnyGrad) {
                    if (live) {
                        // (what a logit is less, so that the difference comes before the product with c: next to
                        // 1, p is off by roundings of the difference, not of lse log2(e), 5e-6 for an lse of 100)
                        shift = q.grad_scale * q.lse[t];
                        coef = q.dloss[(int64_t)t * q.dloss_stride] * q.grad_scale * scale;
                    }
                }
            }
            auto release = [&](uint32_t buf) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (kPair)
                        rg::mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&ctrl->tmem_empty[buf]), 0));
                    else
                        mbar_arrive(smem_u32(&ctrl->tmem_empty[buf]));
                }
            };
            const float c = q.log2_scale;
            const Parts<kPair, kMode, kMany> parts(k.kb0, k.kb1, q.bk);
            uint32_t taddr = 0;
            auto filled = [&]() {  // the accumulator of the next part
                const uint32_t buf = local & 1u, bph = (local >> 1) & 1u;
                taddr = tmem_base + ((quarter * 32u) << 16) + buf * buf_cols;
                if (!__all_sync(0xffffffffu, wait_phase(smem_u32(&ctrl->tmem_full[buf]), bph, ctrl, w, rg::kErrEpi))) return false;
                tc_fence_after();
                return true;
            };
            // This warp's chunks of the tile, summed over the parts of the reduction; the last
            // part's accumulator is still held if `keep`.
            auto sum_parts = [&](float(&z)[2][64], bool keep) {
#pragma unroll
                for (int j = 0; j < 64; ++j) z[0][j] = z[1][j] = 0.0f;
#pragma unroll 1
                for (int32_t part = 0; part < parts.count; ++part) {
                    if (!filled()) return false;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int32_t ch = (int32_t)half + 2 * i;
                        if (ch >= chunks || row0 >= row_end) break;  // (uniform over the warp)
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            float v[16];
                            __syncwarp();
                            tmem_load_16cols(taddr + 64u * (uint32_t)ch + 16u * h, v);
#pragma unroll
                            for (int j = 0; j < 16; ++j) z[i][16 * h + j] += v[j];
                        }
                    }
                    if (keep && part == parts.count - 1) break;
                    release(local & 1u);
                    ++local;
                }
                return true;
            };
            if constexpr (kMode == kStats) {
                float z[2][64];
                if (!sum_parts(z, false)) break;
                Wanted want;
                want.start(q, t, y, live, n0);
                const int32_t n_end = min(q.N, n0 + q.width);
                float m_run = -INFINITY, s_run = 0.0f, t_run = 0.0f;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int32_t ch = (int32_t)half + 2 * i, col = n0 + 64 * ch;
                    if (ch >= chunks || col >= q.N || row0 >= M) break;  // (uniform over the warp)
                    const int32_t here = min(64, n_end - col);           // of the chunk's columns
                    float(&v)[64] = z[i];
                    while (want.next < col) want.advance(q);  // (of the other half's chunk)
                    while (__any_sync(0xffffffffu, want.next - col < here)) {
                        const int32_t at = want.next - col;
                        const float x = pick<0, 64>(v, at);
                        if (at < here) {
                            if (want.weight != 0.0f) t_run = fmaf(want.weight, x, t_run);
                            want.advance(q);
                        }
                    }
                    if (here < 64) {
#pragma unroll
                        for (int j = 0; j < 64; ++j) v[j] = j < here ? v[j] : -INFINITY;
                    }
                    float top[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
                    for (int j = 4; j < 64; ++j) top[j % 4] = fmaxf(top[j % 4], v[j]);
                    const float m_new = fmaxf(fmaxf(m_run, fmaxf(top[0], top[1])), fmaxf(top[2], top[3]));
                    // (infinite maxima: the terms are taken as they are, so that the sum says what the row holds.
                    // The difference before the product: the maximum's own term is then 1, where v c - m c, its
                    // second product rounded, was off by half a unit of m c: at z = 100 5e-6 of a sum that a nearly
                    // certain word leaves at 1, so that half of such losses came out negative)
                    const float ref = fabsf(m_new) == INFINITY ? 0.0f : m_new;
                    const Shifted shifted(ref, c);
                    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int j = 0; j < 64; j += 2) {
                        float x0 = v[j], x1 = v[j + 1];
                        shifted(x0, x1);
                        sum[j % 4] += exp2_fast(x0);
                        sum[j % 4 + 1] += exp2_fast(x1);
                    }
                    s_run = fmaf(s_run, exp2_fast((m_run - ref) * c), (sum[0] + sum[1]) + (sum[2] + sum[3]));
                    m_run = m_new;
                }
                // The two halves' as one: the second hands its numbers to the first in one
                // of two buffers.  (It may be two tiles ahead, whose accumulators are
                // filled once the first has read this tile's, not these numbers: it waits
                // for the buffer.)
                float* const hand = reinterpret_cast<float*>(smem + (ring - smem_u32(smem)) + S * stride) + (tile & 1u) * 384u + quarter * 96u + lane;
                const uint32_t given = smem_u32(&ctrl->extra[2u * quarter + (tile & 1u)]);
                const uint32_t taken = smem_u32(&ctrl->peer[2u * quarter + (tile & 1u)]);
                const uint32_t phase = (tile >> 1) & 1u;
                if (half == 1) {
                    if (!__all_sync(0xffffffffu, wait_phase(taken, phase ^ 1u, ctrl, w, rg::kErrEpi))) break;
                    hand[0] = m_run;
                    hand[32] = s_run;
                    hand[64] = t_run;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(given);
                } else {
                    if (!__all_sync(0xffffffffu, wait_phase(given, phase, ctrl, w, rg::kErrEpi))) break;
                    merge_stats(m_run, s_run, hand[0], hand[32], c);
                    t_run += hand[64];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(taken);
                    if (live) {
                        float* const o = q.stats + (int64_t)k.nt * 3 * q.stats_pitch + r;
                        o[0] = m_run;
                        o[q.stats_pitch] = s_run;
                        o[2 * q.stats_pitch] = t_run;
                    }
                }
                ++tile;
                continue;
            }
            Wanted want;
            if constexpr (kAnyGrad) want.start(q, t, y, live, n0 + q.w_row);
            if (kMany && parts.count > 1) {
                // (back into the last accumulator, from where each chunk is taken as if it were
                // the only part: held in registers beside what the epilogue needs, the gradients
                // of 16 rows, 65536 words of 2048, in parts of 256 were 145.5 us for 143.4)
                float z[2][64];
                if (!sum_parts(z, true)) break;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int32_t ch = (int32_t)half + 2 * i;
                    if (ch >= chunks || row0 >= row_end) break;  // (uniform over the warp)
                    __syncwarp();
                    tmem_store_64cols(taddr + 64u * (uint32_t)ch, z[i]);
                }
            } else if (parts.count > 0 && !filled()) {
                break;
            }
            // kGrad: the last tile's zeros go on to the end of a chunk of 64 columns of G,
            // the others stop where the next one begins, inside a chunk perhaps
            const int32_t stop = !kAnyGrad ? min(q.N, n0 + 64 * chunks) : n0 + q.width >= q.N ? (q.N + 63) & ~63 : n0 + q.width;
            auto chunk = [&](float(&v)[64], int32_t ch) {
                const int32_t col = n0 + 64 * ch, c0 = col + q.w_row;         // (c0: its first word)
                if (ch >= chunks || col >= stop || row0 >= row_end) return;  // (uniform over the warp)
                const int32_t here = kAnyGrad ? min(64, stop - col) : 64;
                if constexpr (kAnyGrad) {
                    while (want.next < c0) want.advance(q);  // (of the other half's chunk)
                    const Shifted shifted(shift, c);
#pragma unroll
                    for (int j = 0; j < 64; j += 2) {
                        shifted(v[j], v[j + 1]);
                        const float p0 = coef * exp2_fast(v[j]), p1 = coef * exp2_fast(v[j + 1]);
                        v[j] = live && col + j < q.N ? p0 : 0.0f;
                        v[j + 1] = live && col + j + 1 < q.N ? p1 : 0.0f;
                    }
                    if (here < 64 || kLow) {
                        // the wanted words, where the row does not go through shared memory in one part
                        while (__any_sync(0xffffffffu, want.next - c0 < here)) {
                            const int32_t at = want.next - c0;
                            if (at < here) {
                                const float p = coef * want.weight;
#pragma unroll
                                for (int j = 0; j < 64; ++j) v[j] = j == at ? v[j] - p : v[j];
                                want.advance(q);
                            }
                        }
                    }
                    if (here < 64) {
                        // part of a chunk (the tile's last): straight from the registers
                        uint32_t x[32];
                        pack_64(x, v, 1.0f, q.bf16);
                        uint16_t* dst = q.grad + (int64_t)r * q.grad_pitch + col;
                        const bool write = r < (kLow ? q.low : q.M);
                        for (int part = 0;; ++part) {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                if (8 * i < here && write)
                                    reinterpret_cast<uint4*>(dst)[i] = make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                            if (part == 1 || !kLow) break;
                            dst += (int64_t)q.low * q.grad_pitch;
                            rest_64(x, v, q.bf16);
                        }
                        return;
                    }
                }
                if constexpr (kAnyGrad || kMode == kWeight) {
                    uint32_t x[32];
                    pack_64(x, v, kMode == kWeight ? scale : 1.0f, q.bf16);
                    for (int part = 0;; ++part) {
                        turn();
#pragma unroll
                        for (uint32_t i = 0; i < 8; ++i)
                            rg::st_shared_v4(staging + lane * 128u + ((i ^ (lane & 7u)) << 4),
                                             make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]));
                        if constexpr (kMode == kGrad) {
                            // the wanted words, over what the row's thread has just written
                            int32_t last = kNone;
                            float g = 0.0f;
                            while (__any_sync(0xffffffffu, want.next - c0 < 64)) {
                                const int32_t at = want.next - c0;
                                const float p = pick<0, 64>(v, at);
                                if (at < 64) {
                                    g = (at == last ? g : p) - coef * want.weight;  // (a word may come twice)
                                    last = at;
                                    st_shared_u16(staging + lane * 128u + ((((uint32_t)at >> 3) ^ (lane & 7u)) << 4) + ((uint32_t)at & 7u) * 2u,
                                                  rg::round16(g, q.bf16));
                                    want.advance(q);
                                }
                            }
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            if (kMode == kWeight && q.once)
                                store_2d_hint(&maps.d, staging, col + q.d_col, row0 + q.d_row, l2_policy_evict_first());
                            else
                                tma_store_2d(kLow && part == 1 ? &maps.low : &maps.d, staging, col + q.d_col, row0 + q.d_row);
                            bulk_commit_group();
                        }
                        if (!kLow || part == 1) break;
                        rest_64(x, v, q.bf16);
                    }
                }
                if constexpr (kMode == kSum) {
                    if (k.kb0 == k.kb1 && !q.first) return;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (col + 32 * h >= q.N) break;
                        turn();
#pragma unroll
                        for (uint32_t i = 0; i < 8; ++i)
                            rg::st_shared_v4(staging + lane * 128u + ((i ^ (lane & 7u)) << 4),
                                             make_uint4(__float_as_uint(v[32 * h + 4 * i]), __float_as_uint(v[32 * h + 4 * i + 1]),
                                                        __float_as_uint(v[32 * h + 4 * i + 2]),
                                                        __float_as_uint(v[32 * h + 4 * i + 3])));
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            if (q.first)
                                rg::store_3d(&maps.d, staging, col + 32 * h, row0, k.split);
                            else
                                reduce_add_3d(&maps.d, staging, col + 32 * h, row0, k.split);
                            bulk_commit_group();
                        }
                    }
                }
            };
#pragma unroll 1
            for (int32_t ch = (int32_t)half; ch < chunks; ch += 2) {
                float v[64];
                if (parts.count > 0 && row0 < row_end) {
                    __syncwarp();
                    tmem_load_64cols(taddr + 64u * (uint32_t)ch, v);
                } else {
#pragma unroll
                    for (int j = 0; j < 64; ++j) v[j] = 0.0f;
                }
                chunk(v, ch);
            }
            if (parts.count > 0) {
                release(local & 1u);
                ++local;
            }
            // zeros of the last tile beyond its last chunk
            if constexpr (kAnyGrad) {
                const int32_t from = n0 + 64 * chunks;
                if (half == 0 && from < stop && r < (kLow ? q.low : q.M)) {
                    uint16_t* const dst = q.grad + (int64_t)r * q.grad_pitch;
                    for (int32_t col = from; col < stop; col += 8) {
                        *reinterpret_cast<uint4*>(dst + col) = make_uint4(0, 0, 0, 0);
                        if constexpr (kLow) *reinterpret_cast<uint4*>(dst + (int64_t)q.low * q.grad_pitch + col) = make_uint4(0, 0, 0, 0);
                    }
                }
            }
        }
        if (lane == 0) bulk_wait_group_all();
        __syncwarp();
    }

    if (q.late) grid_dependency_wait();
    if constexpr (kMode == kWeight) {
        if (q.finish.dX) finish_dx(q.finish, kThreads);  // the sums are complete
    }
    __syncthreads();
    if (threadIdx.x == 0 && *(volatile int32_t*)&ctrl->abort_flag) rg::drain_ring(ctrl, full0, S);
    tc_fence_before();
    if (kPair)
        cluster_sync_relaxed();  // the other CTA's accesses to this one's shared memory are done
    else
        __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<kCG>(tmem_base, q.tmem_cols);
    }
}

}  // namespace ls
}  // namespace gr
