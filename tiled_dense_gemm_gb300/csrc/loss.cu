// C entry points of the losses over a vocabulary: cross entropy and
// distillation from a teacher's best words, each with its gradients.  Argument
// checks, plan, tensor maps, launches; the kernels are in loss_kernel.cuh and
// loss_rows.cuh.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <mutex>

#include "gemm_relu.h"
#include "launch.h"
#include "loss_kernel.cuh"
#include "loss_plan.h"
#include "loss_rows.cuh"
#include "runtime.h"

namespace gr {
namespace ls {

using rt::DeviceState;
using rt::encode_rows;
using rt::launch;
using rt::misaligned;

// What a call is given.
struct Call {
    const void *X, *W;
    int64_t T, V, D, ldx;
    bool nk, bf16;
    const int32_t* targets;  // or
    const int32_t* ids;      // a teacher's words
    const void* logits;
    int64_t k, ld_ids, ld_logits;
    int logits_type;
    float tau;
    float *loss, *lse_out;   // forward
    const float *lse, *dloss;  // backward
    int64_t dloss_stride;
    void *dX, *dW;
    int64_t ld_dx;
    uint8_t* ws;
    cudaStream_t st;
};

// Sums in 32 bits, a plane per share: boxes of 32 x 32.
static int encode_sums(CUtensorMap* map, void* ptr, int64_t D, int64_t T, int64_t splits) {
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)T, (cuuint64_t)splits};
    cuuint64_t strides[2] = {(cuuint64_t)D * 4, (cuuint64_t)(D * T) * 4};
    cuuint32_t box[3] = {32, 32, 1}, step[3] = {1, 1, 1};
    const CUresult r = rt::g_encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, ptr, dims, strides, box, step,
                                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? GEMM_OK : GEMM_ERR_INVALID_ARG;
}

template <bool kPair, int kMode, bool kMany>
static int launch_kernel(DeviceState& d, const TilePlan& t, const LossMaps& m, const LossParams& q, cudaStream_t st) {
    auto fn = loss_kernel<kPair, kMode, kMany>;
    bool& set = d.ls_attr_set[4 * kMode + 2 * kMany + kPair];
    if (!set) {
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, rt::kMaxDynSmem) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_LAUNCH;
        }
        set = true;
    }
    return launch(fn, t.grid, kThreads, (size_t)t.smem_bytes, kPair ? 2 : 1, st, m, q);
}

template <bool kPair, int kMode>
static int launch_tiles(DeviceState& d, const TilePlan& t, const LossMaps& m, const LossParams& q, cudaStream_t st) {
    if constexpr (kMode != kStats) {
        const int64_t blocks = ((int64_t)q.K + q.bk - 1) / q.bk, share = (blocks + q.splits - 1) / q.splits;
        if (share * q.bk <= Parts<kPair, kMode, true>::kPart) return launch_kernel<kPair, kMode, false>(d, t, m, q, st);
    }
    return launch_kernel<kPair, kMode, true>(d, t, m, q, st);
}

// Up to so many rows (four row tiles of a pair) the weights are read from memory,
// and their gradients written, with lines that leave L2 first: they are met once
// or by CTAs that run together, and otherwise push out what is reused (us, without
// / with; 32768 words of 1024: one row 18.0 / 16.6, gradients 50.3 / 46.6; 65536 of
// 2048: 16 rows 52.2 / 46.1, 147 / 132; 100 rows 54.5 / 50.6, 158 / 146; 300 97 /
// 93, 259 / 249; 32768 of 1024, 1000 rows: 56 / 56, 155.5 / 152.8; but 65536 of
// 4096, 4096 rows: 1185 / 1188, 3903 / 3947).
constexpr int64_t kStreamRows = 1024;

template <int kMode>
static int launch_mode(DeviceState& d, const TilePlan& t, const LossMaps& m, LossParams& q, int64_t rows, cudaStream_t st) {
    q.width = t.width;
    q.bk = t.bk;
    q.once = rows <= kStreamRows;
    q.n_tiles = t.n_tiles;
    q.group_m = t.group_m;
    q.splits = t.splits;
    q.a_bytes = (uint32_t)t.a_bytes;
    q.stage_bytes = (uint32_t)t.stage_bytes;
    q.num_stages = t.num_stages;
    q.tmem_cols = (uint32_t)t.tmem_cols;
    q.err = d.d_err;
    const int64_t blocks = ((int64_t)q.K + q.bk - 1) / q.bk;
    q.timeout_ns = 2000000000ull + 2000ull * (uint64_t)blocks;
    if (kMode == kStats) {
        const int rc = rt::test_hook(!t.pair, (int32_t)std::min<int64_t>(blocks, kNone), &q.test_drop_kb, &q.timeout_ns);
        if (rc != GEMM_OK) return rc;
    }
    if constexpr (kMode != kGradLow)
        if (t.pair) return launch_tiles<true, kMode>(d, t, m, q, st);
    return launch_tiles<false, kMode>(d, t, m, q, st);  // (few rows: never pairs)
}

// A row is in use where its flag is in [0, limit).
static const int32_t* flags_of(const Call& c, const LossPlan& p, int64_t b0) {
    return c.ids ? reinterpret_cast<const int32_t*>(c.ws + p.flags) : c.targets + b0;
}

static int32_t limit_of(const Call& c) { return c.ids ? 1 : (int32_t)c.V; }

// The teacher's words of rows [b0, b0 + T).
static int run_teacher(const Call& c, const LossPlan& p, int64_t b0, int64_t T, DeviceState& d) {
    int rc;
    if (c.ids) {
        TeacherParams q;
        memset(&q, 0, sizeof(q));
        q.ids = c.ids + b0 * c.ld_ids;
        q.logits = reinterpret_cast<const uint8_t*>(c.logits) + b0 * c.ld_logits * (c.logits_type == GEMM_LOGITS_F32 ? 4 : 2);
        q.ld_ids = c.ld_ids;
        q.ld_logits = c.ld_logits;
        q.logits_type = c.logits_type;
        q.T = (int32_t)T;
        q.k = (int32_t)c.k;
        q.V = (int32_t)c.V;
        q.before = p.masked;
        q.inv_tau = 1.0f / c.tau;
        q.sorted = reinterpret_cast<int32_t*>(c.ws + p.sorted);
        q.weights = reinterpret_cast<float*>(c.ws + p.weights);
        q.flags = reinterpret_cast<int32_t*>(c.ws + p.flags);
        q.entropy = reinterpret_cast<float*>(c.ws + p.entropy);
        q.err = d.d_err;
        const int grid = (int)std::min<int64_t>((T + kTeacherWarps - 1) / kTeacherWarps, 16 * d.sm_count);
        rc = launch(loss_teacher_kernel, grid, 32 * kTeacherWarps, (size_t)kTeacherWarps * ((c.k + 3) / 4 * 4) * 8, 1, c.st, q);
        if (rc != GEMM_OK) return rc;
    }
    return GEMM_OK;
}

// What the largest |dloss tau| is scaled to.  The largest entries of G, a (p - 1)
// of wanted words that are not foreseen, are near the top of a binade, where a
// 16-bit type rounds finest, and the limit itself is exact; binary16 besides keeps
// what it can of small ones.
static float top_of(const Call& c) { return c.bf16 ? 255.0f / 128.0f : 2047.0f / 1024.0f * 16384.0f; }

// What the logits of single words are summed from (up to 128 rows).
static WordSums word_sums(const Call& c, const LossPlan& p) {
    WordSums s;
    memset(&s, 0, sizeof(s));
    s.X = reinterpret_cast<const uint16_t*>(c.X);
    s.ldx = c.ldx;
    s.W = reinterpret_cast<const uint16_t*>(c.W);
    s.w_word = c.nk ? c.D : 1;
    s.w_depth = c.nk ? 1 : c.V;
    s.targets = c.targets;
    if (c.ids) {
        s.ids = reinterpret_cast<const int32_t*>(c.ws + p.sorted);
        s.weights = reinterpret_cast<const float*>(c.ws + p.weights);
        s.k = (int32_t)c.k;
    }
    s.D = (int32_t)c.D;
    s.bf16 = c.bf16 ? 1 : 0;
    return s;
}

// Which rows [b0, b0 + T) are in use, and a copy of those.
static int run_rows(const Call& c, const LossPlan& p, int64_t b0, int64_t T, DeviceState& d, int64_t p0 = 0) {
    RowsParams q;
    memset(&q, 0, sizeof(q));
    q.flags = flags_of(c, p, b0);
    q.limit = limit_of(c);
    q.T = (int32_t)T;
    q.D = (int32_t)c.D;
    q.X = reinterpret_cast<const uint16_t*>(c.X) + b0 * c.ldx;
    q.ldx = c.ldx;
    q.pitch = (int32_t)p.pitch;
    // X's pitch not a multiple of 128 bytes: the copy's is (5000 rows, 50021 words of
    // 1544: 547 us from X, 536 from the copy; the gradients 1856 and 1805).
    q.always = T > 128 && (c.ldx % 64 != 0 || misaligned(q.X, 128));
    q.gathered = reinterpret_cast<uint16_t*>(c.ws + p.gathered);
    q.index = reinterpret_cast<int32_t*>(c.ws + p.index);
    q.rows = reinterpret_cast<RowsHeader*>(c.ws + p.header);
    q.dloss = c.dloss;
    q.dloss_stride = c.dloss_stride;
    q.grad_scale = c.ids ? c.tau : 1.0f;
    q.top = top_of(c);
    q.err = d.d_err;
    if (p.masked) {
        q.rows_of = (int32_t)p.g_rows;
        q.period = p.low ? p.low : (int32_t)T;
        q.sums = word_sums(c, p);
        q.tau = c.ids ? c.tau : 1.0f;
        q.lse = c.lse;
        q.grad = reinterpret_cast<uint16_t*>(c.ws + p.grad);
        q.grad_pitch = p.piece;
        q.from = (int32_t)p0;
        q.words = (int32_t)std::min(p.piece, c.V - p0);
        q.low = p.low;
        return launch(loss_mask_kernel, q.rows_of, kRowsThreads, 0, 1, c.st, q);
    }
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>((T + 7) / 8, 4 * d.sm_count));
    return launch(loss_rows_kernel, grid, kRowsThreads, 0, 1, c.st, q);
}

static float log2_scale(float tau) { return 1.4426950408889634f / tau; }

// The wanted words and the rows, for kStats and kGrad.
static void wanted(const Call& c, const LossPlan& p, int64_t b0, LossParams& q) {
    q.rows = p.gather ? reinterpret_cast<const RowsHeader*>(c.ws + p.header) : nullptr;
    q.rows_m = p.gather ? 1 : 0;
    q.index = reinterpret_cast<const int32_t*>(c.ws + p.index);
    if (c.ids) {
        q.ids = reinterpret_cast<const int32_t*>(c.ws + p.sorted);
        q.weights = reinterpret_cast<const float*>(c.ws + p.weights);
        q.k = (int32_t)c.k;
    } else {
        q.targets = c.targets + b0;
    }
    q.V = (int32_t)c.V;
    q.log2_scale = log2_scale(c.tau);
}

// An mn-major operand of `rows` x `width` (k and its rows' index): the chunks of a
// stage in one copy, but chunk by chunk through `edge` where a row's end cuts
// through the last.  (Copies issue one after another, 450 clocks each: two of 64
// columns per stage held a pair's k-block of 64 at 900.)
static int encode_chunks(CUtensorMap* map, CUtensorMap* edge, const void* ptr, int64_t width, int64_t rows, int64_t pitch, int bk,
                         int chunks, bool bf16, int32_t* in_one, int32_t* blocks) {
    *in_one = width >= 64;
    *blocks = width % 64 == 0 ? kNone : (int32_t)(width / 64);
    int rc = encode_rows(edge, ptr, (uint64_t)width, (uint64_t)rows, (uint64_t)pitch, (uint32_t)bk, 0, bf16);
    if (rc != GEMM_OK) return rc;
    if (*in_one) return encode_rows(map, ptr, (uint64_t)width, (uint64_t)rows, (uint64_t)pitch, (uint32_t)bk, (uint32_t)chunks, bf16);
    *map = *edge;
    return GEMM_OK;
}

// W as B's side of the logits (reduction D).
static int encode_words(LossMaps& m, const Call& c, const TilePlan& t, LossParams& q) {
    const int width = t.width / (t.pair ? 2 : 1);
    q.b_mn = c.nk ? 0 : 1;
    int rc;
    if (c.nk) {
        q.b_3d = c.D % 64 == 0;
        rc = encode_rows(&m.b[0], c.W, (uint64_t)c.D, (uint64_t)c.V, (uint64_t)c.D, (uint32_t)width, q.b_3d ? (uint32_t)t.bk / 64 : 0, c.bf16);
    } else {
        rc = encode_chunks(&m.b[0], &m.edge[0], c.W, c.V, c.D, c.V, t.bk, width / 64, c.bf16, &q.b_3d, &q.b_blocks);
        m.edge[1] = m.edge[0];
    }
    m.b[1] = m.b[0];
    return rc;
}

// X's rows and their gathered copy as A's side of the logits.
static int encode_rows_of_x(LossMaps& m, const Call& c, const LossPlan& p, int64_t b0, int64_t T, const TilePlan& t, LossParams& q) {
    q.a_3d = c.D % 64 == 0;
    const uint32_t blocks = q.a_3d ? (uint32_t)t.bk / 64 : 0;
    int rc = encode_rows(&m.a[0], reinterpret_cast<const uint16_t*>(c.X) + b0 * c.ldx, (uint64_t)c.D, (uint64_t)T, (uint64_t)c.ldx,
                         (uint32_t)t.a_rows, blocks, c.bf16);
    m.a[1] = m.a[0];
    if (rc == GEMM_OK && p.gather)
        rc = encode_rows(&m.a[1], c.ws + p.gathered, (uint64_t)c.D, (uint64_t)T, (uint64_t)p.pitch, (uint32_t)t.a_rows, blocks, c.bf16);
    return rc;
}

static int run_forward(const Call& c, const LossPlan& p, DeviceState& d) {
    for (int64_t b0 = 0; b0 < c.T; b0 += p.rows) {
        const int64_t T = std::min(p.rows, c.T - b0);
        int rc = run_teacher(c, p, b0, T, d);
        if (rc == GEMM_OK && p.gather) rc = run_rows(c, p, b0, T, d);
        if (rc != GEMM_OK) return rc;
        TilePlan t = plan_logits(T, c.V, c.D, !c.nk, true, d.sm_count, d.max_pairs);
        LossMaps m;
        LossParams q;
        memset(&q, 0, sizeof(q));
        q.M = (int32_t)T;
        q.N = (int32_t)c.V;
        q.K = (int32_t)c.D;
        q.bf16 = c.bf16 ? 1 : 0;
        wanted(c, p, b0, q);
        q.stats = reinterpret_cast<float*>(c.ws + p.stats);
        q.stats_pitch = (p.rows + 31) / 32 * 32;
        if (!p.gather) {  // (one block of rows)
            q.exact = reinterpret_cast<double*>(c.ws + p.exact);
            q.main_weight = reinterpret_cast<float*>(c.ws + p.main_weight);
            q.sums = word_sums(c, p);
            // a share per warp of the tiles' CTAs, and of others where those are few
            const int64_t most = (c.D + 255) / 256;
            t.grid = (int32_t)std::max<int64_t>(t.grid, std::min<int64_t>(d.sm_count, (T * most + 7) / 8));
            q.shares = (int32_t)std::max<int64_t>(1, std::min(most, std::min<int64_t>(8 * t.grid, kMostShares) / T));
        }
        rc = encode_rows_of_x(m, c, p, b0, T, t, q);
        if (rc == GEMM_OK) rc = encode_words(m, c, t, q);
        if (rc != GEMM_OK) return rc;
        m.d = m.a[0];
        rc = launch_mode<kStats>(d, t, m, q, T, c.st);
        if (rc != GEMM_OK) return rc;
        CombineParams o;
        memset(&o, 0, sizeof(o));
        o.stats = q.stats;
        o.pitch = q.stats_pitch;
        o.parts = t.n_tiles;
        o.T = (int32_t)T;
        o.rows = q.rows;
        o.index = q.index;
        o.flags = flags_of(c, p, b0);
        o.limit = limit_of(c);
        o.entropy = c.ids ? reinterpret_cast<const float*>(c.ws + p.entropy) : nullptr;
        o.exact = q.exact;
        o.shares = q.shares;
        o.main_weight = q.main_weight;
        o.tau = c.tau;
        o.log2_scale = q.log2_scale;
        o.loss = c.loss + b0;
        o.lse = c.lse_out + b0;
        o.err = d.d_err;
        const int grid = (int)((T + 7) / 8);
        rc = !p.gather ? launch(loss_combine_kernel<32, true>, grid, 1024, 0, 1, c.st, o)
             : T <= 1024 ? launch(loss_combine_kernel<32, false>, grid, 1024, 0, 1, c.st, o)
                         : launch(loss_combine_kernel<16, false>, grid, 512, 0, 1, c.st, o);
        if (rc != GEMM_OK) return rc;
    }
    return GEMM_OK;
}

static FinishParams finish_of(const Call& c, const LossPlan& p) {
    FinishParams f;
    memset(&f, 0, sizeof(f));
    f.sums = reinterpret_cast<const float*>(c.ws + p.sums);
    f.splits = p.sum_splits;
    f.T = (int32_t)c.T;
    f.rows_of = (int32_t)p.g_rows;
    f.low = p.low;
    f.D = (int32_t)c.D;
    f.bf16 = c.bf16 ? 1 : 0;
    f.rows = reinterpret_cast<const RowsHeader*>(c.ws + p.header);
    f.index = p.masked ? nullptr : reinterpret_cast<const int32_t*>(c.ws + p.index);
    f.flags = flags_of(c, p, 0);
    f.limit = limit_of(c);
    f.dX = reinterpret_cast<uint16_t*>(c.dX);
    f.ld_dx = c.ld_dx;
    return f;
}

static int run_backward(const Call& c, const LossPlan& p, DeviceState& d) {
    int rc = run_teacher(c, p, 0, c.T, d);
    if (rc == GEMM_OK && p.gather) rc = run_rows(c, p, 0, c.T, d);
    if (rc != GEMM_OK) return rc;
    const RowsHeader* rows = reinterpret_cast<const RowsHeader*>(c.ws + p.header);
    const RowsHeader* counted = p.masked ? nullptr : rows;
    uint16_t* const G = reinterpret_cast<uint16_t*>(c.ws + p.grad);
    float* const sums = reinterpret_cast<float*>(c.ws + p.sums);
    for (int64_t p0 = 0; p0 < c.V; p0 += p.piece) {
        const int64_t vp = std::min(p.piece, c.V - p0);
        LossMaps m;
        LossParams q;
        {  // G of the piece
            // (the rows' kernel beside it, eight blocks on an SM: 65536 words of 2048, 64
            // rows 139 us with none left for it, 136 so; 16 rows 137 and 132)
            const int sms = p.masked ? std::max(d.sm_count - (int)((p.g_rows + 7) / 8), d.sm_count / 2) : d.sm_count;
            const TilePlan t = plan_logits(c.T, vp, c.D, !c.nk, false, sms, d.max_pairs);
            memset(&q, 0, sizeof(q));
            q.M = (int32_t)c.T;
            q.N = (int32_t)vp;
            q.K = (int32_t)c.D;
            q.bf16 = c.bf16 ? 1 : 0;
            wanted(c, p, 0, q);
            q.early = c.ids && p.masked && p0 == 0;  // (behind the teacher's kernel)
            q.w_row = (int32_t)p0;
            q.scale = p.masked ? nullptr : rows;
            q.top = top_of(c);
            if (p.masked) {
                q.flags = flags_of(c, p, 0);
                q.limit = limit_of(c);
            }
            q.lse = c.lse;
            q.dloss = c.dloss;
            q.dloss_stride = c.dloss_stride;
            q.grad_scale = c.ids ? c.tau : 1.0f;
            q.grad = G;
            q.grad_pitch = p.piece;
            rc = encode_rows_of_x(m, c, p, 0, c.T, t, q);
            if (rc == GEMM_OK) rc = encode_words(m, c, t, q);
            if (rc == GEMM_OK)
                rc = encode_rows(&m.d, G, (uint64_t)p.piece, (uint64_t)(p.low ? p.low : c.T), (uint64_t)p.piece, 32, 0, c.bf16);
            if (rc == GEMM_OK && p.low)
                rc = encode_rows(&m.low, G + p.low * p.piece, (uint64_t)p.piece, (uint64_t)p.low, (uint64_t)p.piece, 32, 0, c.bf16);
            q.low = p.low;
            if (rc == GEMM_OK) rc = p.low ? launch_mode<kGradLow>(d, t, m, q, c.T, c.st) : launch_mode<kGrad>(d, t, m, q, c.T, c.st);
            if (rc == GEMM_OK && p.masked) rc = run_rows(c, p, 0, c.T, d, p0);
            if (rc != GEMM_OK) return rc;
        }
        if (c.dX) {  // sums += G W
            const TilePlan t = plan_sum(p.g_rows, c.D, p.sum_splits, p.sum_width, c.nk, d.sm_count, d.max_pairs);
            const uint32_t width = (uint32_t)(t.width / (t.pair ? 2 : 1));
            memset(&q, 0, sizeof(q));
            q.M = (int32_t)p.g_rows;
            q.N = (int32_t)c.D;
            q.K = (int32_t)vp;
            q.bf16 = c.bf16 ? 1 : 0;
            q.rows = counted;
            q.rows_m = counted ? 1 : 0;
            q.first = p0 == 0;
            q.w_k = (int32_t)p0;
            q.b_mn = c.nk ? 1 : 0;
            q.a_3d = 1;  // (G is zero from its last word to the end of that chunk)
            rc = encode_rows(&m.a[0], G, (uint64_t)((vp + 63) / 64 * 64), (uint64_t)p.g_rows, (uint64_t)p.piece, (uint32_t)t.a_rows,
                             (uint32_t)t.bk / 64, c.bf16);
            if (rc == GEMM_OK && c.nk) {
                rc = encode_chunks(&m.b[0], &m.edge[0], c.W, c.D, c.V, c.D, t.bk, (int)width / 64, c.bf16, &q.b_3d, &q.b_blocks);
            } else if (rc == GEMM_OK) {
                q.b_3d = c.V % 64 == 0;
                rc = encode_rows(&m.b[0], c.W, (uint64_t)c.V, (uint64_t)c.D, (uint64_t)c.V, width, q.b_3d ? (uint32_t)t.bk / 64 : 0, c.bf16);
            }
            if (rc == GEMM_OK) rc = encode_sums(&m.d, sums, c.D, p.g_rows, p.sum_splits);
            m.a[1] = m.a[0];
            m.b[1] = m.b[0];
            m.edge[1] = m.edge[0];
            if (rc == GEMM_OK) rc = launch_mode<kSum>(d, t, m, q, c.T, c.st);
            if (rc != GEMM_OK) return rc;
        }
        if (c.dW) {  // dW[piece] = G^T X, or its transpose
            const int64_t M = c.nk ? vp : c.D, N = c.nk ? c.D : vp;
            const TilePlan t = plan_weight(M, N, d.sm_count, d.max_pairs);
            const int b_chunks = t.width / (t.pair ? 2 : 1) / 64, g_chunks = c.nk ? 2 : b_chunks, x_chunks = c.nk ? b_chunks : 2;
            memset(&q, 0, sizeof(q));
            q.M = (int32_t)M;
            q.N = (int32_t)N;
            q.K = (int32_t)p.g_rows;
            q.bf16 = c.bf16 ? 1 : 0;
            q.rows = counted;
            q.rows_k = counted ? 1 : 0;
            q.scale = rows;
            q.late = c.dX ? 1 : 0;  // (beside the end of kSum, which has waited for G)
            if (c.dX && p0 + p.piece >= c.V) q.finish = finish_of(c, p);
            q.a_mn = q.b_mn = 1;
            (c.nk ? q.d_row : q.d_col) = (int32_t)p0;
            CUtensorMap* const mg = c.nk ? m.a : m.b;
            CUtensorMap* const mx = c.nk ? m.b : m.a;
            (c.nk ? q.a_3d : q.b_3d) = 1;
            (c.nk ? q.a_blocks : q.b_blocks) = kNone;
            int32_t* const x_in_one = c.nk ? &q.b_3d : &q.a_3d;
            int32_t* const x_blocks = c.nk ? &q.b_blocks : &q.a_blocks;
            rc = encode_rows(&mg[0], G, (uint64_t)p.piece, (uint64_t)p.g_rows, (uint64_t)p.piece, (uint32_t)t.bk, (uint32_t)g_chunks, c.bf16);
            mg[1] = mg[0];
            // the copy: where rows are masked, the only one (the kernel takes the first map then)
            if (rc == GEMM_OK)
                rc = encode_chunks(&mx[1], &m.edge[1], c.ws + p.gathered, c.D, p.g_rows, p.pitch, t.bk, x_chunks, c.bf16, x_in_one, x_blocks);
            mx[0] = mx[1];
            m.edge[0] = m.edge[1];
            if (rc == GEMM_OK && !p.masked)
                rc = encode_chunks(&mx[0], &m.edge[0], c.X, c.D, c.T, c.ldx, t.bk, x_chunks, c.bf16, x_in_one, x_blocks);
            if (rc == GEMM_OK)
                rc = c.nk ? encode_rows(&m.d, c.dW, (uint64_t)c.D, (uint64_t)c.V, (uint64_t)c.D, 32, 0, c.bf16)
                          : encode_rows(&m.d, c.dW, (uint64_t)c.V, (uint64_t)c.D, (uint64_t)c.V, 32, 0, c.bf16);
            if (rc == GEMM_OK) rc = launch_mode<kWeight>(d, t, m, q, c.T, c.st);
            if (rc != GEMM_OK) return rc;
        }
    }
    if (!c.dX || c.dW) return GEMM_OK;
    const int64_t vecs = c.T * (c.D / 8);
    return launch(loss_finish_kernel, (int)std::min<int64_t>((vecs + 255) / 256, 8 * d.sm_count), 256, 0, 1, c.st, finish_of(c, p));
}

// ------------------------------------------------------------------ checks

static int check_sizes(int64_t T, int64_t V, int64_t D, int64_t k) {
    if (T < 0 || T > GEMM_RELU_MAX_LOSS_ROWS || V < 1 || V > GEMM_RELU_MAX_WORDS || D < 1 ||
        D > GEMM_RELU_MAX_LOSS_WIDTH || k < 0 || k > GEMM_RELU_MAX_TEACHER_WORDS)
        return GEMM_ERR_INVALID_ARG;
    return D % 8 != 0 ? GEMM_ERR_ALIGNMENT : GEMM_OK;
}

static int check_floats(const void* p) {
    if (!p) return GEMM_ERR_INVALID_ARG;
    return misaligned(p, 4) ? GEMM_ERR_ALIGNMENT : GEMM_OK;
}

// Everything but the outputs.
static int check_call(const Call& c, int b_layout, int dtype) {
    int rc = check_sizes(c.T, c.V, c.D, c.k);
    if (rc != GEMM_OK) return rc;
    if ((b_layout != GEMM_B_KN && b_layout != GEMM_B_NK) || (dtype != GEMM_DTYPE_F16 && dtype != GEMM_DTYPE_BF16))
        return GEMM_ERR_INVALID_ARG;
    if (b_layout == GEMM_B_KN && c.V % 8 != 0) return GEMM_ERR_ALIGNMENT;
    if (c.T == 0) return GEMM_OK;
    if ((rc = rt::check_matrix(c.X, c.D, c.ldx)) != GEMM_OK) return rc;
    return rt::check_matrix(c.W, 0, 0);
}

static int check_teacher(const Call& c) {
    if (c.k < 1 || !(c.tau > 0.0f) || !isfinite(c.tau) || !isfinite(log2_scale(c.tau))) return GEMM_ERR_INVALID_ARG;
    if (c.logits_type != GEMM_LOGITS_F16 && c.logits_type != GEMM_LOGITS_BF16 && c.logits_type != GEMM_LOGITS_F32)
        return GEMM_ERR_INVALID_ARG;
    if (c.T == 0) return GEMM_OK;
    if (!c.ids || !c.logits || c.ld_ids < c.k || c.ld_logits < c.k || c.ld_ids > GEMM_RELU_MAX_DIM || c.ld_logits > GEMM_RELU_MAX_DIM)
        return GEMM_ERR_INVALID_ARG;
    return misaligned(c.ids, 4) || misaligned(c.logits, c.logits_type == GEMM_LOGITS_F32 ? 4 : 2) ? GEMM_ERR_ALIGNMENT : GEMM_OK;
}

static int run(Call& c, void* workspace, int64_t workspace_bytes, bool gradient, void* stream) {
    const LossPlan p = plan_loss(c.T, c.V, c.D, c.k, gradient);
    if (p.status != GEMM_OK) return p.status;
    if (!workspace || workspace_bytes < p.bytes) return GEMM_ERR_INVALID_ARG;
    if (misaligned(workspace, 256)) return GEMM_ERR_ALIGNMENT;
    c.ws = reinterpret_cast<uint8_t*>(workspace);
    c.st = reinterpret_cast<cudaStream_t>(stream);
    int dev, rc;
    if ((rc = rt::current_device(&dev)) != GEMM_OK) return rc;
    std::lock_guard<std::mutex> lock(rt::g_mu);
    if ((rc = rt::init_device_locked(dev)) != GEMM_OK) return rc;
    return gradient ? run_backward(c, p, rt::g_dev[dev]) : run_forward(c, p, rt::g_dev[dev]);
}

static int forward(Call& c, void* workspace, int64_t workspace_bytes, void* stream) {
    if (c.T == 0) return GEMM_OK;
    int rc;
    if ((rc = check_floats(c.loss)) != GEMM_OK || (rc = check_floats(c.lse_out)) != GEMM_OK) return rc;
    return run(c, workspace, workspace_bytes, false, stream);
}

static int backward(Call& c, void* workspace, int64_t workspace_bytes, void* stream) {
    int rc;
    if (c.dloss_stride != 0 && c.dloss_stride != 1) return GEMM_ERR_INVALID_ARG;
    if (c.dW && misaligned(c.dW, 16)) return GEMM_ERR_ALIGNMENT;
    if (c.T == 0) {
        if (!c.dW) return GEMM_OK;
        int dev;
        if ((rc = rt::current_device(&dev)) != GEMM_OK) return rc;
        if (cudaMemsetAsync(c.dW, 0, (size_t)c.V * c.D * 2, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_CUDA;
        }
        return GEMM_OK;
    }
    if ((rc = check_floats(c.lse)) != GEMM_OK || (rc = check_floats(c.dloss)) != GEMM_OK) return rc;
    if (c.dX && (rc = rt::check_matrix(c.dX, c.D, c.ld_dx)) != GEMM_OK) return rc;
    if (!c.dX && !c.dW) return GEMM_OK;
    return run(c, workspace, workspace_bytes, true, stream);
}

static Call call_of(const void* X, const void* W, int64_t T, int64_t V, int64_t D, int64_t ldx, int b_layout, int dtype) {
    Call c;
    memset(&c, 0, sizeof(c));
    c.X = X;
    c.W = W;
    c.T = T;
    c.V = V;
    c.D = D;
    c.ldx = ldx;
    c.nk = b_layout == GEMM_B_NK;
    c.bf16 = dtype == GEMM_DTYPE_BF16;
    c.tau = 1.0f;
    return c;
}

}  // namespace ls
}  // namespace gr

using namespace gr;
using namespace gr::ls;

extern "C" int64_t gemm_relu_loss_workspace(int64_t T, int64_t V, int64_t D, int64_t k, int gradient) {
    const int rc = check_sizes(T, V, D, k);
    if (rc != GEMM_OK) return -rc;
    if (T == 0) return 0;
    const LossPlan p = plan_loss(T, V, D, k, gradient != 0);
    return p.status == GEMM_OK ? p.bytes : -p.status;
}

extern "C" int gemm_relu_xent(const void* X, const void* W, const int32_t* targets, float* loss, float* lse, int64_t T,
                              int64_t V, int64_t D, int64_t ldx, int b_layout, int dtype, void* workspace,
                              int64_t workspace_bytes, void* stream) {
    Call c = call_of(X, W, T, V, D, ldx, b_layout, dtype);
    c.targets = targets;
    c.loss = loss;
    c.lse_out = lse;
    int rc = check_call(c, b_layout, dtype);
    if (rc != GEMM_OK) return rc;
    if (T > 0 && (rc = check_floats(targets)) != GEMM_OK) return rc;
    return forward(c, workspace, workspace_bytes, stream);
}

extern "C" int gemm_relu_xent_grad(const void* X, const void* W, const int32_t* targets, const float* lse, const float* dloss,
                                   int64_t dloss_stride, void* dX, void* dW, int64_t T, int64_t V, int64_t D, int64_t ldx,
                                   int64_t ld_dx, int b_layout, int dtype, void* workspace, int64_t workspace_bytes,
                                   void* stream) {
    Call c = call_of(X, W, T, V, D, ldx, b_layout, dtype);
    c.targets = targets;
    c.lse = lse;
    c.dloss = dloss;
    c.dloss_stride = dloss_stride;
    c.dX = dX;
    c.dW = dW;
    c.ld_dx = ld_dx;
    int rc = check_call(c, b_layout, dtype);
    if (rc != GEMM_OK) return rc;
    if (T > 0 && (rc = check_floats(targets)) != GEMM_OK) return rc;
    return backward(c, workspace, workspace_bytes, stream);
}

extern "C" int gemm_relu_distill(const void* X, const void* W, const int32_t* ids, const void* logits, float temperature,
                                 float* loss, float* lse, int64_t T, int64_t V, int64_t D, int64_t k, int64_t ldx,
                                 int64_t ld_ids, int64_t ld_logits, int b_layout, int dtype, int logits_type,
                                 void* workspace, int64_t workspace_bytes, void* stream) {
    Call c = call_of(X, W, T, V, D, ldx, b_layout, dtype);
    c.ids = ids;
    c.logits = logits;
    c.k = k;
    c.ld_ids = ld_ids;
    c.ld_logits = ld_logits;
    c.logits_type = logits_type;
    c.tau = temperature;
    c.loss = loss;
    c.lse_out = lse;
    int rc = check_call(c, b_layout, dtype);
    if (rc == GEMM_OK) rc = check_teacher(c);
    return rc != GEMM_OK ? rc : forward(c, workspace, workspace_bytes, stream);
}

extern "C" int gemm_relu_distill_grad(const void* X, const void* W, const int32_t* ids, const void* logits, float temperature,
                                      const float* lse, const float* dloss, int64_t dloss_stride, void* dX, void* dW,
                                      int64_t T, int64_t V, int64_t D, int64_t k, int64_t ldx, int64_t ld_ids,
                                      int64_t ld_logits, int64_t ld_dx, int b_layout, int dtype, int logits_type,
                                      void* workspace, int64_t workspace_bytes, void* stream) {
    Call c = call_of(X, W, T, V, D, ldx, b_layout, dtype);
    c.ids = ids;
    c.logits = logits;
    c.k = k;
    c.ld_ids = ld_ids;
    c.ld_logits = ld_logits;
    c.logits_type = logits_type;
    c.tau = temperature;
    c.lse = lse;
    c.dloss = dloss;
    c.dloss_stride = dloss_stride;
    c.dX = dX;
    c.dW = dW;
    c.ld_dx = ld_dx;
    int rc = check_call(c, b_layout, dtype);
    if (rc == GEMM_OK) rc = check_teacher(c);
    return rc != GEMM_OK ? rc : backward(c, workspace, workspace_bytes, stream);
}
