// C entry points of the ragged products: experts' products grouped by row
// offsets (forward, data gradient, weight gradient) and low-rank adapters
// beside a shared weight.  Argument checks, plan, tensor maps, workspaces,
// launches; the kernels are in ragged_kernel.cuh and ragged_dw.cuh.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <mutex>

#include "adapters_prep.cuh"
#include "gemm_relu.h"
#include "launch.h"
#include "ragged_dw.cuh"
#include "ragged_kernel.cuh"
#include "ragged_plan.h"
#include "runtime.h"

namespace gr {
namespace rg {

using rt::DeviceState;
using rt::StreamBuffers;
using rt::check_matrix;
using rt::dim_ok;
using rt::encode;
using rt::encode_rows;
using rt::launch;
using rt::misaligned;
using rt::test_hook;

// `count` dense row-major (rows x width) matrices, one after another, read as
// boxes of `box_rows` rows x 64 columns of one of them (4-D: two 64-column
// blocks per box).
static int encode_stack(CUtensorMap* map, const void* ptr, uint64_t width, uint64_t rows, uint64_t count,
                        uint32_t box_rows, bool four_d, bool bf16) {
    if (four_d) {
        const uint64_t dims[4] = {64, rows, width / 64, count}, strides[3] = {width, 64, rows * width};
        const uint32_t box[4] = {64, box_rows, 2, 1};
        return encode(map, ptr, 4, dims, strides, box, bf16);
    }
    const uint64_t dims[3] = {width, rows, count}, strides[2] = {width, rows * width};
    const uint32_t box[3] = {64, box_rows, 1};
    return encode(map, ptr, 3, dims, strides, box, bf16);
}

template <typename F>
static int allow_smem(DeviceState& d, int which, F fn) {
    if (d.rg_attr_set[which]) return GEMM_OK;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, rt::kMaxDynSmem) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    d.rg_attr_set[which] = true;
    return GEMM_OK;
}

template <typename F>
static int prefer_smem(DeviceState& d, int which, F fn) {
    if (d.rg_carveout_set[which]) return GEMM_OK;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) !=
        cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    d.rg_carveout_set[which] = true;
    return GEMM_OK;
}

static int zero_rows(void* y, int64_t ld, int64_t width, int64_t rows, cudaStream_t st) {
    if (cudaMemset2DAsync(y, (size_t)ld * 2, 0, (size_t)width * 2, (size_t)rows, st) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    return GEMM_OK;
}

struct Adapters {
    const void *A, *B;
    const int32_t* ids;
    const float* scale;
    int64_t R, rank;
};

// low for up to kLowRows rows, beside the main kernel.
static int run_low(const void* X, const Adapters& ad, uint16_t* low, int64_t T, int64_t K, int64_t ldx,
                   const RaggedPlan& pl, bool bf16, DeviceState& d, cudaStream_t st) {
    int rc;
    LowParams q;
    memset(&q, 0, sizeof(q));
    q.X = reinterpret_cast<const uint16_t*>(X);
    q.A = reinterpret_cast<const uint16_t*>(ad.A);
    q.ids = ad.ids;
    q.scale = ad.scale;
    q.low = low;
    q.ldx = ldx;
    q.T = (int32_t)T;
    q.K = (int32_t)K;
    q.R = (int32_t)ad.R;
    q.rank = (int32_t)ad.rank;
    q.rank_pad = pl.rank_pad;
    q.bf16 = bf16 ? 1 : 0;
    q.wide = K % 16 == 0 && ldx % 16 == 0 && !misaligned(X, 32) && !misaligned(ad.A, 32);
    q.err = d.d_err;
    // A block's adapters are shared by as many CTAs as it can have, or by two,
    // which take them in turn, where the row blocks are many (times with 2 / 16;
    // 4096 x 4096, 32 adapters of rank 64, another one from row to row: 64 rows 45
    // / 30 us, 128 56 / 42, 400 104 / 109, 512 104 / 116, 1000 147 / 160; 1024 x
    // 1024, 16 of rank 16: 300 rows 27 / 20, 700 25 / 25, 1000 25 / 28; twenty
    // requests in runs, 700 rows, 4096 x 4096: 44 / 51).
    q.slot_step = (int32_t)std::min<int64_t>({T <= 512 ? 16 : 2, T, ad.R});
    const int nt = std::min(pl.rank_box / 8, 2);
    q.passes = pl.rank_pad / (8 * nt);
    const int64_t jobs = (T + 15) / 16 * q.slot_step * q.passes;
    // few jobs share each reduction between the CTAs of a cluster (one CTA
    // per multiprocessor leaves room there for one of the main kernel)
    q.k_split = (int32_t)std::max<int64_t>(1, std::min<int64_t>({8, d.sm_count / jobs, (K + 255) / 256}));
    auto fn = nt == 2 ? adapters_low_kernel<2> : adapters_low_kernel<1>;
    // the main kernel joins this one on its multiprocessors: the same split
    // between shared memory and L1
    if ((rc = prefer_smem(d, nt - 1, fn)) != GEMM_OK) return rc;
    return launch(fn, (int)jobs * q.k_split, kLowWarps * 32, 0, q.k_split, st, q);
}

// Y[t] = epilogue(X[t] W[g(t)]): X (T, K), Y (T, N); W[g] (K, N), or (N, K)
// where w_kmajor.  offsets null: one W for all rows.
static int run_forward(const void* X, const void* W, void* Y, const int32_t* offsets, const void* act, int64_t T,
                       int64_t G, int64_t N, int64_t K, int64_t ldx, int64_t ldy, int64_t ld_act, bool relu,
                       bool w_kmajor, bool bf16, const Adapters* ad, cudaStream_t st, int dev) {
    DeviceState& d = rt::g_dev[dev];
    const RaggedPlan pl = plan_rows(T, G, N, K, ad ? ad->R : 0, ad ? ad->rank : 0, d.sm_count, d.max_pairs);
    if (pl.status != GEMM_OK) return pl.status;
    Maps m;
    memset(&m, 0, sizeof(m));
    Params p;
    memset(&p, 0, sizeof(p));
    p.T = (int32_t)T;
    p.G = (int32_t)G;
    p.N = (int32_t)N;
    p.K = (int32_t)K;
    p.num_kb = pl.num_kb;
    p.n_tiles = pl.n_tiles;
    p.cap = pl.cap;
    p.cluster = pl.cluster;
    p.num_stages = pl.num_stages;
    p.stage_bytes = pl.stage_bytes;
    p.turn_off = pl.num_stages * pl.stage_bytes;
    const int threads = pl.low_grid ? kHelped : row_threads(ad != nullptr);
    p.table_off = p.turn_off + (threads - 96) * (int)kTurnPitch;
    p.tmem_cols = (uint32_t)pl.tmem_cols;
    p.w_kmajor = w_kmajor ? 1 : 0;
    p.w4d = (w_kmajor ? K : N) % 64 == 0;
    p.x3d = K % 64 == 0;
    p.apply_relu = relu ? 1 : 0;
    p.bf16 = bf16 ? 1 : 0;
    p.offsets = offsets;
    p.Y = reinterpret_cast<uint16_t*>(Y);
    p.ldy = ldy;
    p.act = reinterpret_cast<const uint16_t*>(act);
    p.ld_act = ld_act;
    p.err = d.d_err;
    p.timeout_ns = 2000000000ull + 2000ull * (uint64_t)pl.num_kb;
    int rc = test_hook(!pl.pair && pl.cluster == 1 && !ad, pl.num_kb, &p.test_drop_kb, &p.timeout_ns);
    if (rc != GEMM_OK) return rc;
    // weights: K-major, 128 rows x 64 k; else 128 k-rows x 64 columns
    rc = w_kmajor ? encode_stack(&m.w, W, (uint64_t)K, (uint64_t)N, (uint64_t)G, 128, p.w4d, bf16)
                  : encode_stack(&m.w, W, (uint64_t)N, (uint64_t)K, (uint64_t)G, kBK, p.w4d, bf16);
    const int boxes = pl.cap / (pl.pair ? 2 : 1) / 16;
    for (int i = 0; rc == GEMM_OK && i < boxes; ++i)
        rc = encode_rows(&m.x[i], X, (uint64_t)K, (uint64_t)T, (uint64_t)ldx, 16u * (uint32_t)(i + 1),
                         p.x3d ? kBK / 64 : 0, bf16);
    if (rc != GEMM_OK) return rc;
    StreamBuffers& sb = rt::buffers_for_locked(d, st);
    if (ad) {
        p.ids = ad->ids;
        p.B = reinterpret_cast<const uint16_t*>(ad->B);
        p.row_tiles = pl.row_tiles;
        p.rank = (int32_t)ad->rank;
        p.R = (int32_t)ad->R;
        p.rank_box = pl.rank_box;
        p.rank_pad = pl.rank_pad;
        p.box_shift = pl.rank_box == 8 ? 3 : pl.rank_box == 16 ? 4 : pl.rank_box == 32 ? 5 : 6;
        p.per_slot = pl.rank_pad / pl.rank_box;
        p.b4d = N % 64 == 0;
        rc = encode_stack(&m.b, ad->B, (uint64_t)N, (uint64_t)ad->rank, (uint64_t)ad->R, (uint32_t)pl.rank_box, p.b4d,
                          bf16);
        if (rc != GEMM_OK) return rc;
        const int64_t tiles = pl.row_tiles;
        // one buffer: the low-rank rows, the tiles' slot lists, their lengths
        const size_t low_bytes = ((size_t)T * 2 * pl.rank_pad * 2 + 255) / 256 * 256;
        const size_t slot_bytes = (size_t)tiles * pl.cap * 4;
        rc = rt::grow(&sb.rg_misc, &sb.rg_misc_bytes, low_bytes + slot_bytes + (size_t)tiles * 4, st, false);
        if (rc != GEMM_OK) return rc;
        uint8_t* base = reinterpret_cast<uint8_t*>(sb.rg_misc);
        p.low = reinterpret_cast<const uint16_t*>(base);
        if (pl.pair) {
            SlotParams q;
            memset(&q, 0, sizeof(q));
            q.ids = ad->ids;
            q.slots = reinterpret_cast<int32_t*>(base + low_bytes);
            q.nslots = reinterpret_cast<int32_t*>(base + low_bytes + slot_bytes);
            q.T = (int32_t)T;
            q.R = (int32_t)ad->R;
            q.cap = pl.cap;
            q.tile_w = pl.row_width;
            q.err = d.d_err;
            rc = launch(adapters_slots_kernel, (int)tiles, 256, 0, 1, st, q);
            if (rc != GEMM_OK) return rc;
            p.slots = q.slots;
            p.nslots = q.nslots;
        }
        if (pl.low_grid) {
            const uint64_t dims[3] = {(uint64_t)K, (uint64_t)ad->rank, (uint64_t)ad->R};
            const uint64_t strides[2] = {(uint64_t)K, (uint64_t)(K * ad->rank)};
            const uint32_t box[3] = {64, (uint32_t)pl.rank_box, 1};
            rc = encode(&m.a, ad->A, 3, dims, strides, box, bf16);
            p.a4d = K % 64 == 0;
            if (rc == GEMM_OK && p.a4d)
                rc = encode_stack(&m.a4, ad->A, (uint64_t)K, (uint64_t)ad->rank, (uint64_t)ad->R,
                                  (uint32_t)pl.rank_box, true, bf16);
            if (rc != GEMM_OK) return rc;
            // the low-rank products as items of the same kernel, in a launch of their
            // own: tiles of Y wait for it as a whole, never for other CTAs of theirs
            p.low_out = reinterpret_cast<uint16_t*>(base);
            p.scale = ad->scale;
            if ((rc = allow_smem(d, 0, ragged_kernel<true, true>)) != GEMM_OK) return rc;
            rc = launch(ragged_kernel<true, true>, pl.low_grid, row_threads(true), (size_t)pl.smem_bytes, 2, st, m, p);
            if (rc != GEMM_OK) return rc;
            p.low_out = nullptr;
        } else {
            rc = run_low(X, *ad, reinterpret_cast<uint16_t*>(base), T, K, ldx, pl, bf16, d, st);
            if (rc != GEMM_OK) return rc;
        }
    }
    const size_t smem = (size_t)pl.smem_bytes;
    if (ad) {
        if (pl.pair) {
            if ((rc = allow_smem(d, 0, ragged_kernel<true, true>)) != GEMM_OK) return rc;
            return launch(ragged_kernel<true, true>, pl.grid, threads, smem, 2, st, m, p);
        }
        if ((rc = allow_smem(d, 1, ragged_kernel<false, true>)) != GEMM_OK) return rc;
        return launch(ragged_kernel<false, true>, pl.grid, row_threads(true), smem, pl.cluster, st, m, p);
    }
    if (pl.pair) {
        if ((rc = allow_smem(d, 2, ragged_kernel<true, false>)) != GEMM_OK) return rc;
        return launch(ragged_kernel<true, false>, pl.grid, row_threads(false), smem, 2, st, m, p);
    }
    if ((rc = allow_smem(d, 3, ragged_kernel<false, false>)) != GEMM_OK) return rc;
    return launch(ragged_kernel<false, false>, pl.grid, row_threads(false), smem, pl.cluster, st, m, p);
}

// D[g] (P, Q) = U[rows of g]^T V[rows of g]
static int run_dw(const void* U, const void* V, void* D, const int32_t* offsets, int64_t T, int64_t G, int64_t P,
                  int64_t Q, int64_t ldu, int64_t ldv, bool bf16, cudaStream_t st, int dev) {
    DeviceState& d = rt::g_dev[dev];
    const DwPlan pl = plan_dw(T, G, P, Q, d.sm_count, d.max_pairs);
    if (pl.status != GEMM_OK) return pl.status;
    DwPrepMaps base;
    DwMaps out;
    DwParams q;
    memset(&q, 0, sizeof(q));
    q.u3d = P % 64 == 0;
    q.v3d = Q % 64 == 0;
    q.timeout_ns = 2000000000ull + 2000ull * (uint64_t)((T + kBK - 1) / kBK);
    int rc = test_hook(!pl.pair && pl.cluster == 1, 1, &q.test_drop_kb, &q.timeout_ns);
    if (rc == GEMM_OK) rc = encode_rows(&base.u, U, (uint64_t)P, (uint64_t)T, (uint64_t)ldu, kBK, q.u3d ? 2 : 0, bf16);
    if (rc == GEMM_OK)
        rc = encode_rows(&base.v, V, (uint64_t)Q, (uint64_t)T, (uint64_t)ldv, kBK, q.v3d ? 2 : 0, bf16);
    if (rc == GEMM_OK) rc = encode_stack(&out.d, D, (uint64_t)Q, (uint64_t)P, (uint64_t)G, 32, false, bf16);
    if (rc != GEMM_OK) return rc;
    out.u = base.u;
    out.v = base.v;
    StreamBuffers& sb = rt::buffers_for_locked(d, st);
    const size_t map_bytes = (size_t)G * 2 * sizeof(CUtensorMap);
    rc = rt::grow(&sb.rg_misc, &sb.rg_misc_bytes, map_bytes + (size_t)G * sizeof(DwGroup), st, false);
    if (rc != GEMM_OK) return rc;
    CUtensorMap* maps = reinterpret_cast<CUtensorMap*>(sb.rg_misc);
    DwGroup* groups = reinterpret_cast<DwGroup*>(reinterpret_cast<uint8_t*>(sb.rg_misc) + map_bytes);
    rc = launch(dw_prep_kernel, (int)G, 32, 0, 1, st, base, offsets, (int32_t)G, (int32_t)T, groups, maps, d.d_err);
    if (rc != GEMM_OK) return rc;
    q.T = (int32_t)T;
    q.G = (int32_t)G;
    q.P = (int32_t)P;
    q.Q = (int32_t)Q;
    q.p_tiles = pl.p_tiles;
    q.q_tiles = pl.q_tiles;
    q.num_stages = pl.num_stages;
    q.bf16 = bf16 ? 1 : 0;
    q.cluster = pl.cluster;
    q.D = reinterpret_cast<uint16_t*>(D);
    q.groups = groups;
    q.maps = maps;
    q.err = d.d_err;
    if (pl.pair) {
        if ((rc = allow_smem(d, 4, ragged_dw_kernel<true>)) != GEMM_OK) return rc;
        return launch(ragged_dw_kernel<true>, pl.grid, kDwThreads, (size_t)pl.smem_bytes, 2, st, out, q);
    }
    if ((rc = allow_smem(d, 5, ragged_dw_kernel<false>)) != GEMM_OK) return rc;
    return launch(ragged_dw_kernel<false>, pl.grid, kDwThreads, (size_t)pl.smem_bytes, pl.cluster, st, out, q);
}

// ------------------------------------------------------------------ checks

// Grouped products: no row number of a call, nor a sum of one with a tile count
// or a tile's width, leaves 32 bits on the device.
static bool rows_ok(int64_t T) { return T <= GEMM_RELU_MAX_ROWS; }

static int check_common(int64_t T, int64_t G, int64_t N, int64_t K, int b_layout, int dtype) {
    if (!dim_ok(T) || !dim_ok(N) || !dim_ok(K) || G < 0 || G > GEMM_RELU_MAX_GROUPS) return GEMM_ERR_INVALID_ARG;
    if ((b_layout != GEMM_B_KN && b_layout != GEMM_B_NK) || (dtype != GEMM_DTYPE_F16 && dtype != GEMM_DTYPE_BF16))
        return GEMM_ERR_INVALID_ARG;
    if (N % 8 != 0 || K % 8 != 0) return GEMM_ERR_ALIGNMENT;
    return GEMM_OK;
}

static int check_offsets(const int32_t* offsets) {
    if (!offsets) return GEMM_ERR_INVALID_ARG;
    return misaligned(offsets, 4) ? GEMM_ERR_ALIGNMENT : GEMM_OK;
}

}  // namespace rg
}  // namespace gr

using namespace gr;
using namespace gr::rg;

extern "C" int gemm_relu_grouped(const void* X, const void* W, void* Y, const int32_t* offsets, int64_t T, int64_t G,
                                 int64_t N, int64_t K, int64_t ldx, int64_t ldy, int apply_relu, int b_layout,
                                 int dtype, void* stream) {
    int rc = check_common(T, G, N, K, b_layout, dtype);
    if (rc != GEMM_OK) return rc;
    if (!rows_ok(T)) return GEMM_ERR_INVALID_ARG;
    if (T == 0 || N == 0) return GEMM_OK;
    if ((rc = check_matrix(Y, N, ldy)) != GEMM_OK) return rc;
    const bool empty = G == 0 || K == 0;
    if (!empty) {
        if ((rc = check_matrix(X, K, ldx)) != GEMM_OK) return rc;
        if ((rc = check_matrix(W, 0, 0)) != GEMM_OK) return rc;
        if ((rc = check_offsets(offsets)) != GEMM_OK) return rc;
    }
    int dev;
    if ((rc = rt::current_device(&dev)) != GEMM_OK) return rc;
    std::lock_guard<std::mutex> lock(rt::g_mu);
    if ((rc = rt::init_device_locked(dev)) != GEMM_OK) return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (empty) return zero_rows(Y, ldy, N, T, st);
    return run_forward(X, W, Y, offsets, nullptr, T, G, N, K, ldx, ldy, 0, apply_relu != 0, b_layout == GEMM_B_NK,
                       dtype == GEMM_DTYPE_BF16, nullptr, st, dev);
}

extern "C" int gemm_relu_grouped_dx(const void* dY, const void* W, void* dX, const int32_t* offsets, const void* act,
                                    int64_t T, int64_t G, int64_t N, int64_t K, int64_t ld_dy, int64_t ld_dx,
                                    int64_t ld_act, int b_layout, int dtype, void* stream) {
    int rc = check_common(T, G, N, K, b_layout, dtype);
    if (rc != GEMM_OK) return rc;
    if (!rows_ok(T)) return GEMM_ERR_INVALID_ARG;
    if (T == 0 || K == 0) return GEMM_OK;
    if ((rc = check_matrix(dX, K, ld_dx)) != GEMM_OK) return rc;
    const bool empty = G == 0 || N == 0;
    if (!empty) {
        if ((rc = check_matrix(dY, N, ld_dy)) != GEMM_OK) return rc;
        if ((rc = check_matrix(W, 0, 0)) != GEMM_OK) return rc;
        if ((rc = check_offsets(offsets)) != GEMM_OK) return rc;
        if (act && (rc = check_matrix(act, K, ld_act)) != GEMM_OK) return rc;
    }
    int dev;
    if ((rc = rt::current_device(&dev)) != GEMM_OK) return rc;
    std::lock_guard<std::mutex> lock(rt::g_mu);
    if ((rc = rt::init_device_locked(dev)) != GEMM_OK) return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (empty) return zero_rows(dX, ld_dx, K, T, st);
    // the same product with the other dimension of W reduced: W (K, N) is
    // contiguous along N, the reduction
    return run_forward(dY, W, dX, offsets, act, T, G, K, N, ld_dy, ld_dx, ld_act, false, b_layout == GEMM_B_KN,
                       dtype == GEMM_DTYPE_BF16, nullptr, st, dev);
}

extern "C" int gemm_relu_grouped_dw(const void* X, const void* dY, void* dW, const int32_t* offsets, int64_t T,
                                    int64_t G, int64_t N, int64_t K, int64_t ldx, int64_t ld_dy, int b_layout,
                                    int dtype, void* stream) {
    int rc = check_common(T, G, N, K, b_layout, dtype);
    if (rc != GEMM_OK) return rc;
    if (!rows_ok(T)) return GEMM_ERR_INVALID_ARG;
    if (G == 0 || N == 0 || K == 0) return GEMM_OK;
    if ((rc = check_matrix(dW, 0, 0)) != GEMM_OK) return rc;
    if (T > 0) {
        if ((rc = check_matrix(X, K, ldx)) != GEMM_OK) return rc;
        if ((rc = check_matrix(dY, N, ld_dy)) != GEMM_OK) return rc;
        if ((rc = check_offsets(offsets)) != GEMM_OK) return rc;
    }
    int dev;
    if ((rc = rt::current_device(&dev)) != GEMM_OK) return rc;
    std::lock_guard<std::mutex> lock(rt::g_mu);
    if ((rc = rt::init_device_locked(dev)) != GEMM_OK) return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0) return zero_rows(dW, N * K, N * K, G, st);
    const bool bf16 = dtype == GEMM_DTYPE_BF16;
    return b_layout == GEMM_B_KN ? run_dw(X, dY, dW, offsets, T, G, K, N, ldx, ld_dy, bf16, st, dev)
                                 : run_dw(dY, X, dW, offsets, T, G, N, K, ld_dy, ldx, bf16, st, dev);
}

extern "C" int gemm_relu_adapters(const void* X, const void* W, const void* A, const void* B, const int32_t* ids,
                                  const float* scale, void* Y, int64_t T, int64_t N, int64_t K, int64_t R,
                                  int64_t rank, int64_t ldx, int64_t ldy, int apply_relu, int b_layout, int dtype,
                                  void* stream) {
    int rc = check_common(T, 1, N, K, b_layout, dtype);
    if (rc != GEMM_OK) return rc;
    if (!dim_ok(R) || R == 0 || rank < 1 || rank > GEMM_RELU_MAX_RANK) return GEMM_ERR_INVALID_ARG;
    if (T == 0 || N == 0) return GEMM_OK;
    if ((rc = check_matrix(Y, N, ldy)) != GEMM_OK) return rc;
    if (K > 0) {
        if ((rc = check_matrix(X, K, ldx)) != GEMM_OK) return rc;
        if ((rc = check_matrix(W, 0, 0)) != GEMM_OK) return rc;
        if ((rc = check_matrix(A, 0, 0)) != GEMM_OK) return rc;
        if ((rc = check_matrix(B, 0, 0)) != GEMM_OK) return rc;
        if (!ids) return GEMM_ERR_INVALID_ARG;
        if (misaligned(ids, 4) || misaligned(scale, 4)) return GEMM_ERR_ALIGNMENT;
    }
    int dev;
    if ((rc = rt::current_device(&dev)) != GEMM_OK) return rc;
    std::lock_guard<std::mutex> lock(rt::g_mu);
    if ((rc = rt::init_device_locked(dev)) != GEMM_OK) return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (K == 0) return zero_rows(Y, ldy, N, T, st);
    // (a launch lists its row tiles in shared memory: row blocks of what fits)
    const int64_t block = (int64_t)GEMM_RELU_MAX_GROUPS * 256;
    for (int64_t t = 0; t < T && rc == GEMM_OK; t += block) {
        const Adapters ad = {A, B, ids + t, scale, R, rank};
        rc = run_forward(reinterpret_cast<const uint16_t*>(X) + t * ldx, W, reinterpret_cast<uint16_t*>(Y) + t * ldy,
                         nullptr, nullptr, std::min(block, T - t), 1, N, K, ldx, ldy, 0, apply_relu != 0,
                         b_layout == GEMM_B_NK, dtype == GEMM_DTYPE_BF16, &ad, st, dev);
    }
    return rc;
}
