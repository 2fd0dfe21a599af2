// Weight gradients of ragged groups, for sm_103a:
//
//   D[g] (P x Q) = U[rows of g, :]^T V[rows of g, :]
//
// a product whose reduction runs over the rows of group g, so its length is
// known on the device only.  Both operands are read as stored (rows of P or
// Q contiguous elements): MN-major for the tensor core, no transposition.
//
// A group may end anywhere inside a 128-row block.  The rows after it belong
// to another group and must not enter the sum, whatever they hold (0 x NaN is
// NaN), so a group's last block is read through its own pair of tensor maps
// whose row extent ends with the group: the copies fill the rows beyond with
// zeros and fetch nothing for them.  (Whole blocks go through the maps of the
// whole operands: a map's first use costs its fetch.)  A small kernel before
// this one makes the maps from the host's by setting that one extent (one warp
// per group), and orders the groups by length, longest first, so that the last
// items of the persistent grid are short ones.
//
// Tile 128 x 128 per CTA, or 256 x 256 per CTA pair; stages of 128 rows; roles
// and waits as in the ragged forward kernel, but eight epilogue warps (2-5 and
// 7-10, each half of a quarter's columns): a group's reduction is often only a
// few stages long, and with four warps writing a tile took longer than
// computing it (32 groups of 512 rows on average, gradients of 2048 x 4096:
// 239 us with four, 216 with eight; 199 with the accumulator released before
// the stores behind it are visible).
//
// Few tiles of long groups are computed by clusters, whose CTAs take shares of
// the group's blocks and add them up through distributed shared memory, in
// their order.
//
// Bound.  Sums are in 32 bits, rounded once.  At the tensor rate a CTA of a
// pair takes in 64 bytes per clock, close to what copies reach, and a tile's
// start and end hide only behind its neighbours' four blocks: that case runs
// at 1390 TFLOP/s (198 us; stages of 64 rows: 202).  With 1000 rows in 24
// groups (gradients of 1032 x 520) two launches and a clipped block per tile
// are nearly all there is: 15 us.
#pragma once

#include "ragged_kernel.cuh"

namespace gr {
namespace rg {

struct DwGroup {
    int32_t g, lo, hi, pad;
};

struct DwMaps {
    CUtensorMap d;     // the gradients, 3-D
    CUtensorMap u, v;  // the operands
};

struct DwParams {
    int32_t T, G, P, Q;
    int32_t p_tiles, q_tiles;
    int32_t num_stages;
    int32_t u3d, v3d;     // one copy per stage of the operand's two 64-column chunks
    int32_t bf16;
    int32_t cluster;      // single CTAs: > 1: the CTAs of a cluster share each tile's rows
    uint16_t* D;
    const DwGroup* groups;      // by length, longest first
    const CUtensorMap* maps;    // [2 * position]: U's and V's of that group
    int32_t* err;
    uint64_t timeout_ns;
    int32_t test_drop_kb;  // as of the forward kernel: a block of U's rows
};

struct DwPrepMaps {
    CUtensorMap u, v;
};

// One warp per group g: its position by length, its bounds, its two maps.
__global__ void __launch_bounds__(32) dw_prep_kernel(const __grid_constant__ DwPrepMaps base, const int32_t* offsets,
                                                     int32_t G, int32_t T, DwGroup* groups, CUtensorMap* maps,
                                                     int32_t* err) {
    __shared__ __align__(128) CUtensorMap edit[2];
    const int32_t g = (int32_t)blockIdx.x, lane = (int32_t)threadIdx.x;
    grid_dependency_wait();
    grid_launch_dependents();
    // clamped to [0, T] and to be non-decreasing, as the forward kernel reads them
    const int32_t a = __ldcg(offsets + g), b = __ldcg(offsets + g + 1);
    const int32_t mine = min(max(b, 0), T) - min(max(a, 0), T);
    int32_t before = 0, lo = 0;
    for (int32_t j = lane; j < G; j += 32) {
        const int32_t x = min(max(__ldcg(offsets + j), 0), T), y = min(max(__ldcg(offsets + j + 1), 0), T);
        const int32_t len = y - x;
        before += (len > mine || (len == mine && j < g)) ? 1 : 0;
        if (j <= g) lo = max(lo, x);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, d);
        lo = max(lo, __shfl_xor_sync(0xffffffffu, lo, d));
    }
    const int32_t hi = max(lo, min(max(b, 0), T));
    if (lane == 0) {
        if (a != min(max(a, 0), T) || b != min(max(b, 0), T) || b < a) atomicCAS(err + 1, 0, (int32_t)kBadOffsets);
        DwGroup o;
        o.g = g;
        o.lo = lo;
        o.hi = hi;
        o.pad = 0;
        groups[before] = o;
    }
    reinterpret_cast<uint32_t*>(&edit[0])[lane] = reinterpret_cast<const uint32_t*>(&base.u)[lane];
    reinterpret_cast<uint32_t*>(&edit[1])[lane] = reinterpret_cast<const uint32_t*>(&base.v)[lane];
    __syncwarp();
    if (lane == 0 && hi > lo) {
        map_set_rows(smem_u32(&edit[0]), (uint32_t)hi);
        map_set_rows(smem_u32(&edit[1]), (uint32_t)hi);
    }
    __syncwarp();
    map_publish(maps + 2 * before, smem_u32(&edit[0]));
    map_publish(maps + 2 * before + 1, smem_u32(&edit[1]));
}

constexpr int kDwThreads = 352;

template <bool kPair>
__global__ void __launch_bounds__(kDwThreads, 1)
    ragged_dw_kernel(const __grid_constant__ DwMaps out, const __grid_constant__ DwParams q) {
    constexpr int kCG = kPair ? 2 : 1;
    constexpr uint32_t kTile = kPair ? 256 : 128;  // rows and columns of D per tile
    constexpr uint32_t kCols = kTile;              // TMEM columns per accumulator
    constexpr uint32_t kOperand = 128 * kBK * 2;   // bytes per operand, stage and CTA
    constexpr uint32_t stride = 2 * kOperand;
    extern __shared__ __align__(1024) uint8_t smem[];
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem);
    const uint32_t ring = (smem_u32(smem) + (uint32_t)sizeof(Ctrl) + 1023u) & ~1023u;
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = kPair ? cluster_ctarank() : 0u;
    const bool clustered = !kPair && q.cluster > 1;  // (one item per cluster)
    const uint32_t share = clustered ? cluster_ctarank() : 0u;
    const uint32_t worker = kPair ? blockIdx.x / 2 : blockIdx.x / (uint32_t)q.cluster;
    const uint32_t workers = kPair ? gridDim.x / 2 : gridDim.x / (uint32_t)q.cluster;
    Params w;  // what wait_phase reads
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
        ctrl->abort_flag = 0;
        ctrl->ring_s = ctrl->ring_ph = ctrl->ring_lap = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc<kCG>(smem_u32(&ctrl->tmem_addr), 2 * kCols);
        tmem_relinquish<kCG>();
    }
    __syncwarp();
    tc_fence_before();
    if (kPair)
        cluster_sync();
    else
        cta_barrier_sync();
    tc_fence_after();
    grid_launch_dependents();
    grid_dependency_wait();
    const uint32_t tmem_base = ctrl->tmem_addr;
    const uint32_t S = (uint32_t)q.num_stages;
    const uint32_t full0 = smem_u32(&ctrl->full[0]), empty0 = smem_u32(&ctrl->empty[0]);
    const uint32_t per_group = (uint32_t)(q.p_tiles * q.q_tiles);
    const uint32_t items = (uint32_t)q.G * per_group;

    // item -> position in the length order, tile; groups without a row have
    // no k-block.  The next item's group is on its way while this one runs.
    struct Work {
        int32_t pos, g, lo, hi, pt, qt;
    };
    uint32_t item = worker;
    int4 ahead = make_int4(0, 0, 0, 0);
    auto look = [&]() {
        if (item < items) ahead = __ldcg(reinterpret_cast<const int4*>(q.groups + item / per_group));
    };
    look();
    auto next = [&](Work& k) {
        if (item >= items) return false;
        k.pos = (int32_t)(item / per_group);
        const uint32_t l = item - (uint32_t)k.pos * per_group;
        k.qt = (int32_t)(l / (uint32_t)q.p_tiles);
        k.pt = (int32_t)(l - (uint32_t)k.qt * (uint32_t)q.p_tiles);
        k.g = ahead.x;
        k.lo = ahead.y;
        k.hi = ahead.z;
        if (clustered) {
            // an even share of the group's blocks
            const int32_t blocks = (k.hi - k.lo + kBK - 1) / kBK, c = q.cluster, lo = k.lo;
            k.lo = lo + (int32_t)share * blocks / c * kBK;
            k.hi = min(k.hi, lo + ((int32_t)share + 1) * blocks / c * kBK);
        }
        item += workers;
        look();
        return true;
    };
    Work k;

    if (warp == 0 || warp == 6) {
        // warp 0 copies U's tiles and arms the stages, warp 6 V's
        if (lane == 0) {
            const bool is_u = warp == 0;
            uint32_t s = 0, ph = 0;
            int32_t issued = 0, seen = -1;
            bool ok = true;
            while (ok && next(k)) {
                if (k.hi == k.lo) continue;
                const CUtensorMap* const last = q.maps + 2 * k.pos + (is_u ? 0 : 1);
                if (k.pos != seen && (k.hi - k.lo) % kBK != 0) {
                    map_acquire(last);
                    tma_prefetch_desc(last);
                }
                seen = k.pos;
                const int32_t c0 = (is_u ? k.pt : k.qt) * (int32_t)kTile + 128 * (int32_t)rank;
                for (int32_t r = k.lo; r < k.hi; r += kBK) {
                    if (!wait_phase(empty0 + 8u * s, ph ^ 1u, ctrl, w, is_u ? kErrTokens : kErrWeights)) {
                        ok = false;
                        break;
                    }
                    const uint32_t full = full0 + 8u * s;
                    if (is_u) {
                        if (!kPair || rank == 0) mbar_arrive_expect_tx(full, (kPair ? 2u : 1u) * stride);
                        ++issued;
                    }
                    const uint32_t bar = kPair ? mapa_shared(full, 0) : full;
                    const uint32_t dst = ring + s * stride + (is_u ? 0u : kOperand);
                    const CUtensorMap* const m = k.hi - r < kBK ? last : is_u ? &out.u : &out.v;
                    if (!kPair && is_u && issued == q.test_drop_kb && q.test_drop_kb > 0) {
                        // (test hook: not copied)
                    } else if (is_u ? q.u3d : q.v3d) {
                        load_3d<kPair>(dst, m, bar, 0, r, c0 / 64);
                    } else {
                        load_2d<kPair>(dst, m, bar, c0, r);
                        load_2d<kPair>(dst + (uint32_t)kBK * 128u, m, bar, c0 + 64, r);
                    }
                    if (++s == S) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (is_u && (!kPair || rank == 0)) {
                ctrl->ring_s = (int32_t)s;
                ctrl->ring_ph = (int32_t)ph;
                ctrl->ring_lap = issued >= (int32_t)S ? 1 : 0;
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0 && (!kPair || rank == 0)) {
            const uint32_t tfull0 = smem_u32(&ctrl->tmem_full[0]), tempty0 = smem_u32(&ctrl->tmem_empty[0]);
            const uint32_t idesc = make_idesc_f16_f32(kTile, kTile, true, true, q.bf16 != 0);
            const uint64_t a_desc0 = make_sw128_desc(ring, (uint32_t)kBK * 128u, 1024);
            const uint64_t b_desc0 = make_sw128_desc(ring + kOperand, (uint32_t)kBK * 128u, 1024);
            uint32_t s = 0, ph = 0, local = 0;
            bool ok = true;
            while (ok && next(k)) {
                if (k.hi == k.lo) continue;
                const uint32_t buf = local & 1u, bph = (local >> 1) & 1u;
                if (!wait_phase(tempty0 + 8u * buf, bph ^ 1u, ctrl, w, kErrAccum)) break;
                tc_fence_after();
                const uint32_t d = tmem_base + buf * kCols;
                uint32_t acc = 0;
                for (int32_t r = k.lo; r < k.hi; r += kBK) {
                    if (!wait_phase(full0 + 8u * s, ph, ctrl, w, kErrStage)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t a_desc = a_desc0 + (uint64_t)(s * (stride >> 4));
                    const uint64_t b_desc = b_desc0 + (uint64_t)(s * (stride >> 4));
                    if (k.hi - r >= kBK) {
#pragma unroll
                        for (uint32_t i = 0; i < kBK / 16; ++i)
                            mma_f16_ss<kCG>(d, a_desc + i * 128u, b_desc + i * 128u, idesc, i > 0 ? 1u : acc);
                    } else {
                        const uint32_t steps = (uint32_t)(k.hi - r + 15) / 16;  // the rest of the block is zeros
                        for (uint32_t i = 0; i < steps; ++i)
                            mma_f16_ss<kCG>(d, a_desc + i * 128u, b_desc + i * 128u, idesc, i > 0 ? 1u : acc);
                    }
                    acc = 1;
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
            mma_commit<kCG>(smem_u32(&ctrl->final_bar), 0x1);
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(smem_u32(&ctrl->final_bar), 0))
                if (globaltimer_ns() - t0 > q.timeout_ns) {
                    atomicCAS(q.err, 0, (int32_t)kErrFinal);
                    break;
                }
        }
        __syncwarp();
    } else {
        const uint32_t quarter = warp & 3u, half = warp >= 7 ? 1u : 0u;
        const uint32_t staging = ring + S * stride + (quarter + 4u * half) * 4096u;
        uint32_t local = 0;
        if (clustered && next(k)) {
            // this CTA's share in 32 bits into its ring (idle by now), column
            // by column; the cluster adds the shares up below
            const bool some = k.hi > k.lo;
            float v[64];
#pragma unroll
            for (int j = 0; j < 64; ++j) v[j] = 0.0f;
            if (some && __all_sync(0xffffffffu, wait_phase(smem_u32(&ctrl->tmem_full[0]), 0, ctrl, w, kErrEpi))) {
                tc_fence_after();
                tmem_load_64cols(tmem_base + ((quarter * 32u) << 16) + 64u * half, v);
                tc_fence_before();
            }
#pragma unroll
            for (int j = 0; j < 64; ++j)
                st_shared_f32(ring + ((64u * half + (uint32_t)j) * 128u + 32u * quarter + lane) * 4u, v[j]);
        }
        while (!clustered && next(k)) {
            const bool some = k.hi > k.lo;
            const uint32_t buf = local & 1u, bph = (local >> 1) & 1u;
            if (some) {
                if (!__all_sync(0xffffffffu, wait_phase(smem_u32(&ctrl->tmem_full[buf]), bph, ctrl, w, kErrEpi))) break;
                tc_fence_after();
            }
            const uint32_t taddr = tmem_base + ((quarter * 32u) << 16) + buf * kCols;
            const int32_t row0 = k.pt * (int32_t)kTile + 128 * (int32_t)rank + 32 * (int32_t)quarter;
            for (uint32_t c = half * (kCols / 2); c < (half + 1u) * (kCols / 2); c += 64) {
                const int32_t col = k.qt * (int32_t)kTile + (int32_t)c;
                if (col >= q.Q || row0 >= q.P) break;  // (uniform over the warp)
                uint32_t x[32];
                if (some) {
                    float v[64];
                    __syncwarp();
                    tmem_load_64cols(taddr + c, v);
#pragma unroll
                    for (int j = 0; j < 32; ++j) x[j] = pack16(v[2 * j], v[2 * j + 1], q.bf16);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) x[j] = 0u;
                }
                // the copy issued from this buffer before must have read it
                if (lane == 0) bulk_wait_group_read<0>();
                __syncwarp();
#pragma unroll
                for (uint32_t u = 0; u < 8; ++u)
                    st_shared_v4(staging + lane * 128u + ((u ^ (lane & 7u)) << 4),
                                 make_uint4(x[4 * u], x[4 * u + 1], x[4 * u + 2], x[4 * u + 3]));
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    store_3d(&out.d, staging, col, row0, k.g);
                    bulk_commit_group();
                }
            }
            if (some) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (kPair)
                        mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&ctrl->tmem_empty[buf]), 0));
                    else
                        mbar_arrive(smem_u32(&ctrl->tmem_empty[buf]));
                }
                ++local;
            }
        }
        if (lane == 0) bulk_wait_group_all();
        __syncwarp();
    }

    if (clustered) {
        // sums of the shares, in their order: a warp for 32 rows x 16 columns
        __syncwarp();
        cluster_sync();
        item = worker;
        look();
        if (warp >= 2 && warp != 6 && next(k)) {
            for (uint32_t task = share * 8u + (warp < 6 ? warp - 2u : warp - 3u); task < 32u; task += 8u * (uint32_t)q.cluster) {
                const uint32_t at = 32u * (task & 3u) + lane, c0 = 16u * (task >> 2);
                float x[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = 0.0f;
                for (uint32_t r = 0; r < (uint32_t)q.cluster; ++r) {
                    const uint32_t from = mapa_shared(ring + (c0 * 128u + at) * 4u, r);
#pragma unroll
                    for (int j = 0; j < 16; ++j) x[j] += ld_shared_cluster(from + (uint32_t)j * 512u);
                }
                const int32_t row = k.pt * (int32_t)kTile + (int32_t)at, col = k.qt * (int32_t)kTile + (int32_t)c0;
                uint16_t* const d = q.D + ((int64_t)k.g * q.P + row) * q.Q + col;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (row < q.P && col + 8 * h < q.Q)
                        *reinterpret_cast<uint4*>(d + 8 * h) =
                            make_uint4(pack16(x[8 * h], x[8 * h + 1], q.bf16), pack16(x[8 * h + 2], x[8 * h + 3], q.bf16),
                                       pack16(x[8 * h + 4], x[8 * h + 5], q.bf16),
                                       pack16(x[8 * h + 6], x[8 * h + 7], q.bf16));
            }
        }
    }
    __syncthreads();
    if (threadIdx.x == 0 && *(volatile int32_t*)&ctrl->abort_flag) drain_ring(ctrl, full0, S);
    tc_fence_before();
    if (kPair || clustered)
        cluster_sync_relaxed();  // the other CTAs' accesses to this one's shared memory are done
    else
        __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<kCG>(tmem_base, 2 * kCols);
    }
}

}  // namespace rg
}  // namespace gr
