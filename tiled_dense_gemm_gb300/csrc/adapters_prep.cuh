// What the adapters' product needs beside its main kernel: the rows' low-rank
// parts and, where the rows need several tiles, the list of each tile's
// distinct adapters.
//
//   low[t, j] = scale[i] * sum_k X[t, k] A[i][j, k],   i = ids[t]
//
// The sums are taken in 32 bits, scaled there, and handed on as two numbers
// of the element type, hi = round(v) and lo = round(v - hi): together they
// hold v to 2^-16 (bfloat16) or 2^-22 (binary16), so the low-rank part loses
// nothing that the last rounding of Y would show.  The tensor cores multiply
// both with the same B, which costs them twice a product that is a few
// percent of the whole, and no memory traffic.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "ragged_kernel.cuh"

namespace gr {
namespace rg {

constexpr int kLowWarps = 8;
constexpr int64_t kLowRows = 1024;  // most rows of the kernel beside the main one

struct LowParams {
    const uint16_t* X;   // (T, K), pitch ldx
    const uint16_t* A;   // (R, rank, K)
    const int32_t* ids;  // (T)
    const float* scale;  // (R), or null: 1
    uint16_t* low;       // (T, 2, rank_pad): hi, lo
    int64_t ldx;
    int32_t T, K, R, rank, rank_pad, bf16;
    int32_t slot_step;   // CTAs that share a row block's adapters
    int32_t passes;      // CTAs that share a rank (8 * kNT products each)
    int32_t k_split;     // CTAs (a cluster) that share a reduction
    int32_t* err;
};

struct SlotParams {
    const int32_t* ids;
    int32_t* slots;      // [tile][cap]
    int32_t* nslots;     // [tile]
    int32_t T, R, cap, tile_w;
};

// One row tile's distinct adapters, in order of first appearance.  (Indexes
// outside [0, R) count as no adapter; low_kernel reports them.)
__global__ void __launch_bounds__(256) adapters_slots_kernel(const __grid_constant__ SlotParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    __shared__ int32_t id[256];
    __shared__ int32_t count[8];
    const int32_t i = (int32_t)threadIdx.x, warp = i / 32, lane = i % 32;
    const int32_t row0 = (int32_t)blockIdx.x * p.tile_w;
    const int32_t rows = min(p.tile_w, p.T - row0);
    int32_t mine = -1;
    if (i < rows) {
        mine = __ldcg(p.ids + row0 + i);
        if (mine < 0 || mine >= p.R) mine = -1;
    }
    id[i] = mine;
    __syncthreads();
    bool first = mine >= 0;
    for (int32_t j = 0; j < i; ++j) first = first && id[j] != mine;
    const uint32_t votes = __ballot_sync(0xffffffffu, first);
    if (lane == 0) count[warp] = __popc(votes);
    __syncthreads();
    int32_t at = __popc(votes & ((1u << lane) - 1u));
    for (int32_t w = 0; w < warp; ++w) at += count[w];
    if (first) p.slots[(int64_t)blockIdx.x * p.cap + at] = mine;
    if (i == 0) {
        int32_t n = 0;
        for (int32_t w = 0; w < 8; ++w) n += count[w];
        p.nslots[blockIdx.x] = n;
    }
}

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1, int32_t bf16) {
    if (bf16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
            " {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
            " {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// What rounding x to `hi` left out, rounded (nothing where hi is not finite).
__device__ __forceinline__ uint16_t rest16(float x, uint16_t hi, int32_t bf16) {
    const float back = bf16 ? __uint_as_float((uint32_t)hi << 16) : __half2float(__ushort_as_half(hi));
    return round16(isfinite(back) ? x - back : 0.0f, bf16);
}

__device__ __forceinline__ float ld_shared_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// 16 bytes from global memory, or zeros, without a branch.
__device__ __forceinline__ uint4 load_or_zero(const uint16_t* src, bool in) {
    uint4 q;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@p ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(q.x), "=&r"(q.y), "=&r"(q.z), "=&r"(q.w)
        : "l"(reinterpret_cast<uint64_t>(src)), "r"((uint32_t)in));
    return q;
}

// low for blocks of 16 rows: one adapter of the block and 8 kNT of its rank
// per job; the warps, and the CTAs of a cluster where jobs are few, split K.
//
// This product is a few percent of the main one's operations and all
// latency: it runs beside the main kernel (which starts while it runs and
// needs low only for its last k-blocks) in the registers and shared memory
// that kernel leaves, which rules out TMEM and a TMA ring; warp-level MMAs
// with operands straight from global memory fit.  The order of k inside an
// MMA does not matter as long as both operands agree, so each thread loads
// 16 contiguous bytes of its row and feeds two MMAs with them.
template <int kNT>
__global__ void __launch_bounds__(kLowWarps * 32, 2) adapters_low_kernel(const __grid_constant__ LowParams p) {
    __shared__ float part[kLowWarps / 2][kNT * 4 * 32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int32_t warp = (int32_t)threadIdx.x / 32, lane = (int32_t)threadIdx.x % 32;
    const int32_t g = lane >> 2, tig = lane & 3;
    const int32_t rank = p.k_split > 1 ? (int32_t)cluster_ctarank() : 0;
    const int32_t job = (int32_t)blockIdx.x / p.k_split;
    const int32_t j0 = job % p.passes * 8 * kNT;  // first of the rank's products
    const int32_t y = job / p.passes % p.slot_step, row0 = job / p.passes / p.slot_step * 16;
    // this warp's chunks of 32 k: kw0, kw0 + kw_step, ...
    const int32_t kw0 = (rank * kLowWarps + warp) * 32, kw_step = p.k_split * kLowWarps * 32;
    // the block's distinct adapters, in each warp's registers: lane = row
    int32_t mine = -1;
    if (lane < 16 && row0 + lane < p.T) {
        mine = __ldcg(p.ids + row0 + lane);
        if (mine < -1 || mine >= p.R) {
            atomicCAS(p.err + 1, 0, (int32_t)kBadIds);
            mine = -1;
        }
    }
    const uint32_t same = __match_any_sync(0xffffffffu, mine);
    uint32_t firsts = __ballot_sync(0xffffffffu, mine >= 0 && (same & ((1u << lane) - 1u)) == 0);
    for (int32_t s = 0; firsts; ++s) {
        const int32_t src = __ffs((int)firsts) - 1;
        firsts &= firsts - 1;
        if (s % p.slot_step != y) continue;
        const int32_t id = __shfl_sync(0xffffffffu, mine, src);
        float acc[kNT][4];
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[n][c] = 0.0f;
        // rows of other adapters are left out (their results are not kept)
        const bool in0 = __shfl_sync(0xffffffffu, mine, g) == id, in1 = __shfl_sync(0xffffffffu, mine, g + 8) == id;
        const uint16_t* x0 = p.X + (int64_t)(in0 ? row0 + g : row0) * p.ldx;
        const uint16_t* x1 = p.X + (int64_t)(in1 ? row0 + g + 8 : row0) * p.ldx;
        const uint16_t* a = p.A + ((int64_t)id * p.rank + j0 + g) * p.K;
        // kU chunks of 32 k per warp in flight at once: one round trip to
        // DRAM for each 256 x kU x k_split of K
        constexpr int kU = kNT == 8 ? 2 : kNT == 4 ? 4 : 6;
        for (int32_t kw = kw0; kw < p.K; kw += kw_step * kU) {
            uint4 xv[kU][2], av[kU][kNT];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int32_t k = kw + u * kw_step + tig * 8;
                const bool in = k < p.K;
                xv[u][0] = load_or_zero(x0 + k, in && in0);
                xv[u][1] = load_or_zero(x1 + k, in && in1);
#pragma unroll
                for (int n = 0; n < kNT; ++n)
                    av[u][n] = load_or_zero(a + (int64_t)n * 8 * p.K + k, in && j0 + n * 8 + g < p.rank);
            }
#pragma unroll
            for (int u = 0; u < kU; ++u)
#pragma unroll
                for (int n = 0; n < kNT; ++n) {
                    mma_16816(acc[n], xv[u][0].x, xv[u][1].x, xv[u][0].y, xv[u][1].y, av[u][n].x, av[u][n].y, p.bf16);
                    mma_16816(acc[n], xv[u][0].z, xv[u][1].z, xv[u][0].w, xv[u][1].w, av[u][n].z, av[u][n].w, p.bf16);
                }
        }
        const float scale = p.scale ? __ldcg(p.scale + id) : 1.0f;
        // sum over the warps: halves in turn, in a fixed order
#pragma unroll
        for (int half = kLowWarps / 2; half > 0; half /= 2) {
            __syncthreads();
            if (warp >= half && warp < 2 * half)
#pragma unroll
                for (int n = 0; n < kNT; ++n)
#pragma unroll
                    for (int c = 0; c < 4; ++c) part[warp - half][(n * 4 + c) * 32 + lane] = acc[n][c];
            __syncthreads();
            if (warp < half)
#pragma unroll
                for (int n = 0; n < kNT; ++n)
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[n][c] += part[warp][(n * 4 + c) * 32 + lane];
        }
        if (p.k_split > 1) {
            // the cluster's sums, in rank order, by its first CTA
            __syncthreads();
            if (warp == 0 && rank != 0)
#pragma unroll
                for (int n = 0; n < kNT; ++n)
#pragma unroll
                    for (int c = 0; c < 4; ++c) part[0][(n * 4 + c) * 32 + lane] = acc[n][c];
            cluster_sync();
            if (warp == 0 && rank == 0)
                for (int32_t r = 1; r < p.k_split; ++r) {
                    const uint32_t from = mapa_shared(smem_u32(&part[0][lane]), (uint32_t)r);
#pragma unroll
                    for (int n = 0; n < kNT; ++n)
#pragma unroll
                        for (int c = 0; c < 4; ++c) acc[n][c] += ld_shared_cluster(from + (n * 4 + c) * 128u);
                }
            cluster_sync();  // its reads are done
        }
        if (warp == 0 && rank == 0) {
#pragma unroll
            for (int n = 0; n < kNT; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (!(h ? in1 : in0)) continue;
                    const int32_t j = j0 + n * 8 + tig * 2;
                    uint32_t hi = 0, rest = 0;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        // columns past the rank are zeros whatever the scale is
                        const float v = j + c < p.rank ? acc[n][2 * h + c] * scale : 0.0f;
                        const uint16_t b = round16(v, p.bf16);
                        hi |= (uint32_t)b << (16 * c);
                        rest |= (uint32_t)rest16(v, b, p.bf16) << (16 * c);
                    }
                    uint16_t* dst = p.low + (int64_t)(row0 + 8 * h + g) * 2 * p.rank_pad + j;
                    *reinterpret_cast<uint32_t*>(dst) = hi;
                    *reinterpret_cast<uint32_t*>(dst + p.rank_pad) = rest;
                }
        }
    }
}

// ------------------------------------------------------------------ many rows

struct LowTileMaps {
    CUtensorMap x;  // rows: boxes of `cap` rows x 64 k (two of them where x3d)
    CUtensorMap a;  // first factors: boxes of rank_box rows x 64 k of one adapter
};

struct LowTileParams {
    const int32_t* ids;
    const float* scale;
    uint16_t* low;
    int32_t T, R, num_kb, cap, rank, rank_pad, rank_box, bf16, x3d, num_stages;
    uint32_t tmem_cols;
    int32_t* err;
    uint64_t timeout_ns;
};

// low for many rows, on the tensor cores: a block takes `cap` rows (16 to
// 128), and the ranks of its rows' distinct adapters side by side, 128 at a
// time, are the MMA's M side.  X is read once where the block has at most
// 128 ranks in all; each adapter's columns keep only its own rows' results.
__global__ void __launch_bounds__(kThreads, 1)
    adapters_low_tile_kernel(const __grid_constant__ LowTileMaps maps, const __grid_constant__ LowTileParams q) {
    extern __shared__ __align__(1024) uint8_t smem[];
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem);
    __shared__ int32_t slots[128], windows[128], row_id[128], count[4], nslots;
    const uint32_t ring = (smem_u32(smem) + (uint32_t)sizeof(Ctrl) + 1023u) & ~1023u;
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t stride = kWBytes + (uint32_t)q.cap * (kBK * 2);
    const int32_t row0 = (int32_t)blockIdx.x * q.cap;
    Params p;  // what wait_phase and list_slots read
    p.err = q.err;
    p.timeout_ns = q.timeout_ns;
    p.ids = q.ids + row0;
    p.T = min(q.cap, q.T - row0);
    p.R = q.R;
    if (warp == 6 && lane == 0) {
        for (int s = 0; s < q.num_stages; ++s) {
            mbar_init(smem_u32(&ctrl->full[s]), 1);
            mbar_init(smem_u32(&ctrl->empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&ctrl->tmem_full[b]), 1);
            mbar_init(smem_u32(&ctrl->tmem_empty[b]), kEpiThreads / 32);
        }
        mbar_init(smem_u32(&ctrl->final_bar), 1);
        ctrl->abort_flag = 0;
        ctrl->ring_s = ctrl->ring_ph = ctrl->ring_lap = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc<1>(smem_u32(&ctrl->tmem_addr), q.tmem_cols);
        tmem_relinquish<1>();
    }
    grid_dependency_wait();
    grid_launch_dependents();
    if (warp >= 2 && warp <= 5) {
        const int32_t i = (int32_t)threadIdx.x - 64;
        list_slots(p, row_id, slots, windows, count, &nslots, i);
    }
    __syncwarp();
    tc_fence_before();
    cta_barrier_sync();
    tc_fence_after();
    const uint32_t tmem_base = ctrl->tmem_addr;
    const uint32_t S = (uint32_t)q.num_stages, cols = q.tmem_cols / 2;
    const uint32_t full0 = smem_u32(&ctrl->full[0]), empty0 = smem_u32(&ctrl->empty[0]);
    const int32_t per = 128 / q.rank_box, per_slot = q.rank_pad / q.rank_box;
    const int32_t pieces = nslots * per_slot;
    const int32_t groups = (pieces + per - 1) / per;
    if (warp == 0 || warp == 6) {
        uint32_t s = 0, ph = 0;
        int32_t issued = 0;
        bool ok = true;
        for (int32_t m = 0; ok && m < groups; ++m) {
            const int32_t n = min(per, pieces - m * per);
            for (int32_t kb = 0; kb < q.num_kb; ++kb) {
                ok = wait_phase(empty0 + 8u * s, ph ^ 1u, ctrl, p, warp == 0 ? kErrTokens : kErrWeights);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const uint32_t full = full0 + 8u * s, dst = ring + s * stride;
                if (warp == 0) {
                    if (lane == 0) {
                        mbar_arrive_expect_tx(full, (uint32_t)(n * q.rank_box) * 256u + (uint32_t)q.cap * 256u);
                        ++issued;
                        if (q.x3d) {
                            load_3d<false>(dst + kWBytes, &maps.x, full, 0, row0, kb * (kBK / 64));
                        } else {
                            load_2d<false>(dst + kWBytes, &maps.x, full, kb * kBK, row0);
                            load_2d<false>(dst + kWBytes + (uint32_t)q.cap * 128u, &maps.x, full, kb * kBK + 64, row0);
                        }
                    }
                } else if ((int32_t)(lane >> 1) < n) {
                    const int32_t piece = m * per + (int32_t)(lane >> 1), slot = piece / per_slot;
                    load_3d<false>(dst + (lane & 1u) * (128u * 128u) + (lane >> 1) * (uint32_t)q.rank_box * 128u,
                                   &maps.a, full, kb * kBK + 64 * (int32_t)(lane & 1u),
                                   (piece - slot * per_slot) * q.rank_box, slots[slot]);
                }
                __syncwarp();
                if (++s == S) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        if (warp == 0 && lane == 0) {
            ctrl->ring_s = (int32_t)s;
            ctrl->ring_ph = (int32_t)ph;
            ctrl->ring_lap = issued >= (int32_t)S ? 1 : 0;
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = make_idesc_f16_f32(128, (uint32_t)q.cap, false, false, q.bf16 != 0);
            const uint64_t a_desc0 = make_sw128_desc(ring, 16, 1024);
            const uint64_t b_desc0 = make_sw128_desc(ring + kWBytes, 16, 1024);
            const uint32_t half16 = (uint32_t)q.cap * 128u >> 4;
            uint32_t s = 0, ph = 0;
            bool ok = true;
            for (int32_t m = 0; ok && m < groups; ++m) {
                const uint32_t buf = (uint32_t)m & 1u, bph = ((uint32_t)m >> 1) & 1u;
                if (!wait_phase(smem_u32(&ctrl->tmem_empty[buf]), bph ^ 1u, ctrl, p, kErrAccum)) break;
                tc_fence_after();
                for (int32_t kb = 0; kb < q.num_kb; ++kb) {
                    if (!wait_phase(full0 + 8u * s, ph, ctrl, p, kErrStage)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t a_desc = a_desc0 + (uint64_t)(s * (stride >> 4));
                    const uint64_t b_desc = b_desc0 + (uint64_t)(s * (stride >> 4));
#pragma unroll
                    for (uint32_t k = 0; k < kBK / 16; ++k)
                        mma_f16_ss<1>(tmem_base + buf * cols, a_desc + (k / 4) * (128u * 128u >> 4) + (k % 4) * 2u,
                                      b_desc + (k / 4) * half16 + (k % 4) * 2u, idesc, (kb | (int32_t)k) > 0 ? 1u : 0u);
                    mma_commit<1>(empty0 + 8u * s);
                    if (++s == S) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (ok) mma_commit<1>(smem_u32(&ctrl->tmem_full[buf]));
            }
            mma_commit<1>(smem_u32(&ctrl->final_bar));
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(smem_u32(&ctrl->final_bar), 0))
                if (globaltimer_ns() - t0 > q.timeout_ns) {
                    atomicCAS(q.err, 0, (int32_t)kErrFinal);
                    break;
                }
        }
        __syncwarp();
    } else {
        const uint32_t quarter = warp & 3u;
        float v[32];
        for (int32_t m = 0; m < groups; ++m) {
            const uint32_t buf = (uint32_t)m & 1u, bph = ((uint32_t)m >> 1) & 1u;
            bool ok = wait_phase(smem_u32(&ctrl->tmem_full[buf]), bph, ctrl, p, kErrEpi);
            ok = named_bar_and(kEpiBarrier, kEpiThreads, ok);
            if (!ok) break;
            tc_fence_after();
            // this lane's product: number j of its adapter's rank
            const int32_t r = (int32_t)(quarter * 32 + lane);
            const int32_t piece = m * per + r / q.rank_box, slot = piece / per_slot;
            const int32_t j = (piece - slot * per_slot) * q.rank_box + r % q.rank_box;
            const int32_t id = piece < pieces ? slots[slot] : -2;
            const float scale = id >= 0 && q.scale ? __ldcg(q.scale + id) : 1.0f;
            for (int32_t c = 0; c < q.cap; c += 32) {
                __syncwarp();
                tmem_load_32cols(tmem_base + ((quarter * 32u) << 16) + buf * cols + (uint32_t)c, v);
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    if (c + i < p.T && row_id[c + i] == id) {
                        // columns past the rank are zeros whatever the scale is
                        const float x = j < q.rank ? v[i] * scale : 0.0f;
                        const uint16_t hi = round16(x, q.bf16);
                        uint16_t* dst = q.low + (int64_t)(row0 + c + i) * 2 * q.rank_pad + j;
                        dst[0] = hi;
                        dst[q.rank_pad] = rest16(x, hi, q.bf16);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ctrl->tmem_empty[buf]));
        }
    }
    __syncthreads();
    if (threadIdx.x == 0 && *(volatile int32_t*)&ctrl->abort_flag) drain_ring(ctrl, full0, S);
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<1>(tmem_base, q.tmem_cols);
    }
}

}  // namespace rg
}  // namespace gr
