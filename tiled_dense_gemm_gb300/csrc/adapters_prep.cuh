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
    uint32_t* low_done;  // [tile], set to zero
    int32_t T, R, cap, tile_w;
    int32_t* err;
};

// One row tile's distinct adapters, in order of first appearance.
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
        if (mine < -1 || mine >= p.R) {
            atomicCAS(p.err + 1, 0, (int32_t)kBadIds);
            mine = -1;
        }
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
        p.low_done[blockIdx.x] = 0u;
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
//
// Bound: DRAM, which it shares with the main kernel's weights.  64 rows with
// 48 adapters of rank 32, 8192 x 8192: its 25 MB are in 32-38 us after the
// start, with the main kernel's 134 MB beside them.  Asking for both
// factors in L2 first (this one here, the second in the main kernel) keeps
// them from queueing behind the weights (16 rows with 16 adapters: 43 us for
// the whole call without, 37 with).
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
    // kU chunks of 32 k per warp in flight at once, side by side: one round
    // trip to DRAM for each 256 x kU x k_split of K
    constexpr int kU = kNT == 8 ? 2 : kNT == 4 ? 4 : 6;
    const int32_t kw0 = (rank * kLowWarps + warp) * (32 * kU), kw_step = p.k_split * kLowWarps * (32 * kU);
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
        // all of it to L2 first, ahead of the main kernel's copies
        for (int32_t i = (int32_t)threadIdx.x; i < kNT * 8 * ((p.K + 63) / 64); i += kLowWarps * 32) {
            const int32_t chunk = i / (kNT * 8), row = i % (kNT * 8), k = chunk * 64;
            // (chunks of 64 k that this CTA of the cluster reads)
            if (k / (kLowWarps * 32 * kU) % p.k_split == rank && j0 + row < p.rank)
                prefetch_line(p.A + ((int64_t)id * p.rank + j0 + row) * p.K + k);
        }
        for (int32_t kw = kw0; kw < p.K; kw += kw_step) {
            uint4 xv[kU][2], av[kU][kNT];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int32_t k = kw + u * 32 + tig * 8;
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
                    // columns past the rank are zeros whatever the scale is
                    const float v0 = j < p.rank ? acc[n][2 * h] * scale : 0.0f;
                    const float v1 = j + 1 < p.rank ? acc[n][2 * h + 1] * scale : 0.0f;
                    const uint32_t hi = pack16(v0, v1, p.bf16);
                    uint16_t* dst = p.low + (int64_t)(row0 + 8 * h + g) * 2 * p.rank_pad + j;
                    *reinterpret_cast<uint32_t*>(dst) = hi;
                    *reinterpret_cast<uint32_t*>(dst + p.rank_pad) = rest16x2(v0, v1, hi, p.bf16);
                }
        }
    }
}

}  // namespace rg
}  // namespace gr
