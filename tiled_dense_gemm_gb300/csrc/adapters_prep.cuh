// What the adapters' product needs beside its main kernel: the rows' low-rank
// parts and, where the rows need several tiles, the list of each tile's
// distinct adapters.
//
//   low[t, j] = scale[i] * sum_k X[t, k] A[i][j, k],   i = ids[t]
//
// The sums are taken in 32 bits, scaled there, and handed on as two numbers
// of the element type, hi = round(v) and lo = round(v - hi): together they
// hold v to 2^-16 |v| (bfloat16), or to 2^-22 |v| or 2^-25, whichever is larger
// (binary16, whose smallest step is 2^-24 and whose values end at 65504).  For
// values of ordinary size the low-rank part so loses nothing that the last
// rounding of Y would show; small ones lose in binary16 (2^-14: 2^-11 of it),
// since the scale is in v.  The tensor cores multiply
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
    int32_t wide;        // rows of X and A start on 32 bytes
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
    int32_t* err;
};

// One row tile's distinct adapters, in order of first appearance.
__global__ void __launch_bounds__(256) adapters_slots_kernel(const __grid_constant__ SlotParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    __shared__ __align__(16) int32_t id[256];
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
    // the first of its own warp, and in none of the warps before
    const uint32_t same = __match_any_sync(0xffffffffu, mine);
    bool first = mine >= 0 && (same & ((1u << lane) - 1u)) == 0;
#pragma unroll 8
    for (int32_t j = 0; j < 8 * warp; ++j) {
        const int4 q = reinterpret_cast<const int4*>(id)[j];
        first = first & (q.x != mine) & (q.y != mine) & (q.z != mine) & (q.w != mine);
    }
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

// 32 bytes from global memory: in one load where addresses allow it (a whole
// line for the four lanes of a row: half the requests), else in two.
__device__ __forceinline__ void load_32(uint4 (&q)[2], const uint16_t* src, bool wide) {
    if (wide)
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(q[0].x), "=r"(q[0].y), "=r"(q[0].z), "=r"(q[0].w), "=r"(q[1].x), "=r"(q[1].y),
                       "=r"(q[1].z), "=r"(q[1].w)
                     : "l"(reinterpret_cast<uint64_t>(src)));
    else
        asm volatile(
            "ld.global.v4.b32 {%0, %1, %2, %3}, [%8];\n\t"
            "ld.global.v4.b32 {%4, %5, %6, %7}, [%8 + 16];"
            : "=&r"(q[0].x), "=&r"(q[0].y), "=&r"(q[0].z), "=&r"(q[0].w), "=&r"(q[1].x), "=&r"(q[1].y),
              "=&r"(q[1].z), "=&r"(q[1].w)
            : "l"(reinterpret_cast<uint64_t>(src)));
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
// 32 contiguous bytes of its row and feeds four MMAs with them.
//
// Bound: DRAM, which it shares with the main kernel's weights.  64 rows with
// 48 adapters of rank 32, 8192 x 8192: its 25 MB are in and multiplied 23 us
// after the main kernel's start, with that one's 134 MB beside them.  Asking for both
// factors in L2 first (this one here, the second in the main kernel) keeps
// them from queueing behind the weights (16 rows with 16 adapters, the whole
// call: 43 us without, 37 with; 32 with whole lines per load as well).
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
    // K in chunks of 64 (a line of each row), in turn with the other warps
    // (and CTAs of the cluster).  kD of them are in flight while one is
    // multiplied: what 128 registers hold without spilling, and with more a
    // CTA of the main kernel no longer fits beside (64 rows, 48 adapters of
    // rank 32, the whole call: 16 products per pass with two chunks 56 us, 32
    // with two 59, with 136 registers 61).
    constexpr int kD = kNT == 2 ? 2 : 4;
    const uint32_t part_of = (uint32_t)(rank * kLowWarps + warp), parts = (uint32_t)(p.k_split * kLowWarps);
    const uint32_t K = (uint32_t)p.K, whole = K / 64;
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
        const float scale = p.scale ? __ldcg(p.scale + id) : 1.0f;
        // Every product of the MMAs that is kept has its own row of X and its
        // own row of A; the others (rows of other adapters, past the rank)
        // read some row that exists and go nowhere.
        const uint32_t his = __ballot_sync(0xffffffffu, lane < 16 && mine == id);
        const uint16_t* const x0 = p.X + (int64_t)(row0 + ((his >> g) & 1u ? g : src)) * p.ldx + tig * 16;
        const uint16_t* const x1 = p.X + (int64_t)(row0 + ((his >> (g + 8)) & 1u ? g + 8 : src)) * p.ldx + tig * 16;
        const uint16_t* const a0 = p.A + (int64_t)id * p.rank * p.K + tig * 16;
        auto a_row = [&](int n) { return a0 + (uint64_t)(uint32_t)min(j0 + n * 8 + g, p.rank - 1) * K; };
        uint4 xv[kD][2][2], av[kD][kNT][2];
        float acc[kNT][4];
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[n][c] = 0.0f;
        auto load = [&](int d, uint32_t c) {
#pragma unroll
            for (int n = 0; n < kNT; ++n) load_32(av[d][n], a_row(n) + 64ull * c, p.wide);
            load_32(xv[d][0], x0 + 64ull * c, p.wide);
            load_32(xv[d][1], x1 + 64ull * c, p.wide);
        };
        auto multiply = [&](int d) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int n = 0; n < kNT; ++n) {
                    const uint4 &xa = xv[d][0][h], &xb = xv[d][1][h], &w = av[d][n][h];
                    mma_16816(acc[n], xa.x, xb.x, xa.y, xb.y, w.x, w.y, p.bf16);
                    mma_16816(acc[n], xa.z, xb.z, xa.w, xb.w, w.z, w.w, p.bf16);
                }
        };
#pragma unroll
        for (int d = 0; d < kD; ++d)
            if (part_of + d * parts < whole) load(d, part_of + d * parts);
        // what this warp reads later to L2 first, ahead of the main kernel's
        // copies: a lane per row and line
        for (uint32_t c = part_of + kD * parts; c < whole; c += parts)
            for (int32_t r = lane; r < kNT * 8; r += 32)
                if (j0 + r < p.rank) prefetch_line(p.A + ((int64_t)id * p.rank + j0 + r) * p.K + 64ull * c);
        for (uint32_t c0 = part_of; c0 < whole; c0 += kD * parts)
#pragma unroll
            for (int d = 0; d < kD; ++d) {
                const uint32_t c = c0 + d * parts;
                if (c >= whole) break;
                multiply(d);
                if (c + kD * parts < whole) load(d, c + kD * parts);
            }
        if (K % 64 != 0 && whole % parts == part_of) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool in = whole * 64 + (uint32_t)(tig * 16 + 8 * h) < K;
#pragma unroll
                for (int n = 0; n < kNT; ++n) av[0][n][h] = load_or_zero(a_row(n) + 64ull * whole + 8 * h, in);
                xv[0][0][h] = load_or_zero(x0 + 64ull * whole + 8 * h, in);
                xv[0][1][h] = load_or_zero(x1 + 64ull * whole + 8 * h, in);
            }
            multiply(0);
        }
        // Sums over the warps and the CTAs of the cluster, in a fixed order:
        // warps 4-7 to warps 0-3, then a thread per element
        __syncthreads();
        if (warp >= kLowWarps / 2)
#pragma unroll
            for (int n = 0; n < kNT; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c) part[warp - kLowWarps / 2][(n * 4 + c) * 32 + lane] = acc[n][c];
        __syncthreads();
        if (warp < kLowWarps / 2)
#pragma unroll
            for (int n = 0; n < kNT; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c) part[warp][(n * 4 + c) * 32 + lane] += acc[n][c];
        __syncthreads();
        constexpr int kE = (kNT * 128 + kLowWarps * 32 - 1) / (kLowWarps * 32);  // elements of a thread
        float v[kE];
#pragma unroll
        for (int i = 0; i < kE; ++i) {
            const int32_t e = (int32_t)threadIdx.x + i * kLowWarps * 32;
            v[i] = 0.0f;
            if (e < kNT * 128) v[i] = (part[0][e] + part[1][e]) + (part[2][e] + part[3][e]);
        }
        if (p.k_split > 1) {
#pragma unroll
            for (int i = 0; i < kE; ++i) {
                const int32_t e = (int32_t)threadIdx.x + i * kLowWarps * 32;
                if (e < kNT * 128) part[0][e] = v[i];
            }
            cluster_sync();
            if (rank == 0) {
#pragma unroll
                for (int i = 0; i < kE; ++i) {
                    const int32_t e = (int32_t)threadIdx.x + i * kLowWarps * 32;
                    if (e >= kNT * 128) continue;
                    const uint32_t at = smem_u32(&part[0][e]);
                    float w[7];
#pragma unroll
                    for (int r = 1; r < 8; ++r) w[r - 1] = r < p.k_split ? ld_shared_cluster(mapa_shared(at, (uint32_t)r)) : 0.0f;
#pragma unroll
                    for (int r = 1; r < 8; ++r) v[i] += w[r - 1];
                }
            }
            cluster_sync();  // its reads are done
        }
        if (rank == 0) {
#pragma unroll
            for (int i = 0; i < kE; ++i) {
                const int32_t e = (int32_t)threadIdx.x + i * kLowWarps * 32;
                if (e >= kNT * 128) continue;
                // element (n, c, lane) of the fragments: its row, its product
                const int32_t l = e & 31, c = (e >> 5) & 3, n = e >> 7;
                const int32_t row = (l >> 2) + 8 * (c >> 1), j = j0 + n * 8 + (l & 3) * 2 + (c & 1);
                if (((his >> row) & 1u) == 0) continue;
                // columns past the rank are zeros whatever the scale is
                const float low = j < p.rank ? v[i] * scale : 0.0f;
                const uint32_t hi = pack16(low, 0.0f, p.bf16);
                uint16_t* dst = p.low + (int64_t)(row0 + row) * 2 * p.rank_pad + j;
                dst[0] = (uint16_t)hi;
                dst[p.rank_pad] = (uint16_t)rest16x2(low, 0.0f, hi, p.bf16);
            }
        }
    }
}

}  // namespace rg
}  // namespace gr
