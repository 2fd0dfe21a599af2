// What the adapters' product needs before its main kernel: the rows' low-rank
// parts and, for each row tile, the list of its distinct adapters.
//
//   low[t, j] = scale[i] * sum_k X[t, k] A[i][j, k],   i = ids[t]
//
// The sums are taken in 32 bits and rounded once, after the scale, to the
// element type: low is the operand of a tensor-core product next, as the
// activations between two layers are.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "ragged_kernel.cuh"

namespace gr {
namespace rg {

constexpr int kPrepWarps = 8;

struct PrepParams {
    const uint16_t* X;   // (T, K), pitch ldx
    const uint16_t* A;   // (R, rank, K)
    const int32_t* ids;  // (T)
    const float* scale;  // (R), or null: 1
    uint16_t* low;       // (T, rank_pad)
    int32_t* slots;      // [tile][cap]
    int32_t* nslots;     // [tile]
    int64_t ldx;
    int32_t T, K, R, rank, rank_pad, cap, tile_w, tiles, bf16;
    int32_t* err;
};

__device__ __forceinline__ float2 unpack16(uint32_t x, int32_t bf16) {
    if (bf16) return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&x));
}

// Blocks [0, tiles): one row tile each, its adapters in order of first
// appearance.  The others: a warp per row and eight of its rank's products.
__global__ void __launch_bounds__(kPrepWarps * 32) adapters_prep_kernel(const __grid_constant__ PrepParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int32_t warp = (int32_t)threadIdx.x / 32, lane = (int32_t)threadIdx.x % 32;
    if ((int32_t)blockIdx.x < p.tiles) {
        __shared__ int32_t id[256];
        __shared__ int32_t count[kPrepWarps];
        const int32_t i = (int32_t)threadIdx.x;
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
            for (int32_t w = 0; w < kPrepWarps; ++w) n += count[w];
            p.nslots[blockIdx.x] = n;
        }
        return;
    }
    const int32_t groups = p.rank_pad / 8;
    const int64_t job = (int64_t)(blockIdx.x - p.tiles) * kPrepWarps + warp;
    if (job >= (int64_t)p.T * groups) return;
    const int32_t t = (int32_t)(job / groups), j0 = (int32_t)(job - (int64_t)t * groups) * 8;
    const int32_t id = __ldcg(p.ids + t);
    if (id < 0 || id >= p.R) return;  // no slot of the row's tile matches it: its low row is not read
    const int32_t nj = min(8, p.rank - j0);
    const uint16_t* x = p.X + (int64_t)t * p.ldx;
    const uint16_t* a = p.A + ((int64_t)id * p.rank + j0) * p.K;
    float sum[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
    for (int32_t k = lane * 8; k < p.K; k += 256) {
        const uint4 xv = *reinterpret_cast<const uint4*>(x + k);
        uint4 av[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            av[j] = j < nj ? *reinterpret_cast<const uint4*>(a + (int64_t)j * p.K + k) : make_uint4(0, 0, 0, 0);
        const uint32_t xs[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t as[4] = {av[j].x, av[j].y, av[j].z, av[j].w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float2 xf = unpack16(xs[c], p.bf16), af = unpack16(as[c], p.bf16);
                sum[j] = fmaf(xf.x, af.x, sum[j]);
                sum[j] = fmaf(xf.y, af.y, sum[j]);
            }
        }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], d);
    if (lane == 0) {
        const float s = p.scale ? __ldcg(p.scale + id) : 1.0f;
        uint4 q;
        // (columns past the rank are zeros whatever the scale is)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = j < nj ? sum[j] * s : 0.0f;
        q.x = pack16(sum[0], sum[1], p.bf16);
        q.y = pack16(sum[2], sum[3], p.bf16);
        q.z = pack16(sum[4], sum[5], p.bf16);
        q.w = pack16(sum[6], sum[7], p.bf16);
        *reinterpret_cast<uint4*>(p.low + (int64_t)t * p.rank_pad + j0) = q;
    }
}

}  // namespace rg
}  // namespace gr
