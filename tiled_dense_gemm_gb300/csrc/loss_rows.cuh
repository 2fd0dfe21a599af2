// The losses' small kernels, row by row: the teacher's words, the rows in use,
// the losses from the tiles' statistics, dX from its sums in 32 bits.
#pragma once

#include "loss_kernel.cuh"

namespace gr {
namespace ls {

constexpr int kMaxWords = 1024;  // of a teacher, per row

// ------------------------------------------------------------------ teacher

struct TeacherParams {
    const int32_t* ids;    // (T, k), negative: none
    const void* logits;    // (T, k)
    int64_t ld_ids, ld_logits;
    int32_t logits_type;   // 0 binary16, 1 bfloat16, 2 32 bits
    int32_t T, k, V;
    float inv_tau;
    int32_t* sorted;       // (T, k), kNone behind the last
    float* weights;        // (T, k) q
    int32_t* flags;        // per row: 0, or -1: no word
    float* entropy;        // per row: sum of q log q
    int32_t* err;
};

__device__ __forceinline__ float load_logit(const TeacherParams& p, int64_t at) {
    if (p.logits_type == 2) return __ldg(reinterpret_cast<const float*>(p.logits) + at);
    const uint16_t x = __ldg(reinterpret_cast<const uint16_t*>(p.logits) + at);
    return p.logits_type == 1 ? __uint_as_float((uint32_t)x << 16) : __half2float(__ushort_as_half(x));
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
    return x;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

constexpr int kTeacherWarps = 4;

// One warp per row: the softmax over its k words in 32 bits, and the words in
// rising order by counting, for each, the smaller ones (k^2 comparisons out of
// shared memory; ties in their given order, so that a word given twice is two
// entries).
__global__ void __launch_bounds__(32 * kTeacherWarps) loss_teacher_kernel(const __grid_constant__ TeacherParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const int32_t warp = (int32_t)threadIdx.x / 32, lane = (int32_t)threadIdx.x % 32;
    const int32_t padded = (p.k + 3) & ~3;
    int32_t* const key = reinterpret_cast<int32_t*>(smem) + 2 * warp * padded;
    float* const e = reinterpret_cast<float*>(key + padded);
    grid_launch_dependents();
    grid_dependency_wait();
    for (int64_t t = (int64_t)blockIdx.x * kTeacherWarps + warp; t < p.T; t += (int64_t)gridDim.x * kTeacherWarps) {
        float top = -INFINITY;
        bool some = false;
        for (int32_t j = lane; j < padded; j += 32) {
            int32_t id = -1;
            float l = -INFINITY;
            if (j < p.k) {
                id = __ldg(p.ids + t * p.ld_ids + j);
                if (id >= p.V) {
                    atomicCAS(p.err + 1, 0, (int32_t)rg::kBadIds);
                    id = -1;
                }
                if (id >= 0) l = load_logit(p, t * p.ld_logits + j);
            }
            key[j] = id < 0 ? kNone : id;
            e[j] = l;
            some |= id >= 0 && l != -INFINITY;
            top = fmaxf(top, l);
        }
        top = warp_max(top);
        some = __any_sync(0xffffffffu, some);
        __syncwarp();
        float sum = 0.0f;
        for (int32_t j = lane; j < p.k; j += 32) {
            const float l = e[j];
            const float x = l == -INFINITY ? -INFINITY : (l - top) * p.inv_tau;
            sum += expf(x);
            e[j] = x;
        }
        sum = warp_sum(sum);
        const float log_sum = logf(sum), inv = 1.0f / sum;
        float h = 0.0f;
        __syncwarp();
        for (int32_t j = lane; j < p.k; j += 32) {
            const float x = e[j], q = expf(x) * inv;
            if (q != 0.0f) h += q * (x - log_sum);
            const int32_t mine = key[j];
            int32_t at = 0;
            for (int32_t i = 0; i < padded; i += 4) {
                const int4 o = *reinterpret_cast<const int4*>(key + i);
                at += (o.x < mine || (o.x == mine && i < j)) + (o.y < mine || (o.y == mine && i + 1 < j)) +
                      (o.z < mine || (o.z == mine && i + 2 < j)) + (o.w < mine || (o.w == mine && i + 3 < j));
            }
            p.sorted[t * p.k + at] = some ? mine : kNone;
            p.weights[t * p.k + at] = mine == kNone || !some ? 0.0f : q;
        }
        h = warp_sum(h);
        if (lane == 0) {
            p.flags[t] = some ? 0 : -1;
            p.entropy[t] = h;
        }
        __syncwarp();
    }
}

// ------------------------------------------------------------------ rows in use

struct RowsParams {
    const int32_t* flags;   // targets, or the teacher's
    int32_t limit;          // values from here on are reported and count as none
    int32_t T, D;
    const uint16_t* X;
    int64_t ldx;
    uint16_t* gathered;     // (T, D)
    int32_t* index;         // the rows in use, then the others
    RowsHeader* rows;
    const float* dloss;     // null: no scale wanted
    int64_t dloss_stride;
    float grad_scale;
    float top;              // what the largest |dloss grad_scale| is scaled to
    int32_t* err;
};

constexpr int kRowsThreads = 256;

// Which rows have a wanted word, gathered to the front where some have none.
// Each block counts for itself what lies before its rows (T flags out of L2, a
// few microseconds beside products of milliseconds), so no block waits for
// another.
__global__ void __launch_bounds__(kRowsThreads) loss_rows_kernel(const __grid_constant__ RowsParams p) {
    __shared__ int32_t part[2][kRowsThreads / 32];
    __shared__ float parts[kRowsThreads / 32];
    __shared__ int32_t where[kRowsThreads];
    const int32_t i = (int32_t)threadIdx.x, warp = i / 32, lane = i % 32;
    grid_launch_dependents();
    grid_dependency_wait();
    const int32_t each = (p.T + (int32_t)gridDim.x - 1) / (int32_t)gridDim.x;
    const int32_t r0 = min(p.T, (int32_t)blockIdx.x * each), r1 = min(p.T, r0 + each);
    int32_t before = 0, total = 0;
    bool bad = false;
    for (int32_t t = i; t < p.T; t += kRowsThreads) {
        const int32_t y = __ldcg(p.flags + t);
        const bool in = y >= 0 && y < p.limit;
        bad |= y >= p.limit;
        total += in;
        before += in && t < r0;
    }
    if (bad && blockIdx.x == 0) atomicCAS(p.err + 1, 0, (int32_t)rg::kBadIds);
    before = __reduce_add_sync(0xffffffffu, before);
    total = __reduce_add_sync(0xffffffffu, total);
    if (lane == 0) {
        part[0][warp] = before;
        part[1][warp] = total;
    }
    __syncthreads();
    before = total = 0;
    for (int32_t j = 0; j < kRowsThreads / 32; ++j) {
        before += part[0][j];
        total += part[1][j];
    }
    __syncthreads();
    const bool gather = total < p.T;
    for (int32_t b = r0; b < r1; b += kRowsThreads) {
        const int32_t t = b + i;
        bool in = false;
        if (t < r1) {
            const int32_t y = __ldcg(p.flags + t);
            in = y >= 0 && y < p.limit;
        }
        const uint32_t votes = __ballot_sync(0xffffffffu, in);
        if (lane == 0) part[0][warp] = __popc(votes);
        __syncthreads();
        int32_t at = before + __popc(votes & ((1u << lane) - 1u));
        for (int32_t j = 0; j < warp; ++j) at += part[0][j];
        for (int32_t j = 0; j < kRowsThreads / 32; ++j) before += part[0][j];
        if (t < r1) p.index[in ? at : total + (t - at)] = t;
        where[i] = in ? at : -1;
        __syncthreads();
        if (gather) {
            const int32_t vecs = p.D / 8;
            for (int32_t j = warp; j < min(kRowsThreads, r1 - b); j += kRowsThreads / 32) {
                const int32_t to = where[j];
                if (to < 0) continue;
                const uint4* const src = reinterpret_cast<const uint4*>(p.X + (int64_t)(b + j) * p.ldx);
                uint4* const dst = reinterpret_cast<uint4*>(p.gathered + (int64_t)to * p.D);
                for (int32_t c = lane; c < vecs; c += 32) dst[c] = __ldg(src + c);
            }
        }
        __syncthreads();
    }
    if (blockIdx.x != gridDim.x - 1) return;
    // the last block: zeros up to the end of the reduction's last k-block, and
    // what the later kernels read of the rows
    if (gather) {
        const int32_t end = min(p.T, (total + kBK - 1) / kBK * kBK);
        const int64_t n = (int64_t)(end - total) * (p.D / 8);
        uint4* const dst = reinterpret_cast<uint4*>(p.gathered + (int64_t)total * p.D);
        for (int64_t c = i; c < n; c += kRowsThreads) dst[c] = make_uint4(0, 0, 0, 0);
    }
    float scale = 1.0f;
    if (p.dloss) {
        float top = 0.0f;
        if (p.dloss_stride == 0) {
            top = fabsf(__ldg(p.dloss));
        } else {
            for (int32_t t = i; t < p.T; t += kRowsThreads) {
                const int32_t y = __ldcg(p.flags + t);
                if (y >= 0 && y < p.limit) top = fmaxf(top, fabsf(__ldg(p.dloss + t)));
            }
        }
        top = warp_max(top);
        if (lane == 0) parts[warp] = top;
        __syncthreads();
        top = 0.0f;
        for (int32_t j = 0; j < kRowsThreads / 32; ++j) top = fmaxf(top, parts[j]);
        top *= p.grad_scale;
        if (top > 1e-30f && top < 1e30f) scale = p.top / top;
    }
    if (i == 0) {
        p.rows->valid = total;
        p.rows->compact = gather ? 1 : 0;
        p.rows->scale = scale;
        p.rows->unscale = 1.0f / scale;
    }
}

// ------------------------------------------------------------------ losses

struct CombineParams {
    const float* stats;     // [part][3][pitch]
    int64_t pitch;
    int32_t parts, T;
    const RowsHeader* rows; // null: all rows are in their places
    const int32_t* index;
    const int32_t* flags;
    int32_t limit;
    const float* entropy;   // teacher; null: targets
    float tau, log2_scale;
    float* loss;
    float* lse;
    int32_t* err;
};

// A block for 32 rows, a lane for each; its warps take the parts in turn and
// are merged in their order.
template <int kWarps>
__global__ void __launch_bounds__(32 * kWarps) loss_combine_kernel(const __grid_constant__ CombineParams p) {
    __shared__ float part[3][kWarps][32];
    const int32_t warp = (int32_t)threadIdx.x / 32, lane = (int32_t)threadIdx.x % 32;
    grid_launch_dependents();
    grid_dependency_wait();
    const int32_t r = (int32_t)blockIdx.x * 32 + lane;
    const int32_t valid = p.rows ? __ldcg(&p.rows->valid) : p.T;
    const float c = p.log2_scale;
    float m = -INFINITY, s = 0.0f, z = 0.0f;
    auto merge = [&](float m1, float s1, float z1) {
        const float top = fmaxf(m, m1);
        const float ref = fabsf(top) == INFINITY ? 0.0f : top;
        // (a sum taken at an infinite maximum is itself infinite or zero and needs no other reference)
        const float f0 = fabsf(m) == INFINITY ? 1.0f : exp2_fast((m - ref) * c);
        const float f1 = fabsf(m1) == INFINITY ? 1.0f : exp2_fast((m1 - ref) * c);
        s = s * f0 + s1 * f1;
        z += z1;
        m = top;
    };
    if (r < valid) {
        const float* at = p.stats + r + (int64_t)warp * 3 * p.pitch;
#pragma unroll 4
        for (int32_t j = warp; j < p.parts; j += kWarps, at += 3 * kWarps * p.pitch)
            merge(__ldcg(at), __ldcg(at + p.pitch), __ldcg(at + 2 * p.pitch));
    }
    part[0][warp][lane] = m;
    part[1][warp][lane] = s;
    part[2][warp][lane] = z;
    __syncthreads();
    if (warp != 0 || r >= p.T) return;
    const int32_t t = p.rows ? __ldcg(p.index + r) : r;
    bool in = r < valid;
    if (!p.rows) {
        const int32_t y = __ldcg(p.flags + r);
        if (y >= p.limit) atomicCAS(p.err + 1, 0, (int32_t)rg::kBadIds);
        in = y >= 0 && y < p.limit;
    }
    float loss = 0.0f, lse = 0.0f;
    if (in) {
        m = -INFINITY;
        s = z = 0.0f;
        for (int32_t j = 0; j < kWarps; ++j) merge(part[0][j][lane], part[1][j][lane], part[2][j][lane]);
        lse = (fabsf(m) == INFINITY ? 0.0f : m / p.tau) + logf(s);
        loss = p.entropy ? p.tau * p.tau * (__ldcg(p.entropy + t) - z / p.tau + lse) : lse - z;
    }
    p.loss[t] = loss;
    p.lse[t] = lse;
}

// ------------------------------------------------------------------ dX

struct FinishParams {
    const float* sums;       // [splits][T][D]
    int32_t splits, T, D, bf16;
    const RowsHeader* rows;
    const int32_t* index;
    uint16_t* dX;
    int64_t ld_dx;
};

// dX[row] from its shares, in their order, rounded once; +0 in the rows that are not in use.
__global__ void __launch_bounds__(256) loss_finish_kernel(const __grid_constant__ FinishParams p) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int32_t valid = __ldcg(&p.rows->valid);
    const float u = __ldcg(&p.rows->unscale);
    const int32_t vecs = p.D / 8;
    const int64_t total = (int64_t)p.T * vecs, share = (int64_t)p.T * p.D;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int32_t r = (int32_t)(i / vecs), c = (int32_t)(i - (int64_t)r * vecs);
        uint4 o = make_uint4(0, 0, 0, 0);
        if (r < valid) {
            float4 a = make_float4(0, 0, 0, 0), b = a;
            const float4* src = reinterpret_cast<const float4*>(p.sums + (int64_t)r * p.D) + 2 * c;
            for (int32_t k = 0; k < p.splits; ++k, src += share / 4) {
                const float4 x = __ldcs(src), y = __ldcs(src + 1);
                a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
                b.x += y.x, b.y += y.y, b.z += y.z, b.w += y.w;
            }
            o = make_uint4(pack16(a.x * u, a.y * u, p.bf16), pack16(a.z * u, a.w * u, p.bf16),
                           pack16(b.x * u, b.y * u, p.bf16), pack16(b.z * u, b.w * u, p.bf16));
        }
        const int32_t t = __ldcg(p.index + r);
        reinterpret_cast<uint4*>(p.dX + (int64_t)t * p.ld_dx)[c] = o;
    }
}

}  // namespace ls
}  // namespace gr
