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
    int32_t before;        // what follows goes by this kernel's wait
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
    if (!p.before) grid_launch_dependents();
    grid_dependency_wait();
    if (p.before) grid_launch_dependents();  // (a G kernel with `early` follows, which goes by that wait)
    for (int64_t t = (int64_t)blockIdx.x * kTeacherWarps + warp; t < p.T; t += (int64_t)gridDim.x * kTeacherWarps) {
        float top = -INFINITY;
        bool some = false;
        for (int32_t j = lane; j < padded; j += 32) {
            int32_t id = -1;
            float l = -INFINITY;
            if (j < p.k) {
                id = __ldg(p.ids + t * p.ld_ids + j);
                l = load_logit(p, t * p.ld_logits + j);
                if (id >= p.V) {
                    atomicCAS(p.err + 1, 0, (int32_t)rg::kBadIds);
                    id = -1;
                }
                if (id < 0) l = -INFINITY;
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
#pragma unroll 4
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
    uint16_t* gathered;     // (T, pitch)
    int32_t* index;         // the rows in use, then the others
    RowsHeader* rows;
    const float* dloss;     // null: no scale wanted
    int64_t dloss_stride;
    float grad_scale;
    float top;              // what the largest |dloss grad_scale| is scaled to
    int32_t pitch;          // of the copy: D rounded up to 64
    int32_t always;         // gather even if all rows are in use
    // masked: rows of the copy, X's over and over after so many (of G's two parts), and
    // what the gradient at a certain word is found from
    int32_t rows_of, period;
    WordSums sums;
    float tau;
    const float* lse;
    uint16_t* grad;           // G
    int64_t grad_pitch;
    int32_t from, words;      // its piece's words
    int32_t low;              // > 0: G's rows from here on take what rounding left
    int32_t* err;
};

constexpr int kRowsThreads = kSumThreads;

// top: the largest |dloss|
__device__ __forceinline__ void write_header(const RowsParams& p, int32_t valid, int32_t compact, float top) {
    const float scale = scale_of(p.top, p.grad_scale, top);
    p.rows->valid = valid;
    p.rows->compact = compact;
    p.rows->scale = scale;
    p.rows->unscale = 1.0f / scale;
}

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
    for (int32_t t0 = i; t0 < p.T; t0 += 8 * kRowsThreads) {
        int32_t y[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int32_t t = t0 + u * kRowsThreads;
            y[u] = t < p.T ? __ldcg(p.flags + t) : -1;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const bool in = y[u] >= 0 && y[u] < p.limit;
            bad |= y[u] >= p.limit;
            total += in;
            before += in && t0 + u * kRowsThreads < r0;
        }
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
    const bool gather = total < p.T || p.always;
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
                uint4* const dst = reinterpret_cast<uint4*>(p.gathered + (int64_t)to * p.pitch);
                for (int32_t c0 = lane; c0 < vecs; c0 += 8 * 32) {
                    uint4 x[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        if (c0 + 32 * u < vecs) x[u] = __ldcs(src + c0 + 32 * u);
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        if (c0 + 32 * u < vecs) dst[c0 + 32 * u] = x[u];
                }
            }
        }
        __syncthreads();
    }
    // zeros up to the end of the reduction's last k-block
    if (gather) {
        const int32_t end = min(p.T, (total + kRowPad - 1) / kRowPad * kRowPad);
        for (int32_t r = total + (int32_t)blockIdx.x; r < end; r += (int32_t)gridDim.x) {
            uint4* const dst = reinterpret_cast<uint4*>(p.gathered + (int64_t)r * p.pitch);
            for (int32_t c = i; c < p.pitch / 8; c += kRowsThreads) dst[c] = make_uint4(0, 0, 0, 0);
        }
    }
    // the last block: what the later kernels read of the rows
    if (blockIdx.x != gridDim.x - 1) return;
    float top = 0.0f;
    if (p.dloss) {
        if (p.dloss_stride == 0) {
            top = fabsf(p.dloss[0]);
        } else {
#pragma unroll 8
            for (int32_t t = i; t < p.T; t += kRowsThreads) {
                const int32_t y = __ldcg(p.flags + t);
                const float d = p.dloss[t];
                if (y >= 0 && y < p.limit) top = fmaxf(top, fabsf(d));
            }
        }
        top = warp_max(top);
        if (lane == 0) parts[warp] = top;
        __syncthreads();
        top = 0.0f;
        for (int32_t j = 0; j < kRowsThreads / 32; ++j) top = fmaxf(top, parts[j]);
    }
    if (i == 0) write_header(p, total, gather ? 1 : 0, top);
}

// Up to 128 rows: nothing is gathered (there is one row tile).  Beside the kernel of
// G (`late`, as there: that one has waited for X and the flags), a block per row:
//
// * a copy of X with zeros in the rows that are not in use, for dW, and the scale;
// * the gradient at the row's main word, if that is all but certain.  Little is
//   left of p - q there, while the tensor core's z is off by up to 6e-6 of itself.  So z
//   is summed once more, without loss, as the forward pass has done for its lse, and 1 +
//   expm1(z / tau - lse) taken for p; that goes over G's entry when the kernel of G is
//   done.  (One row of 576, binary16, 1 - p = 0.003, from an exact lse: dX off by 2.4e-4,
//   its own rounding; 6.7e-3 without.)
//
// Of more rows the certain ones have little part in dX's and dW's size, and G's
// kernel leaves no room beside it: 300 rows, 32008 words of 1000 by columns, 83 us
// without, 94 with a kernel in front of it.
__global__ void __launch_bounds__(kRowsThreads) loss_mask_kernel(const __grid_constant__ RowsParams p) {
    __shared__ double part[kRowsThreads / 32];
    __shared__ int32_t main;
    const int32_t i = (int32_t)threadIdx.x, r = (int32_t)blockIdx.x, warp = i / 32, lane = i % 32;
    grid_launch_dependents();
    const int32_t t = r % p.period;
    const int32_t y = t < p.T ? __ldcg(p.flags + t) : -1;
    if (y >= p.limit && i == 0) atomicCAS(p.err + 1, 0, (int32_t)rg::kBadIds);
    const bool in = y >= 0 && y < p.limit;
    float weight = 1.0f;
    if (warp == 0) {
        const int32_t word = in && r < p.T ? main_word(p.sums, t, weight) : kNone;
        if (lane == 0) main = word >= p.from && word - p.from < p.words ? word : kNone;
    }
    const int32_t vecs = p.D / 8;
    if (in) {
        const uint4* const src = reinterpret_cast<const uint4*>(p.X + (int64_t)t * p.ldx);
        uint4* const dst = reinterpret_cast<uint4*>(p.gathered + (int64_t)r * p.pitch);
        for (int32_t c = i; c < vecs; c += kRowsThreads) dst[c] = __ldg(src + c);
    } else {
        uint4* const dst = reinterpret_cast<uint4*>(p.gathered + (int64_t)r * p.pitch);
        for (int32_t c = i; c < vecs; c += kRowsThreads) dst[c] = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    const int32_t word = main;
    if (word != kNone) {
        double z = some_products(p.sums, t, word, i);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
        if (lane == 0) part[warp] = z;
        __syncthreads();
    }
    float top = 0.0f, g = 0.0f;
    bool sure = false;
    if (warp == 0) {
        top = largest_dloss(p.flags, p.limit, p.dloss, p.dloss_stride, p.T);
        if (word != kNone && lane == 0) {
            double z = 0.0;
            for (int32_t j = 0; j < kRowsThreads / 32; ++j) z += part[j];
            if (p.tau != 1.0f) z /= (double)p.tau;
            const float rest = expm1f((float)(z - (double)p.lse[t]));
            sure = rest > -0.5f;  // (that leaves one word of a row)
            g = p.dloss[(int64_t)t * p.dloss_stride] * p.grad_scale * scale_of(p.top, p.grad_scale, top) * (rest + (1.0f - weight));
        }
        if (r == 0 && lane == 0) write_header(p, p.T, 0, top);
    }
    grid_dependency_wait();
    if (sure) {
        uint16_t* const at = p.grad + (int64_t)t * p.grad_pitch + (word - p.from);
        const uint32_t x = rg::pack16(g, 0.0f, p.sums.bf16);
        at[0] = (uint16_t)x;
        if (p.low) at[(int64_t)p.low * p.grad_pitch] = (uint16_t)rg::rest16x2(g, 0.0f, x, p.sums.bf16);
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
    int32_t shares;            // kExact (up to 128 rows): so many shares of
    const double* exact;       // ... the logit of a row's main word,
    const float* main_weight;  // ... and that word's weight
    float* loss;
    float* lse;
    int32_t* err;
};

// A block for eight rows (a sector of the statistics), so that a row's parts are
// in flight at once: its threads take them in turn and are merged in a fixed
// order.
template <int kWarps, bool kExact>
__global__ void __launch_bounds__(32 * kWarps) loss_combine_kernel(const __grid_constant__ CombineParams p) {
    constexpr int kRows = 8, kLanes = 32 / kRows;  // lanes of a warp per row
    __shared__ float part[3][kWarps][kRows];
    const int32_t warp = (int32_t)threadIdx.x / 32, lane = (int32_t)threadIdx.x % 32;
    const int32_t row = lane % kRows;
    grid_launch_dependents();
    grid_dependency_wait();
    const int32_t r = (int32_t)blockIdx.x * kRows + row;
    const int32_t valid = p.rows ? __ldcg(&p.rows->valid) : p.T;
    const float c = p.log2_scale;
    double exact = 0.0;
    float weight = 1.0f;
    if (kExact && warp == 0 && r < p.T) {
#pragma unroll 8
        for (int32_t j = lane / kRows; j < p.shares; j += kLanes) exact += __ldcg(p.exact + (int64_t)r * p.shares + j);
        if (p.entropy) weight = __ldcg(p.main_weight + r);
    }
    float m = -INFINITY, s = 0.0f, z = 0.0f;
    if (r < valid) {
        const float* const at = p.stats + r;
#pragma unroll 4
        for (int32_t j = kLanes * warp + lane / kRows; j < p.parts; j += kLanes * kWarps) {
            const float* const x = at + (int64_t)j * 3 * p.pitch;
            merge_stats(m, s, __ldcg(x), __ldcg(x + p.pitch), c);
            z += __ldcg(x + 2 * p.pitch);
        }
    }
    auto across = [&]() {  // the lanes of a row
#pragma unroll
        for (int d = kRows; d < 32; d <<= 1) {
            const float m1 = __shfl_xor_sync(0xffffffffu, m, d), s1 = __shfl_xor_sync(0xffffffffu, s, d);
            // (both lanes merge in the same order: the lower lane's first)
            float a = lane & d ? m1 : m, b = lane & d ? s1 : s;
            merge_stats(a, b, lane & d ? m : m1, lane & d ? s : s1, c);
            m = a;
            s = b;
            z += __shfl_xor_sync(0xffffffffu, z, d);
        }
    };
    across();
    if (lane < kRows) {
        part[0][warp][row] = m;
        part[1][warp][row] = s;
        part[2][warp][row] = z;
    }
    __syncthreads();
    if (warp != 0) return;
    m = -INFINITY;
    s = z = 0.0f;
    for (int32_t j = lane / kRows; j < kWarps; j += kLanes) {
        merge_stats(m, s, part[0][j][row], part[1][j][row], c);
        z += part[2][j][row];
    }
    across();
    if constexpr (kExact) {
#pragma unroll
        for (int d = kRows; d < 32; d <<= 1) exact += __shfl_xor_sync(0xffffffffu, exact, d);
    }
    if (r >= p.T || lane >= kRows) return;
    const int32_t t = p.rows ? __ldcg(p.index + r) : r;
    bool in = r < valid;
    if (!p.rows) {
        const int32_t y = __ldcg(p.flags + r);
        if (y >= p.limit) atomicCAS(p.err + 1, 0, (int32_t)rg::kBadIds);
        in = y >= 0 && y < p.limit;
    }
    float loss = 0.0f, lse = 0.0f;
    if (in) {
        // (the maximum meets the wanted logit before the logarithm is added: where a
        // word is nearly certain they are equal, and the loss is the logarithm)
        const float ref = fabsf(m) == INFINITY ? 0.0f : m;
        float log_s = logf(s), gap = ref - z;  // (gap: to the wanted logits' mean)
        lse = ref / p.tau + log_s;
        if constexpr (kExact) {
            // Up to 128 rows, a main word of more than 1/2 (it is the maximum then): its
            // logit from the exact sum, the others' share, s - 1, against that.  The
            // gradients take p - 1 there from that sum and lse, which from the truncated
            // one was off by up to 3e-5 (z = 28 over 2048).
            const double over = exact - (double)ref;
            const float d = (float)(over / (double)p.tau);
            if (fabsf(m) != INFINITY && expf(d) > 0.501f * s) {
                log_s = log1pf((s - 1.0f) * expf(-d));
                lse = (float)(exact / (double)p.tau + (double)log_s);
                gap = (float)((double)gap + over - (double)weight * over);
            }
        }
        // (tau^2 (entropy + gap / tau + log s), without a square that leaves 32 bits)
        loss = p.entropy ? p.tau * (gap + p.tau * (__ldcg(p.entropy + t) + log_s)) : gap + log_s;
    }
    p.loss[t] = loss;
    p.lse[t] = lse;
}

// ------------------------------------------------------------------ dX

__global__ void __launch_bounds__(256) loss_finish_kernel(const __grid_constant__ FinishParams p) {
    grid_launch_dependents();
    grid_dependency_wait();
    finish_dx(p, 256);
}

}  // namespace ls
}  // namespace gr
