// What the ragged products' and the losses' entry points share: tensor maps of
// 16-bit matrices, launches that may overlap the previous kernel's end, checks
// of matrix arguments.  Host code only.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdlib.h>

#include <utility>

#include "runtime.h"

namespace gr {
namespace rt {

// A tensor map of 16-bit elements with the 128-byte swizzle; strides in
// elements (the innermost one is 1).
inline int encode(CUtensorMap* map, const void* ptr, int rank, const uint64_t* dims, const uint64_t* strides,
                  const uint32_t* box, bool bf16) {
    cuuint64_t d[4], s[3];
    cuuint32_t b[4], e[4] = {1, 1, 1, 1};
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        b[i] = box[i];
        if (i > 0) s[i - 1] = strides[i - 1] * 2;
    }
    const CUresult r = g_encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                                    (cuuint32_t)rank, const_cast<void*>(ptr), d, s, b, e,
                                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? GEMM_OK : GEMM_ERR_INVALID_ARG;
}

// A (rows x width) matrix of row pitch `pitch`, read as boxes of `box_rows`
// rows x 64 columns; where `blocks` > 0 as a 3-D view of 64-column blocks
// (the width a multiple of 64), `blocks` of them per box.
inline int encode_rows(CUtensorMap* map, const void* ptr, uint64_t width, uint64_t rows, uint64_t pitch,
                       uint32_t box_rows, uint32_t blocks, bool bf16) {
    if (blocks) {
        const uint64_t dims[3] = {64, rows, width / 64}, strides[2] = {pitch, 64};
        const uint32_t box[3] = {64, box_rows, blocks};
        return encode(map, ptr, 3, dims, strides, box, bf16);
    }
    const uint64_t dims[2] = {width, rows}, strides[1] = {pitch};
    const uint32_t box[2] = {64, box_rows};
    return encode(map, ptr, 2, dims, strides, box, bf16);
}

template <typename... P, typename... A>
inline int launch(void (*fn)(P...), int grid, int threads, size_t smem, int cluster, cudaStream_t st, A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    // Set-up may overlap the previous kernel of the stream.  Every kernel here waits for
    // it before it touches global memory, but for four that go by an earlier wait:
    // the adapters' main one, the losses' mask kernel, and their products with `late`
    // or `early`.  (The losses' products also ask for weights in L2 ahead of their
    // wait, which reads nothing into the kernel.)  Such a launch needs two things: its
    // predecessor lets dependents start only behind its own wait (and writes nothing
    // that the launch reads, nor reads what it writes), and the launch waits before it
    // ends, so that its end says that all before it is done.
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    unsigned n = 1;
    if (cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)cluster;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        n = 2;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    if (cudaLaunchKernelEx(&cfg, fn, std::forward<A>(args)...) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

inline bool misaligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

// The test hook of the bounded waits (GEMM_RELU_TEST_DROP_KB=k): plans of
// single CTAs, without clusters and with a k-block k, take it; others refuse.
inline int test_hook(bool single, int32_t blocks, int32_t* drop, uint64_t* timeout_ns) {
    const char* text = getenv("GEMM_RELU_TEST_DROP_KB");
    if (!text || !*text) return GEMM_OK;
    const long kb = strtol(text, nullptr, 10);
    if (kb < 0 || kb >= blocks || !single) return GEMM_ERR_INVALID_ARG;
    *drop = (int32_t)kb + 1;
    *timeout_ns = 1000000;  // 1 ms
    return GEMM_OK;
}

inline bool dim_ok(int64_t v) { return v >= 0 && v <= GEMM_RELU_MAX_DIM; }

// A row-pitched matrix argument of `width` columns.
inline int check_matrix(const void* ptr, int64_t width, int64_t ld) {
    if (!ptr || ld < width || ld > GEMM_RELU_MAX_DIM) return GEMM_ERR_INVALID_ARG;
    if (misaligned(ptr, 16) || ld % 8 != 0) return GEMM_ERR_ALIGNMENT;
    return GEMM_OK;
}

}  // namespace rt
}  // namespace gr
