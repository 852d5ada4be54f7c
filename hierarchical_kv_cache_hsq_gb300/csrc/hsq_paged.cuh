// Building blocks of the paged attention kernels (hsq_shared_attn.cu, hsq_page_attn.cu, hsq_page_select.cu): warp-level
// matrix products, packed fp32 arithmetic, rings of stages, lookups; tensor maps and launches on the host side.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "hsq_ctx.h"
#include "hsq_device.cuh"
#include "hsq_tc.cuh"

namespace hsq_paged {

using namespace hsq_tc;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&x);
}

// two fp32 lanes in one instruction
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ void unpack2(uint64_t d, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(d));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&x)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};\n"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix(uint32_t (&x)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix_trans(uint32_t (&x)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}

// One arrival for the whole warp, after every lane's writes.
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// A place in a ring of N stages, and the parity of its barriers' phase.
template <uint32_t N>
struct Ring {
    uint32_t stage, phase;
    __device__ __forceinline__ void advance() {
        if (++stage == N) {
            stage = 0;
            phase ^= 1;
        }
    }
};

// The last b with at[b] <= x (at ascending, at[0] = 0, n entries), by a whole warp: 32 probes a step.
__device__ __forceinline__ int warp_find(const long long* at, int n, long long x) {
    const int lane = threadIdx.x & 31;
    int lo = 0, len = n;
    while (len > 1) {
        const int step = (len + 31) / 32, i = lo + lane * step;
        const bool le = lane * step < len && at[i] <= x;
        const int k = max(__popc(__ballot_sync(kFull, le)) - 1, 0);
        len = min(step, len - k * step);
        lo += k * step;
    }
    return lo;
}

// The request of a row, and what the row sees of its own tokens.
struct RowOf {
    int b, seen;  // seen: of the request's tokens, the first `seen`
    bool live;    // false: the row belongs to no request, or to one that is left out
};

// By a whole warp, uniformly.  A decode step's rows are its requests: that is looked at first, else 32 probes a step.
__device__ __forceinline__ RowOf warp_row(const int32_t* q_start, const int32_t* lens, int B, int rows, int max_new,
                                          int held_most, int row, int& bad) {
    const int lane = threadIdx.x & 31;
    RowOf r{row, 0, false};
    int s = 0, e = 0, l = 0;
    if (row < B) {
        const int v = lane == 2 ? lens[row] : q_start[row + (lane & 1)];
        s = __shfl_sync(kFull, v, 0);
        e = __shfl_sync(kFull, v, 1);
        l = __shfl_sync(kFull, v, 2);
    }
    if (!(s <= row && row < e)) {
        int lo = 0, len = B;
        while (len > 1) {
            const int step = (len + 31) / 32;
            const bool le = lane * step < len && q_start[lo + lane * step] <= row;
            const int k = max(__popc(__ballot_sync(kFull, le)) - 1, 0);
            len = min(step, len - k * step);
            lo += k * step;
        }
        const int v = lane == 2 ? lens[lo] : q_start[lo + (lane & 1)];
        r.b = lo;
        s = __shfl_sync(kFull, v, 0);
        e = __shfl_sync(kFull, v, 1);
        l = __shfl_sync(kFull, v, 2);
    }
    if (s <= row && row < e) {
        const int n = e - s;
        if (s < 0 || e > rows || n > max_new) {
            bad |= HSQ_DEVERR_LEN;
        } else {
            const int held = min(max(l, 0), held_most);
            if (held != l || l < n) bad |= HSQ_DEVERR_LEN;
            r.seen = min(max(max(l, 0) - n + (row - s) + 1, 0), held);
            r.live = true;
        }
    }
    return r;
}

// Whether the offsets ascend in [0, rows] and the lengths are none below 0, past their table or below the request's rows, by a
// whole CTA of `threads`; what is not so is flagged.  (A request without rows has no CTA that would look at its length.)
__device__ __forceinline__ int requests_bad(const int32_t* q_start, const int32_t* lens, int B, int rows, int held_most, int threads) {
    int bad = 0;
    for (int b = threadIdx.x; b < B; b += threads) {
        const int s = q_start[b], e = q_start[b + 1], l = lens[b];
        if (s < 0 || e < s || e > rows || l < 0 || l > held_most || l < e - s) bad = HSQ_DEVERR_LEN;
    }
    return bad;
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

// bf16 rows of 128, seen as boxes of 64 columns (128-byte swizzle)
inline bool encode_rows(CUtensorMap* map, void* p, uint64_t rows, uint32_t box_rows) {
    const cuuint64_t dims[2] = {128, rows}, strides[1] = {256};
    const cuuint32_t box[2] = {64, box_rows}, es[2] = {1, 1};
    return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same with both halves of a row in one box, the first half's rows before the second's (one copy in place of two: a
// copy takes its thread some 150 cycles to issue).
inline bool encode_halves(CUtensorMap* map, void* p, uint64_t rows, uint32_t box_rows) {
    const cuuint64_t dims[3] = {64, rows, 2}, strides[2] = {256, 128};
    const cuuint32_t box[3] = {64, box_rows, 2}, es[3] = {1, 1, 1};
    return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same in groups of 8 rows: a group's first halves, then its second ones.  rows and box_rows: multiples of 8.
inline bool encode_groups(CUtensorMap* map, void* p, uint64_t rows, uint32_t box_rows) {
    const cuuint64_t dims[4] = {64, 8, 2, rows / 8}, strides[3] = {256, 128, 2048};
    const cuuint32_t box[4] = {64, 8, 2, box_rows / 8}, es[4] = {1, 1, 1, 1};
    return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, p, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// queries [rows][Hq][128]: a box is `tokens` tokens x the r heads of a KV head x 64 columns
inline bool encode_q(CUtensorMap* map, const void* p, uint64_t rows, uint64_t Hq, uint32_t r, uint32_t tokens) {
    const cuuint64_t dims[3] = {128, Hq, rows}, strides[2] = {256, 256 * Hq};
    const cuuint32_t box[3] = {64, r, tokens}, es[3] = {1, 1, 1};
    return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, es,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline cudaError_t launch(const void* fn, int grid, int threads, size_t smem, cudaStream_t st, bool after, void** args) {
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3(grid);
    lc.blockDim = dim3(threads);
    lc.dynamicSmemBytes = smem;
    lc.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = at;
    lc.numAttrs = after ? 1 : 0;
    return cudaLaunchKernelExC(&lc, fn, args);
}

inline cudaError_t launch_cluster(const void* fn, unsigned grid, int threads, int cluster, size_t smem, cudaStream_t st, bool after, void** args) {
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3(grid);
    lc.blockDim = dim3(threads);
    lc.dynamicSmemBytes = smem;
    lc.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = at;
    lc.numAttrs = after ? 2 : 1;
    return cudaLaunchKernelExC(&lc, fn, args);
}

}  // namespace hsq_paged
