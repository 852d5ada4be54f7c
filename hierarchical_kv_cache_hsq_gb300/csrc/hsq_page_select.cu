// Selection of pages by a cheap score (hsq_page_select).
//
// For row i of request b and KV head h, with cq the 8-bit codes of the sum of the head's query rows and
// codes, scale the summary of page p:  score_p = (sum_d cq_d codes_pd) scale_p.  The sum is a whole number below 2^21,
// exact in every order of summation, and the product one rounding, so the selection does not depend on how the work is
// divided.  Taken are the first pages, the row's last ones, and the best of the others, ties to the lower page.
#include <cuda_bf16.h>

#include <algorithm>

#include "hsq_ctx.h"
#include "hsq_paged.cuh"

namespace {

using namespace hsq_paged;

struct SelectArgs {
    const uint16_t* q;
    const int32_t *q_start, *lens, *table, *prefix;
    const int8_t* codes; const float* scale;
    int32_t* sel;
    int rows, B, width, prefix_pages, max_new, n_pages, page_n, page_shift, Hq, Hkv, r, top, first, recent;
    int* err;
};

constexpr int kSelThreads = 256;
constexpr uint32_t kKeyNan = 0xFFFFFFFEu;

// Codes of the sum of r query rows, by a whole warp: lane holds dims 4 lane .. 4 lane + 3, packed.
__device__ __forceinline__ uint32_t query_codes(const uint16_t* q, int r) {
    const int lane = threadIdx.x & 31;
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < r; ++j) {
        const uint2 v = *reinterpret_cast<const uint2*>(q + (size_t)j * 128 + 4 * lane);
        const float y[4] = {__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                            __uint_as_float(v.y & 0xFFFF0000u)};
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = j ? __fadd_rn(x[k], y[k]) : y[k];
    }
    float top = 0.f;
    bool bad = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        top = fmaxf(top, fabsf(x[k]));
        bad |= !(fabsf(x[k]) <= 3.4028234663852886e38f);
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
    bad = __any_sync(kFull, bad) || top < 0x1p-64f;
    const float by = __fdiv_rn(127.f, bad ? 1.f : top);
    uint32_t w = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) w |= (uint32_t)((bad ? 0 : __float2int_rn(__fmul_rn(x[k], by))) & 0xFF) << (8 * k);
    return w;
}

// Order-preserving key of a score, never 0 (which stands for a page that cannot be selected).
__device__ __forceinline__ uint32_t score_key(int dot, float scale) {
    const float s = __fmul_rn((float)dot, scale);
    return s != s ? kKeyNan : max(ordered_key(s), 1u);
}

__global__ void __launch_bounds__(kSelThreads) page_select_kernel(SelectArgs a) {
    extern __shared__ uint32_t s_keys[];
    __shared__ SelectSmem ss;
    __shared__ uint32_t s_q[32];
    __shared__ int s_row[3];
    __shared__ int s_out[HSQ_MAX_BETA];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.x % a.Hkv, row = blockIdx.x / a.Hkv;
    int bad = 0;
    if (warp == 0) {
        const RowOf r = warp_row(a.q_start, a.lens, a.B, a.rows, a.max_new, a.width << a.page_shift, row, bad);
        if (lane == 0) {
            s_row[0] = r.b;
            s_row[1] = r.seen;
            s_row[2] = r.live;
        }
    } else if (warp == 1) {
        s_q[lane] = query_codes(a.q + ((size_t)row * a.Hq + h * a.r) * 128, a.r);
    }
    if (blockIdx.x == 0) bad |= offsets_bad(a.q_start, a.B, a.rows, kSelThreads);
    __syncthreads();
    if (s_row[2]) {
        const int b = s_row[0], c = a.prefix_pages + ((s_row[1] + a.page_n - 1) >> a.page_shift);
        int32_t* out = a.sel + ((size_t)row * a.Hkv + h) * a.top;
        const int G = c - a.first - a.recent, beta = a.top - a.first - a.recent;
        if (c <= a.top) {
            for (int i = tid; i < a.top; i += kSelThreads) out[i] = i < c ? i : -1;
        } else {
            if (beta > 0) {
                const uint4 cq = reinterpret_cast<const uint4*>(s_q)[lane & 7];
                for (int i0 = warp * 32; i0 < G; i0 += kSelThreads) {
                    const int i = i0 + lane, p = a.first + i;
                    int id = -1;
                    if (i < G) {
                        id = p < a.prefix_pages ? a.prefix[p] : a.table[(size_t)b * a.width + p - a.prefix_pages];
                        if (id < 0 || id >= a.n_pages) {
                            id = -1;
                            bad |= HSQ_DEVERR_PAGE;
                        }
                    }
                    const float scale = id >= 0 ? a.scale[(size_t)id * a.Hkv + h] : 0.f;
                    int mine = 0;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {  // four pages at a time, eight lanes each
                        const int of = __shfl_sync(kFull, id, 4 * k + (lane >> 3));
                        int dot = 0;
                        if (of >= 0) {
                            const uint4 m = *reinterpret_cast<const uint4*>(a.codes + ((size_t)of * a.Hkv + h) * 128 + 16 * (lane & 7));
                            dot = __dp4a((int)m.x, (int)cq.x, dot);
                            dot = __dp4a((int)m.y, (int)cq.y, dot);
                            dot = __dp4a((int)m.z, (int)cq.z, dot);
                            dot = __dp4a((int)m.w, (int)cq.w, dot);
                        }
#pragma unroll
                        for (int d = 1; d < 8; d <<= 1) dot += __shfl_xor_sync(kFull, dot, d);
                        const int got = __shfl_sync(kFull, dot, 8 * (lane & 3));
                        if ((lane >> 2) == k) mine = got;
                    }
                    if (i < G) s_keys[i] = id >= 0 ? score_key(mine, scale) : 0u;
                }
                __syncthreads();
                select_top_beta<kSelThreads>(s_keys, G, beta, s_out, ss);
                __syncthreads();
            }
            // the first pages, the selected ones and the last ones (which move up where fewer could be selected)
            for (int i = tid; i < a.first; i += kSelThreads) out[i] = i;
            int n = 0;
            for (int i0 = 0; i0 < beta; i0 += kSelThreads) {
                const int i = i0 + tid;
                const bool got = i < beta && s_out[i] >= 0;
                if (got) out[a.first + i] = a.first + s_out[i];
                n += __syncthreads_count(got);
            }
            for (int i = tid; i < a.recent; i += kSelThreads) out[a.first + n + i] = c - a.recent + i;
            for (int i = a.first + n + a.recent + tid; i < a.top; i += kSelThreads) out[i] = -1;
        }
    }
    if (bad) atomicOr(a.err, bad);
}

}  // namespace

extern "C" {

hsq_status hsq_page_select_workspace_size(const hsq_ctx* ctx, int page_n, int rows, int B, int width, int prefix_len,
                                          int top, int max_new, size_t* bytes) {
    if (!ctx || !bytes) return hsq::fail(nullptr, HSQ_ERR_INVALID, "ctx or bytes is NULL");
    const char* wrong = hsq::selection_shape_wrong(page_n, rows, B, width, prefix_len, top, max_new);
    if (wrong) return hsq::fail(nullptr, HSQ_ERR_INVALID, wrong);
    *bytes = 256;
    return HSQ_OK;
}

hsq_status hsq_page_select(hsq_ctx* ctx, const hsq_pages* pages, const hsq_summaries* sums, int rows, int B, int width,
                           int prefix_len, int top, int first, int recent, int max_new, const void* q,
                           const int32_t* q_start, const int32_t* lens, const int32_t* table, const int32_t* prefix,
                           int32_t* sel, void* workspace, size_t workspace_bytes, hsq_stream_t stream) {
    hsq_status st = hsq::check_pages(ctx, pages, false);
    if (st != HSQ_OK) return st;
    if ((st = hsq::check_summaries(ctx, sums)) != HSQ_OK) return st;
    if (!q || !q_start || !lens || !table || !sel || !workspace)
        return hsq::fail(ctx, HSQ_ERR_INVALID, "an argument of hsq_page_select is NULL");
    const char* wrong = hsq::selection_shape_wrong(pages->page_n, rows, B, width, prefix_len, top, max_new);
    if (wrong) return hsq::fail(ctx, HSQ_ERR_INVALID, wrong);
    if (B > ctx->cfg.max_batch) return hsq::fail(ctx, HSQ_ERR_INVALID, "B above max_batch");
    if (first < 0 || recent < 1 || first > top || recent > top - first)
        return hsq::fail(ctx, HSQ_ERR_INVALID, "first >= 0, recent >= 1 and first + recent <= top");
    if (prefix_len > 0 && !prefix) return hsq::fail(ctx, HSQ_ERR_INVALID, "prefix is NULL with prefix_len > 0");
    if ((uintptr_t)q & 15u) return hsq::fail(ctx, HSQ_ERR_INVALID, "q must be 16-byte aligned");
    if ((uintptr_t)workspace & 255u) return hsq::fail(ctx, HSQ_ERR_INVALID, "workspace must be 256-byte aligned");
    size_t need = 0;
    hsq_page_select_workspace_size(ctx, pages->page_n, rows, B, width, prefix_len, top, max_new, &need);
    if (workspace_bytes < need)
        return hsq::fail(ctx, HSQ_ERR_INVALID, "workspace smaller than hsq_page_select_workspace_size");
    const int Hq = ctx->cfg.n_q_heads, Hkv = ctx->cfg.n_kv_heads, P = pages->page_n, np = (prefix_len + P - 1) / P;
    if ((long long)rows * Hkv >= (1LL << 27)) return hsq::fail(ctx, HSQ_ERR_INVALID, "too many rows");
    const size_t heads = (size_t)pages->n_pages * Hkv;
    const hsq::Span ins[] = {{q, (size_t)rows * Hq * 256}, {q_start, 4 * ((size_t)B + 1)}, {lens, 4 * (size_t)B},
                             {table, 4 * (size_t)B * width}, {prefix_len > 0 ? prefix : nullptr, 4 * (size_t)np},
                             {sums->codes, heads * 128}, {sums->scale, heads * 4}};
    const hsq::Span outs[] = {{sel, (size_t)rows * Hkv * top * 4}, {workspace, need}};
    if (hsq::outputs_overlap(ins, outs))
        return hsq::fail(ctx, HSQ_ERR_INVALID, "sel or the workspace of hsq_page_select overlaps another argument");
    if ((st = hsq::check_device(ctx)) != HSQ_OK) return st;
    SelectArgs a{};
    a.q = static_cast<const uint16_t*>(q);
    a.q_start = q_start; a.lens = lens; a.table = table; a.prefix = prefix;
    a.codes = sums->codes; a.scale = sums->scale; a.sel = sel;
    a.rows = rows; a.B = B; a.width = width; a.prefix_pages = np; a.max_new = max_new;
    a.n_pages = pages->n_pages; a.page_n = P; a.page_shift = P == 16 ? 4 : P == 32 ? 5 : P == 64 ? 6 : 7;
    a.Hq = Hq; a.Hkv = Hkv; a.r = ctx->r; a.top = top; a.first = first; a.recent = recent;
    a.err = ctx->d_err;
    const size_t smem = 4 * (size_t)(np + width);
    cudaError_t e = hsq::raise_smem_limit((const void*)page_select_kernel, ctx->device, smem);
    if (e != cudaSuccess) return hsq::cuda_fail(ctx, e, "cudaFuncSetAttribute(page_select)");
    page_select_kernel<<<rows * Hkv, kSelThreads, smem, reinterpret_cast<cudaStream_t>(stream)>>>(a);
    e = cudaGetLastError();
    return e == cudaSuccess ? HSQ_OK : hsq::cuda_fail(ctx, e, "page_select");
}

}  // extern "C"
