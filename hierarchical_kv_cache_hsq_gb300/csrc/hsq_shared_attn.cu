// Attention of a batch whose requests share a prefix (hsq_shared_attn).
#include <cuda_bf16.h>

#include <algorithm>

#include "hsq_ctx.h"
#include "hsq_device.cuh"
#include "hsq_tc.cuh"

namespace {

struct SharedArgs {
    const uint16_t *q, *pk, *pv;
    const int32_t *q_start, *lens, *table, *prefix;
    uint16_t* out; float* lse;
    int rows, B, width, prefix_len, max_new, n_pages, page_n, Hq, Hkv;
    int* err;
};

// Request b's rows and own tokens, checked: rows [first, first + n), own tokens len.
struct Request { int first, n, len; };

__device__ __forceinline__ Request request_of(const SharedArgs& a, int b, int& bad) {
    Request r;
    const int s = a.q_start[b], e = a.q_start[b + 1];
    r.first = s;
    r.n = e - s;
    if (s < 0 || e < s || e > a.rows || r.n > a.max_new) {
        bad |= HSQ_DEVERR_LEN;
        r.n = 0;
    }
    const int len = a.lens[b];
    const long long cap = (long long)a.width * a.page_n;
    r.len = (int)min((long long)max(len, 0), cap);
    if (len != r.len || r.len < r.n) bad |= HSQ_DEVERR_LEN;
    return r;
}

// One warp per (row, query head): lane l holds dims 4 l .. 4 l + 3, keys one after another.
__global__ void __launch_bounds__(kThreads) shared_attn_simple_kernel(SharedArgs a) {
    const int lane = threadIdx.x & 31;
    const long long w = ((long long)blockIdx.x * kThreads + threadIdx.x) >> 5;
    const int row = (int)(w / a.Hq), jq = (int)(w % a.Hq), h = jq / (a.Hq / a.Hkv);
    if (row >= a.rows) return;
    int lo = 0, hi = a.B;  // the last b with q_start[b] <= row
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.q_start[mid] <= row) lo = mid; else hi = mid;
    }
    int bad = 0;
    const Request rq = request_of(a, lo, bad);
    if (bad && lane == 0) atomicOr(a.err, bad);
    if (row < rq.first || row >= rq.first + rq.n) return;
    const int own = min(rq.len, max(0, rq.len - rq.n + (row - rq.first) + 1));
    const size_t at = ((size_t)row * a.Hq + jq) * kDim + 4 * lane;
    const uint2 qw = *reinterpret_cast<const uint2*>(a.q + at);
    float q[4] = {__uint_as_float(qw.x << 16), __uint_as_float(qw.x & 0xFFFF0000u), __uint_as_float(qw.y << 16),
                  __uint_as_float(qw.y & 0xFFFF0000u)};
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] *= kLogitScaleLog2;
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    auto run = [&](const int32_t* ids, int count) {
        for (int s = 0; s < count; ++s) {
            const int id = ids[s / a.page_n];
            if (id < 0 || id >= a.n_pages) {
                if (lane == 0) atomicOr(a.err, HSQ_DEVERR_PAGE);
                continue;
            }
            const size_t k0 = (((size_t)id * a.Hkv + h) * a.page_n + s % a.page_n) * kDim + 4 * lane;
            const uint2 kw = *reinterpret_cast<const uint2*>(a.pk + k0), vw = *reinterpret_cast<const uint2*>(a.pv + k0);
            float x = q[0] * __uint_as_float(kw.x << 16);
            x = fmaf(q[1], __uint_as_float(kw.x & 0xFFFF0000u), x);
            x = fmaf(q[2], __uint_as_float(kw.y << 16), x);
            x = fmaf(q[3], __uint_as_float(kw.y & 0xFFFF0000u), x);
#pragma unroll
            for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(kFull, x, d);
            const float mn = fmaxf(m, x), c = exp2f(m - mn), p = exp2f(x - mn);
            m = mn;
            l = fmaf(l, c, p);
            o[0] = fmaf(o[0], c, p * __uint_as_float(vw.x << 16));
            o[1] = fmaf(o[1], c, p * __uint_as_float(vw.x & 0xFFFF0000u));
            o[2] = fmaf(o[2], c, p * __uint_as_float(vw.y << 16));
            o[3] = fmaf(o[3], c, p * __uint_as_float(vw.y & 0xFFFF0000u));
        }
    };
    run(a.prefix, a.prefix_len);
    run(a.table + (size_t)lo * a.width, own);
    const float inv = l > 0.f ? 1.0f / l : 0.f;
    const __nv_bfloat162 x = __floats2bfloat162_rn(o[0] * inv, o[1] * inv), y = __floats2bfloat162_rn(o[2] * inv, o[3] * inv);
    *reinterpret_cast<uint2*>(a.out + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
    if (a.lse && lane == 0) a.lse[(size_t)row * a.Hq + jq] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace

extern "C" {

hsq_status hsq_shared_attn_workspace_size(const hsq_ctx* ctx, int rows, int B, int prefix_len, int max_new,
                                          size_t* bytes) {
    if (!ctx || !bytes) return hsq::fail(nullptr, HSQ_ERR_INVALID, "ctx or bytes is NULL");
    if (rows < 1 || B < 1 || prefix_len < 0 || max_new < 1)
        return hsq::fail(nullptr, HSQ_ERR_INVALID, "rows, B and max_new must be positive, prefix_len not negative");
    *bytes = 256;
    return HSQ_OK;
}

hsq_status hsq_shared_attn(hsq_ctx* ctx, const hsq_pages* pages, int rows, int B, int width, int prefix_len,
                           int max_new, const void* q, const int32_t* q_start, const int32_t* lens,
                           const int32_t* table, const int32_t* prefix, void* out, float* lse_opt, void* workspace,
                           size_t workspace_bytes, hsq_stream_t stream) {
    hsq_status st = hsq::check_pages(ctx, pages, true);
    if (st != HSQ_OK) return st;
    if (!q || !q_start || !lens || !table || !out || !workspace)
        return hsq::fail(ctx, HSQ_ERR_INVALID, "an argument of hsq_shared_attn is NULL");
    if (B < 1 || B > ctx->cfg.max_batch || B > HSQ_MAX_REQUESTS)
        return hsq::fail(ctx, HSQ_ERR_INVALID, "B outside [1, min(max_batch, HSQ_MAX_REQUESTS)]");
    if (rows < 1 || width < 1 || max_new < 1 || prefix_len < 0)
        return hsq::fail(ctx, HSQ_ERR_INVALID, "rows, width and max_new must be positive, prefix_len not negative");
    if (prefix_len > 0 && !prefix) return hsq::fail(ctx, HSQ_ERR_INVALID, "prefix is NULL with prefix_len > 0");
    if (((uintptr_t)q | (uintptr_t)out) & 15u)
        return hsq::fail(ctx, HSQ_ERR_INVALID, "q and out must be 16-byte aligned");
    if ((uintptr_t)workspace & 255u) return hsq::fail(ctx, HSQ_ERR_INVALID, "workspace must be 256-byte aligned");
    size_t need = 0;
    if ((st = hsq_shared_attn_workspace_size(ctx, rows, B, prefix_len, max_new, &need)) != HSQ_OK) return st;
    if (workspace_bytes < need)
        return hsq::fail(ctx, HSQ_ERR_INVALID, "workspace smaller than hsq_shared_attn_workspace_size");
    if ((st = hsq::check_device(ctx)) != HSQ_OK) return st;
    SharedArgs a{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(pages->k),
                 static_cast<const uint16_t*>(pages->v), q_start, lens, table, prefix, static_cast<uint16_t*>(out),
                 lse_opt, rows, B, width, prefix_len, max_new, pages->n_pages, pages->page_n, ctx->cfg.n_q_heads,
                 ctx->cfg.n_kv_heads, ctx->d_err};
    const long long warps = (long long)rows * ctx->cfg.n_q_heads;
    const int grid = (int)((warps * 32 + kThreads - 1) / kThreads);
    shared_attn_simple_kernel<<<grid, kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? HSQ_OK : hsq::cuda_fail(ctx, e, "shared_attn");
}

}  // extern "C"
