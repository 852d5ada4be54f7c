// Paged serving: block tables and slot maps from request lengths
// (hsq_page_tables), and the rotated, paged write of a step's keys and values
// (hsq_page_write).
#include <cuda_bf16.h>

#include <algorithm>
#include <climits>

#include "hsq_ctx.h"
#include "hsq_device.cuh"

namespace {

constexpr int kTabThreads = 512;
constexpr int kMaxLen = 1 << 30;

struct TablesArgs {
    const int32_t *cached, *fresh, *free_ids, *used;
    int32_t* table; int64_t* slots; int32_t *pos, *q_start, *lens, *used_out;
    int B, width, rows, n_free, base, n_pages, page_n;
    int* err;
};

// Every CTA scans the lengths itself (B <= 4096: two loads and ten shuffles a
// thread and round) and keeps both prefix sums -- rows, pages taken -- in
// shared memory; then the grid strides over the rows and the new table entries,
// each found by a binary search in them.  So one launch does without any
// exchange between CTAs: nothing that one CTA reads is written by another (a
// token's page is either an old entry of the table or, for a page taken in this
// call, read from the free list itself).  Bound by its latency: launch, length
// loads, scan, search.
__global__ void __launch_bounds__(kTabThreads) page_tables_kernel(TablesArgs a) {
    extern __shared__ int tab_sm[];
    int* s_row = tab_sm;              // [B + 1] rows before request b
    int* s_page = tab_sm + a.B + 1;   // [B + 1] pages taken before request b
    __shared__ int s_wr[kTabThreads / 32], s_wp[kTabThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int shift = __ffs(a.page_n) - 1;
    const bool first = blockIdx.x == 0;
    int bad = 0, row0 = 0, page0 = 0;
    for (int b0 = 0; b0 < a.B; b0 += kTabThreads) {
        const int b = b0 + tid;
        int c = 0, f = 0;
        if (b < a.B) {
            c = a.cached[b];
            f = a.fresh[b];
            if (c < 0 || f < 0 || c > kMaxLen || f > kMaxLen) bad |= HSQ_DEVERR_LEN;
            c = min(max(c, 0), kMaxLen);
            f = min(max(f, 0), kMaxLen - c);
            if ((c + f + a.page_n - 1) >> shift > a.width) bad |= HSQ_DEVERR_LEN;
            if (first) a.lens[b] = c + f;
        }
        // (no page is taken past the table's width; a request's rows saturate at the rows there are)
        const int xi = min(f, a.rows);
        const int yi = min((c + f + a.page_n - 1) >> shift, a.width) - min((c + a.page_n - 1) >> shift, a.width);
        long long X = xi, Y = yi;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(kFull, X, o), w = __shfl_up_sync(kFull, Y, o);
            if (lane >= o) { X += u; Y += w; }
        }
        if (lane == 31) {
            s_wr[warp] = (int)min(X, (long long)INT_MAX);
            s_wp[warp] = (int)min(Y, (long long)INT_MAX);
        }
        __syncthreads();
        long long tr = row0, tp = page0;
        for (int w = 0; w < kTabThreads / 32; ++w) {
            if (w == warp) { X += tr; Y += tp; }
            tr += s_wr[w];
            tp += s_wp[w];
        }
        if (b < a.B) {
            s_row[b] = (int)min(X - xi, (long long)a.rows);
            s_page[b] = (int)min(Y - yi, (long long)INT_MAX);
            if (X > a.rows) bad |= HSQ_DEVERR_LEN;
        }
        row0 = (int)min(tr, (long long)a.rows);
        page0 = (int)min(tp, (long long)INT_MAX);
        __syncthreads();
    }
    if (tid == 0) {
        s_row[a.B] = row0;
        s_page[a.B] = page0;
    }
    int used = *a.used;
    if (used < 0 || used > a.n_free) bad |= HSQ_DEVERR_LEN;
    used = min(max(used, 0), a.n_free);
    if (page0 > a.n_free - used) bad |= HSQ_DEVERR_PAGE;
    __syncthreads();
    if (first) {
        for (int b = tid; b <= a.B; b += kTabThreads) a.q_start[b] = s_row[b];
        if (tid == 0) *a.used_out = used + min(page0, a.n_free - used);
    }
    // id of the e-th page taken in this call, -1 when the list is at its end or holds no page of the pool
    auto taken = [&](int e) {
        int id = -1;
        if (e < a.n_free - used) {
            id = a.free_ids[used + e];
            if (id < 0 || id >= a.n_pages) { id = -1; bad |= HSQ_DEVERR_PAGE; }
        }
        return id;
    };
    auto find = [&](const int* s, int x) {  // the last b with s[b] <= x
        int lo = 0, hi = a.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s[mid] <= x) lo = mid; else hi = mid;
        }
        return lo;
    };
    const int stride = gridDim.x * kTabThreads, at = blockIdx.x * kTabThreads + tid;
    for (int e = at; e < page0; e += stride) {
        const int b = find(s_page, e);
        const int c = min(max(a.cached[b], 0), kMaxLen);
        const int col = ((c + a.page_n - 1) >> shift) + e - s_page[b];
        if (col < a.width) a.table[(size_t)b * a.width + col] = taken(e);
    }
    for (int i = at; i < a.rows; i += stride) {
        long long slot = -1;
        int pos = -1;
        if (i < row0) {
            const int b = find(s_row, i);
            const int c = min(max(a.cached[b], 0), kMaxLen);
            const int p = c + i - s_row[b], col = p >> shift, have = (c + a.page_n - 1) >> shift;
            int id = -1;
            if (col < a.width) {
                if (col >= have) {
                    id = taken(s_page[b] + col - have);
                } else {
                    id = a.table[(size_t)b * a.width + col];
                    if (id < 0 || id >= a.n_pages) { id = -1; bad |= HSQ_DEVERR_PAGE; }
                }
            }
            pos = a.base + p;
            if (id >= 0) slot = ((long long)id << shift) + (p & (a.page_n - 1));
        }
        a.slots[i] = slot;
        a.pos[i] = pos;
    }
    if (bad) atomicOr(a.err, bad);
}

constexpr int kWriteHeads = 8;  // vectors of one row that a half-warp rotates with one set of angles

struct WriteArgs {
    const void *q, *k, *v;
    long long qs, ks, vs;  // elements between rows
    const int32_t* pos; const int64_t* slots;
    uint16_t *q_out, *pk, *pv;
    int rows, Hq, Hkv, n_pages, page_n, units;  // units: groups of kWriteHeads vectors of a row
    int* err;
};

__device__ __forceinline__ void store_bf16x8(uint16_t* p, const float v[8]) {
    const int l = hlane();
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    const __nv_bfloat162 c = __floats2bfloat162_rn(v[4], v[5]), d = __floats2bfloat162_rn(v[6], v[7]);
    *reinterpret_cast<uint2*>(p + 4 * l) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    *reinterpret_cast<uint2*>(p + 64 + 4 * l) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&c), *reinterpret_cast<const uint32_t*>(&d));
}

// One half-warp per (row, up to 8 of its Hq + 2 Hkv vectors): the row's cos / sin
// once, then load, rotate, round, store.  Bound by HBM.
template <bool BF>
__global__ void __launch_bounds__(kThreads) page_write_kernel(WriteArgs a, Tables tb) {
    const int l = hlane();
    const long long unit = ((long long)blockIdx.x * kThreads + threadIdx.x) >> 4;
    const int row = (int)(unit / a.units), g = (int)(unit % a.units);
    if (row >= a.rows) return;
    int p = a.pos[row];
    if (p < 0) return;
    if (p >= tb.max_pos) {
        p = tb.max_pos - 1;
        if (l == 0) atomicOr(a.err, HSQ_DEVERR_POS);
    }
    const int H = a.Hq + 2 * a.Hkv;
    long long slot = a.slots[row];
    if (slot >= (long long)a.n_pages * a.page_n) {
        slot = -1;
        if (l == 0) atomicOr(a.err, HSQ_DEVERR_PAGE);
    }
    const RopeRows rr = rope_rows(p, tb);
    const long long page = slot / a.page_n, off = slot % a.page_n;
#pragma unroll 2
    for (int i = g * kWriteHeads; i < min(H, (g + 1) * kWriteHeads); ++i) {
        const bool is_q = i < a.Hq, is_v = i >= a.Hq + a.Hkv;
        if (!is_q && slot < 0) continue;
        const int h = is_q ? i : is_v ? i - a.Hq - a.Hkv : i - a.Hq;
        const void* src = is_q ? a.q : is_v ? a.v : a.k;
        const long long at = (long long)row * (is_q ? a.qs : is_v ? a.vs : a.ks) + (long long)h * kDim;
        float x[8];
        if (BF) load_bf16x8(static_cast<const uint16_t*>(src) + at, x);
        else load_f32x8(static_cast<const float*>(src) + at, x);
        if (!is_v) rope_apply(x, rr);
        uint16_t* dst = is_q ? a.q_out + ((size_t)row * a.Hq + h) * kDim
                             : (is_v ? a.pv : a.pk) + (((size_t)page * a.Hkv + h) * a.page_n + off) * kDim;
        store_bf16x8(dst, x);
    }
}

}  // namespace

namespace hsq {

hsq_status check_pages(hsq_ctx* ctx, const hsq_pages* pages, bool buffers) {
    if (!ctx) return fail(nullptr, HSQ_ERR_INVALID, "context is NULL");
    if (!pages) return fail(ctx, HSQ_ERR_INVALID, "pages is NULL");
    const int P = pages->page_n;
    if (P != 16 && P != 32 && P != 64 && P != 128) return fail(ctx, HSQ_ERR_INVALID, "page_n must be 16, 32, 64 or 128");
    if (pages->n_pages < 1 || (long long)pages->n_pages * ctx->cfg.n_kv_heads * P >= (1LL << 31))
        return fail(ctx, HSQ_ERR_INVALID, "n_pages out of range");
    if (buffers) {
        if (!pages->k || !pages->v) return fail(ctx, HSQ_ERR_INVALID, "pages->k or pages->v is NULL");
        if (((uintptr_t)pages->k | (uintptr_t)pages->v) & 15u)
            return fail(ctx, HSQ_ERR_INVALID, "pages->k and pages->v must be 16-byte aligned");
    }
    return HSQ_OK;
}

hsq_status check_device(hsq_ctx* ctx) {
    int dev = -1;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(ctx, e, "cudaGetDevice");
    if (dev != ctx->device) return fail(ctx, HSQ_ERR_INVALID, "the current device is not the context's");
    return HSQ_OK;
}

}  // namespace hsq

extern "C" {

hsq_status hsq_page_tables(hsq_ctx* ctx, const hsq_pages* pages, int B, int width, int rows, int n_free, int base,
                           const int32_t* cached, const int32_t* fresh, const int32_t* free_ids,
                           const int32_t* used, int32_t* table, int64_t* slots, int32_t* pos, int32_t* q_start,
                           int32_t* lens, int32_t* used_out, hsq_stream_t stream) {
    hsq_status st = hsq::check_pages(ctx, pages, false);
    if (st != HSQ_OK) return st;
    if (!cached || !fresh || !free_ids || !used || !table || !slots || !pos || !q_start || !lens || !used_out)
        return hsq::fail(ctx, HSQ_ERR_INVALID, "an argument of hsq_page_tables is NULL");
    if (B < 1 || B > ctx->cfg.max_batch || B > HSQ_MAX_REQUESTS)
        return hsq::fail(ctx, HSQ_ERR_INVALID, "B outside [1, min(max_batch, HSQ_MAX_REQUESTS)]");
    if (width < 1 || rows < 1 || n_free < 1 || base < 0)
        return hsq::fail(ctx, HSQ_ERR_INVALID, "width, rows and n_free must be positive, base not negative");
    const void* ins[] = {cached, fresh, free_ids, used};
    const void* outs[] = {table, slots, pos, q_start, lens, used_out};
    for (const void* i : ins)
        for (const void* o : outs)
            if (i == o) return hsq::fail(ctx, HSQ_ERR_INVALID, "an output of hsq_page_tables is one of its inputs");
    if ((st = hsq::check_device(ctx)) != HSQ_OK) return st;
    TablesArgs a{cached, fresh, free_ids, used, table, slots, pos, q_start, lens, used_out,
                 B, width, rows, n_free, base, pages->n_pages, pages->page_n, ctx->d_err};
    const int grid = std::min(2 * ctx->num_sms, (rows + kTabThreads - 1) / kTabThreads);
    page_tables_kernel<<<grid, kTabThreads, 8 * (B + 1), reinterpret_cast<cudaStream_t>(stream)>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? HSQ_OK : hsq::cuda_fail(ctx, e, "page_tables");
}

hsq_status hsq_page_write(hsq_ctx* ctx, const hsq_pages* pages, int rows, const void* q, const void* k, const void* v,
                          int64_t q_stride, int64_t k_stride, int64_t v_stride, hsq_dtype dtype,
                          const int32_t* pos, const int64_t* slots, void* q_out, hsq_stream_t stream) {
    hsq_status st = hsq::check_pages(ctx, pages, true);
    if (st != HSQ_OK) return st;
    if (!k || !v || !pos || !slots) return hsq::fail(ctx, HSQ_ERR_INVALID, "k, v, pos or slots is NULL");
    if (!q != !q_out) return hsq::fail(ctx, HSQ_ERR_INVALID, "q and q_out go together");
    if (dtype != HSQ_DTYPE_F32 && dtype != HSQ_DTYPE_BF16) return hsq::fail(ctx, HSQ_ERR_INVALID, "bad dtype");
    if (rows < 1) return hsq::fail(ctx, HSQ_ERR_INVALID, "rows must be positive");
    const int Hq = q ? ctx->cfg.n_q_heads : 0, Hkv = ctx->cfg.n_kv_heads;
    const int64_t unit = dtype == HSQ_DTYPE_BF16 ? 8 : 4;  // elements of 16 bytes
    if ((q && q_stride < (int64_t)Hq * 128) || k_stride < (int64_t)Hkv * 128 || v_stride < (int64_t)Hkv * 128)
        return hsq::fail(ctx, HSQ_ERR_INVALID, "a row stride is smaller than a row");
    if ((q && q_stride % unit) || k_stride % unit || v_stride % unit ||
        (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)q_out) & 15u))
        return hsq::fail(ctx, HSQ_ERR_INVALID, "rows of q, k, v and q_out must be 16-byte aligned");
    if ((st = hsq::check_device(ctx)) != HSQ_OK) return st;
    const int units = (Hq + 2 * Hkv + kWriteHeads - 1) / kWriteHeads;
    const long long ctas = ((long long)rows * units + kHalves - 1) / kHalves;
    if (ctas > INT_MAX) return hsq::fail(ctx, HSQ_ERR_INVALID, "too many rows");
    WriteArgs a{q, k, v, q_stride, k_stride, v_stride, pos, slots, static_cast<uint16_t*>(q_out),
                static_cast<uint16_t*>(pages->k), static_cast<uint16_t*>(pages->v), rows, Hq, Hkv, pages->n_pages,
                pages->page_n, units, ctx->d_err};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == HSQ_DTYPE_BF16) page_write_kernel<true><<<(int)ctas, kThreads, 0, s>>>(a, make_tables(ctx));
    else page_write_kernel<false><<<(int)ctas, kThreads, 0, s>>>(a, make_tables(ctx));
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? HSQ_OK : hsq::cuda_fail(ctx, e, "page_write");
}

}  // extern "C"
