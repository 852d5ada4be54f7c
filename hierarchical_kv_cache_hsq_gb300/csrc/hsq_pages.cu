// Paged serving: block tables and slot maps from request lengths
// (hsq_page_tables), and the rotated, paged write of a step's keys and values
// (hsq_page_write).
#include <cuda_bf16.h>

#include <algorithm>
#include <climits>
#include <type_traits>

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

// Every CTA scans the lengths itself (B <= 4096: a round of 512 is two loads and ten
// shuffles a thread) and keeps both prefix sums -- rows, pages taken -- and the cached
// lengths in shared memory; then the grid strides over the rows and the new table
// entries, each found by a binary search in them.  So one launch does without any
// exchange between CTAs: nothing that one CTA reads is written by another (a token's
// page is either an old entry of the table or, for a page taken in this call, read
// from the free list itself).  Bound by its latency: launch, length loads, scan,
// search, one more load (6.2 us for 16 decodes, 8.3 us for 256 requests with some prompts among them).
__global__ void __launch_bounds__(kTabThreads) page_tables_kernel(TablesArgs a) {
    extern __shared__ int tab_sm[];
    int* s_row = tab_sm;                 // [B + 1] rows before request b
    int* s_page = s_row + a.B + 1;       // [B + 1] pages taken before request b
    int* s_cached = s_page + a.B + 1;    // [B] cached lengths, checked
    __shared__ uint2 s_w[kTabThreads / 32];
    __shared__ int s_cut, s_cut_pages;   // the request that the end of the rows cuts; pages taken up to its last listed row
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int shift = __ffs(a.page_n) - 1;
    const bool first = blockIdx.x == 0;
    int used = *a.used;
    int bad = 0;
    long long row0 = 0, page0 = 0;  // before the round
    if (tid == 0) s_cut = a.B;
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
            s_cached[b] = c;
        }
        // No page is taken past the table's width; a request's rows saturate just past the rows there are.  (A warp's
        // sums saturate at 2^31 - 1: with a.rows < 2^30 a start of at most a.rows is still exact, and any other stays above.)
        const int xi = min(f, a.rows + 1);
        const int yi = min((c + f + a.page_n - 1) >> shift, a.width) - min((c + a.page_n - 1) >> shift, a.width);
        unsigned x = xi, y = yi;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned u = __shfl_up_sync(kFull, x, o), w = __shfl_up_sync(kFull, y, o);
            if (lane >= o) {
                x = min(x + u, (unsigned)INT_MAX);
                y = min(y + w, (unsigned)INT_MAX);
            }
        }
        if (lane == 31) s_w[warp] = make_uint2(x, y);
        __syncthreads();
        long long tr = row0, tp = page0, X = x, Y = y;
        const int warps = min(kTabThreads, a.B - b0 + 31) >> 5;
        for (int w = 0; w < warps; ++w) {
            if (w == warp) {
                X += tr;
                Y += tp;
            }
            const uint2 v = s_w[w];
            tr += v.x;
            tp += v.y;
        }
        if (b < a.B) {
            // Where the rows end, a request is cut: what has no row counts neither as brought nor as stored (or the
            // attention would take the last listed row for the request's last token, and read keys never written).
            const int start = (int)min(X - xi, (long long)a.rows), listed = min(f, a.rows - start);
            const int page = (int)min(Y - yi, (long long)INT_MAX);
            s_row[b] = start;
            s_page[b] = page;
            if (first) a.lens[b] = c + listed;
            if (listed < f) {
                bad |= HSQ_DEVERR_LEN;
                if (X - xi <= a.rows) {  // the first such request; none after it has a row or a new page
                    const int more = min((c + listed + a.page_n - 1) >> shift, a.width) - min((c + a.page_n - 1) >> shift, a.width);
                    s_cut = b;
                    s_cut_pages = (int)min((long long)page + more, (long long)INT_MAX);
                }
            }
        }
        row0 = tr;
        page0 = tp;
        __syncthreads();
    }
    const int rows = (int)min(row0, (long long)a.rows), cut = s_cut;
    const int pages = cut < a.B ? s_cut_pages : (int)min(page0, (long long)INT_MAX);
    for (int b = cut + 1 + tid; b < a.B; b += kTabThreads) s_page[b] = pages;
    if (tid == 0) {
        s_row[a.B] = rows;
        s_page[a.B] = pages;
    }
    if (used < 0 || used > a.n_free) bad |= HSQ_DEVERR_LEN;
    used = min(max(used, 0), a.n_free);
    if (pages > a.n_free - used) bad |= HSQ_DEVERR_PAGE;
    __syncthreads();
    if (first) {
        for (int b = tid; b <= a.B; b += kTabThreads) a.q_start[b] = s_row[b];
        if (tid == 0) *a.used_out = used + min(pages, a.n_free - used);
    }
    // id of the e-th page taken in this call, -1 when the list is at its end or holds no page of the pool
    auto taken = [&](int e) {
        int id = -1;
        if (e < a.n_free - used) {
            id = a.free_ids[used + e];
            if (id < 0 || id >= a.n_pages) {
                id = -1;
                bad |= HSQ_DEVERR_PAGE;
            }
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
    for (int e = at; e < pages; e += stride) {
        const int b = find(s_page, e);
        const int col = ((s_cached[b] + a.page_n - 1) >> shift) + e - s_page[b];
        if (col < a.width) a.table[(size_t)b * a.width + col] = taken(e);
    }
    for (int i = at; i < a.rows; i += stride) {
        long long slot = -1;
        int pos = -1;
        if (i < rows) {
            const int b = find(s_row, i);
            const int c = s_cached[b];
            const int p = c + i - s_row[b], col = p >> shift, have = (c + a.page_n - 1) >> shift;
            int id = -1;
            if (col < a.width) {
                if (col >= have) {
                    id = taken(s_page[b] + col - have);
                } else {
                    id = a.table[(size_t)b * a.width + col];
                    if (id < 0 || id >= a.n_pages) {
                        id = -1;
                        bad |= HSQ_DEVERR_PAGE;
                    }
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

struct WriteArgs {
    const void *q, *k, *v;
    long long qs, ks, vs;  // elements between rows
    const int32_t* pos; const int64_t* slots;
    uint16_t *q_out, *pk, *pv;
    int rows, Hq, Hkv, page_n, page_shift;
    long long n_slots;
    unsigned units;          // units of a row: V heads each, of the queries, then keys, then values
    int units_q, units_k;
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

// One half-warp per (row, V neighbouring heads of its queries, keys or values): all V
// vectors' loads first, then the row's position, slot, cos and sin (one set for the V
// vectors), then rotate, round, store.  A unit has one kind of vectors, so that its
// pointers are two bases and two strides (with the kind chosen vector by vector, address arithmetic
// took half of the issue slots).  Bound by HBM for many rows, where reads and writes in flight
// decide: a prompt of 32K tokens (32/8 heads, bf16, 806 MB) takes 121 us, 6.7 TB/s, 99 % of a plain copy's rate; with V = 1,
// fewer loads in flight, 185.  For few rows by latency, and V = 1 spreads them over the SMs: 16 rows 4.2 us, with
// V = 8 5.5.  (2531 float32 rows: 25.2 with V = 1, 23.7 with V = 4.)
template <bool BF, int V>
__global__ void __launch_bounds__(kThreads) page_write_kernel(WriteArgs a, Tables tb) {
    using Raw = typename std::conditional<BF, uint2, float4>::type;  // a lane's dims 4 l .. and 64 + 4 l ..
    constexpr int kSize = BF ? 2 : 4;
    const int l = hlane();
    const unsigned unit = blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4);
    const unsigned row_u = unit / a.units;
    const int row = (int)row_u, u = (int)(unit - row_u * a.units);
    if (row >= a.rows) return;
    const bool is_q = u < a.units_q, is_v = u >= a.units_q + a.units_k;
    const int h0 = (is_q ? u : is_v ? u - a.units_q - a.units_k : u - a.units_q) * V;
    const int count = min(V, (is_q ? a.Hq : a.Hkv) - h0);
    const char* src = static_cast<const char*>(is_q ? a.q : is_v ? a.v : a.k) +
                      ((long long)row * (is_q ? a.qs : is_v ? a.vs : a.ks) + h0 * kDim) * kSize + l * sizeof(Raw);
    Raw raw[V][2];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if (j < count) {
            raw[j][0] = __ldg(reinterpret_cast<const Raw*>(src + j * (kDim * kSize)));
            raw[j][1] = __ldg(reinterpret_cast<const Raw*>(src + j * (kDim * kSize) + 64 * kSize));
        }
    }
    int p = a.pos[row];
    long long slot = a.slots[row];
    if (p < 0) return;
    if (p >= tb.max_pos) {
        p = tb.max_pos - 1;
        if (l == 0) atomicOr(a.err, HSQ_DEVERR_POS);
    }
    if (slot >= a.n_slots) {
        slot = -1;
        if (l == 0) atomicOr(a.err, HSQ_DEVERR_PAGE);
    }
    if (!is_q && slot < 0) return;
    uint16_t* dst;
    int step = kDim;  // elements between the unit's heads
    if (is_q) {
        dst = a.q_out + ((size_t)row * a.Hq + h0) * kDim;
    } else {
        step = a.page_n * kDim;
        dst = (is_v ? a.pv : a.pk) +
              (((size_t)(slot >> a.page_shift) * a.Hkv + h0) * a.page_n + (size_t)(slot & (a.page_n - 1))) * kDim;
    }
    RopeRows rr;
    if (!is_v) rr = rope_rows(p, tb);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if (j >= count) break;
        if (BF && is_v) {
            reinterpret_cast<Raw*>(dst + (size_t)j * step)[l] = raw[j][0];
            reinterpret_cast<Raw*>(dst + (size_t)j * step + 64)[l] = raw[j][1];
            continue;
        }
        float x[8];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if constexpr (BF) {
                x[4 * e] = __uint_as_float(raw[j][e].x << 16);
                x[4 * e + 1] = __uint_as_float(raw[j][e].x & 0xFFFF0000u);
                x[4 * e + 2] = __uint_as_float(raw[j][e].y << 16);
                x[4 * e + 3] = __uint_as_float(raw[j][e].y & 0xFFFF0000u);
            } else {
                x[4 * e] = raw[j][e].x;
                x[4 * e + 1] = raw[j][e].y;
                x[4 * e + 2] = raw[j][e].z;
                x[4 * e + 3] = raw[j][e].w;
            }
        }
        if (!is_v) rope_apply(x, rr);
        store_bf16x8(dst + (size_t)j * step, x);
    }
}

template <bool BF, int V>
void launch_write(WriteArgs a, const Tables& tb, cudaStream_t s) {
    a.units_q = (a.Hq + V - 1) / V;
    a.units_k = (a.Hkv + V - 1) / V;
    a.units = a.units_q + 2 * a.units_k;
    const unsigned ctas = (unsigned)(((unsigned long long)a.rows * a.units + kHalves - 1) / kHalves);
    page_write_kernel<BF, V><<<ctas, kThreads, 0, s>>>(a, tb);
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
    // (past 2^30 the kernel's sums and its strides over rows and pages no longer fit 32 bits)
    if (width < 1 || rows < 1 || rows >= kMaxLen || n_free < 1 || n_free >= kMaxLen || base < 0 || base >= kMaxLen)
        return hsq::fail(ctx, HSQ_ERR_INVALID, "width must be positive, rows and n_free in [1, 2^30), base in [0, 2^30)");
    const size_t n = 4 * (size_t)B;
    const hsq::Span ins[] = {{cached, n}, {fresh, n}, {free_ids, 4 * (size_t)n_free}, {used, 4}};
    const hsq::Span outs[] = {{table, n * width}, {slots, 8 * (size_t)rows}, {pos, 4 * (size_t)rows}, {q_start, n + 4}, {lens, n}, {used_out, 4}};
    if (hsq::outputs_overlap(ins, outs))
        return hsq::fail(ctx, HSQ_ERR_INVALID, "an output of hsq_page_tables overlaps another argument");
    if ((st = hsq::check_device(ctx)) != HSQ_OK) return st;
    TablesArgs a{cached, fresh, free_ids, used, table, slots, pos, q_start, lens, used_out,
                 B, width, rows, n_free, base, pages->n_pages, pages->page_n, ctx->d_err};
    const int grid = std::min(2 * ctx->num_sms, (rows + kTabThreads - 1) / kTabThreads);
    const size_t smem = 4 * (3 * (size_t)B + 2);
    cudaError_t e = hsq::raise_smem_limit((const void*)page_tables_kernel, ctx->device, smem);
    if (e != cudaSuccess) return hsq::cuda_fail(ctx, e, "cudaFuncSetAttribute(page_tables)");
    page_tables_kernel<<<grid, kTabThreads, smem, reinterpret_cast<cudaStream_t>(stream)>>>(a);
    e = cudaGetLastError();
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
    const long long vectors = (long long)rows * (Hq + 2 * Hkv);
    if (vectors >= (1LL << 31)) return hsq::fail(ctx, HSQ_ERR_INVALID, "too many rows");
    const size_t size = dtype == HSQ_DTYPE_BF16 ? 2 : 4, pool = (size_t)pages->n_pages * Hkv * pages->page_n * 256;
    auto strided = [&](const void* p, int64_t stride, int heads) {
        return hsq::Span{p, ((size_t)(rows - 1) * stride + (size_t)heads * 128) * size};
    };
    const hsq::Span ins[] = {strided(q, q_stride, Hq), strided(k, k_stride, Hkv), strided(v, v_stride, Hkv),
                             {pos, 4 * (size_t)rows}, {slots, 8 * (size_t)rows}};
    const hsq::Span outs[] = {{q_out, (size_t)rows * Hq * 256}, {pages->k, pool}, {pages->v, pool}};
    if (hsq::outputs_overlap(ins, outs))
        return hsq::fail(ctx, HSQ_ERR_INVALID, "q_out or the pool's k or v overlaps another argument of hsq_page_write");
    if ((st = hsq::check_device(ctx)) != HSQ_OK) return st;
    const int shift = pages->page_n == 16 ? 4 : pages->page_n == 32 ? 5 : pages->page_n == 64 ? 6 : 7;
    WriteArgs a{q, k, v, q_stride, k_stride, v_stride, pos, slots, static_cast<uint16_t*>(q_out),
                static_cast<uint16_t*>(pages->k), static_cast<uint16_t*>(pages->v), rows, Hq, Hkv, pages->page_n, shift,
                (long long)pages->n_pages * pages->page_n, 0, 0, 0, ctx->d_err};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const Tables tb = make_tables(ctx);
    // one vector a half-warp until the GPU's warps (32 a SM) are all in use, then as many as fit its registers
    const bool few = vectors <= 64LL * ctx->num_sms;
    if (dtype == HSQ_DTYPE_BF16) {
        if (few) launch_write<true, 1>(a, tb, s);
        else launch_write<true, 8>(a, tb, s);
    } else {
        if (few) launch_write<false, 1>(a, tb, s);
        else launch_write<false, 4>(a, tb, s);
    }
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? HSQ_OK : hsq::cuda_fail(ctx, e, "page_write");
}

}  // extern "C"
