// Paged serving: block tables and slot maps from request lengths
// (hsq_page_tables), the rotated, paged write of a step's keys and values
// (hsq_page_write, and with a model's own rotation hsq_page_write_rope), and
// the summaries of the pages that a step fills (hsq_page_summaries).
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
    const float* rope;       // hsq_rope's table, row length and limit (with the context's rotation not read)
    int rope_dims, rope_pos;
    int* err;
};

// What turns a half-warp's vectors.  kOwnRope: the context's rotation.  Else the first `dims` dims by hsq_rope's
// table, in pairs (i, i + dims / 2) (kHalfRope) or (2 i, 2 i + 1) (kPairRope).  A table costs no time over the
// context's rotation.
enum { kOwnRope, kHalfRope, kPairRope };

// The two quads of dims that lane l holds: what it turns lies in its own registers (pair k of it has frequency 4 l +
// k), and lanes past the rotated dims hold those left as they are.
template <int ROPE>
__device__ __forceinline__ void lane_quads(int l, int dims, int& qa, int& qb) {
    if (ROPE == kOwnRope) {
        qa = 4 * l;
        qb = 64 + 4 * l;
    } else if (ROPE == kPairRope || 8 * l >= dims) {
        qa = 8 * l;
        qb = 8 * l + 4;
    } else {
        qa = 4 * l;
        qb = (dims >> 1) + 4 * l;
    }
}

template <int ROPE>
__device__ __forceinline__ RopeRows rope_rows_of(int p, const WriteArgs& a, const Tables& tb) {
    if constexpr (ROPE == kOwnRope) {
        return rope_rows(p, tb);
    } else {
        RopeRows r{};
        const int l = hlane(), half = a.rope_dims >> 1;
        if (8 * l < a.rope_dims) {
            const float* lo = a.rope + (p & 255) * a.rope_dims + 4 * l;
            const float* hi = a.rope + (size_t)(256 + (p >> 8)) * a.rope_dims + 4 * l;
            r.cl = __ldg(reinterpret_cast<const float4*>(lo));
            r.sl = __ldg(reinterpret_cast<const float4*>(lo + half));
            r.ch = __ldg(reinterpret_cast<const float4*>(hi));
            r.sh = __ldg(reinterpret_cast<const float4*>(hi + half));
        }
        return r;
    }
}

template <int ROPE>
__device__ __forceinline__ void turn(float (&x)[8], const RopeRows& r, int dims) {
    if (ROPE == kOwnRope) {
        rope_apply(x, r);
    } else if (8 * hlane() < dims) {
        if (ROPE == kHalfRope) {
            rope_apply(x, r);
        } else {  // the pairs side by side: (0, 1), (2, 3), ..
            float y[8] = {x[0], x[2], x[4], x[6], x[1], x[3], x[5], x[7]};
            rope_apply(y, r);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                x[2 * k] = y[k];
                x[2 * k + 1] = y[4 + k];
            }
        }
    }
}

__device__ __forceinline__ void store_bf16x8(uint16_t* pa, uint16_t* pb, const float v[8]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    const __nv_bfloat162 c = __floats2bfloat162_rn(v[4], v[5]), d = __floats2bfloat162_rn(v[6], v[7]);
    *reinterpret_cast<uint2*>(pa) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    *reinterpret_cast<uint2*>(pb) = make_uint2(*reinterpret_cast<const uint32_t*>(&c), *reinterpret_cast<const uint32_t*>(&d));
}

// One half-warp per (row, V neighbouring heads of its queries, keys or values): all V
// vectors' loads first, then the row's position, slot, cos and sin (one set for the V
// vectors), then rotate, round, store.  A unit has one kind of vectors, so that its
// pointers are two bases and two strides (with the kind chosen vector by vector, address arithmetic
// took half of the issue slots).  Bound by HBM for many rows, where reads and writes in flight
// decide: a prompt of 32K tokens (32/8 heads, bf16, 806 MB) takes 121 us, 6.7 TB/s, 99 % of a plain copy's rate;
// with V = 1, fewer loads in flight, 187.  For few rows by latency, and V = 1 spreads them over the SMs: 16 rows 2.0
// us, with V = 8 2.9.  (2531 float32 rows: 20.1 with V = 1, 17.1 with V = 4.  Replayed from a graph, the inputs in L2
// where they fit; with other inputs in turn 16 rows take 4.2.)
template <bool BF, int V, int ROPE>
__global__ void __launch_bounds__(kThreads) page_write_kernel(WriteArgs a, Tables tb) {
    using Raw = typename std::conditional<BF, uint2, float4>::type;  // a quad of dims
    constexpr int kSize = BF ? 2 : 4;
    const int l = hlane();
    int qa, qb;
    lane_quads<ROPE>(l, a.rope_dims, qa, qb);
    const unsigned unit = blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4);
    const unsigned row_u = unit / a.units;
    const int row = (int)row_u, u = (int)(unit - row_u * a.units);
    if (row >= a.rows) return;
    const bool is_q = u < a.units_q, is_v = u >= a.units_q + a.units_k;
    const int h0 = (is_q ? u : is_v ? u - a.units_q - a.units_k : u - a.units_q) * V;
    const int count = min(V, (is_q ? a.Hq : a.Hkv) - h0);
    const char* src = static_cast<const char*>(is_q ? a.q : is_v ? a.v : a.k) +
                      ((long long)row * (is_q ? a.qs : is_v ? a.vs : a.ks) + h0 * kDim) * kSize;
    Raw raw[V][2];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if (j < count) {
            raw[j][0] = __ldg(reinterpret_cast<const Raw*>(src + j * (kDim * kSize) + qa * kSize));
            raw[j][1] = __ldg(reinterpret_cast<const Raw*>(src + j * (kDim * kSize) + qb * kSize));
        }
    }
    int p = a.pos[row];
    long long slot = a.slots[row];
    if (p < 0) return;
    const int max_pos = ROPE == kOwnRope ? tb.max_pos : a.rope_pos;
    if (p >= max_pos) {
        p = max_pos - 1;
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
    if (!is_v) rr = rope_rows_of<ROPE>(p, a, tb);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if (j >= count) break;
        if (BF && is_v) {
            *reinterpret_cast<Raw*>(dst + (size_t)j * step + qa) = raw[j][0];
            *reinterpret_cast<Raw*>(dst + (size_t)j * step + qb) = raw[j][1];
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
        if (!is_v) turn<ROPE>(x, rr, a.rope_dims);
        store_bf16x8(dst + (size_t)j * step + qa, dst + (size_t)j * step + qb, x);
    }
}

template <bool BF, int V, int ROPE>
void launch_write(WriteArgs a, const Tables& tb, cudaStream_t s) {
    a.units_q = (a.Hq + V - 1) / V;
    a.units_k = (a.Hkv + V - 1) / V;
    a.units = a.units_q + 2 * a.units_k;
    const unsigned ctas = (unsigned)(((unsigned long long)a.rows * a.units + kHalves - 1) / kHalves);
    page_write_kernel<BF, V, ROPE><<<ctas, kThreads, 0, s>>>(a, tb);
}

template <int ROPE>
void launch_write(const WriteArgs& a, bool bf, bool few, const Tables& tb, cudaStream_t s) {
    if (bf) {
        if (few) launch_write<true, 1, ROPE>(a, tb, s);
        else launch_write<true, 8, ROPE>(a, tb, s);
    } else {
        if (few) launch_write<false, 1, ROPE>(a, tb, s);
        else launch_write<false, 4, ROPE>(a, tb, s);
    }
}

// ---- summaries ------------------------------------------------------------------------------

struct SumsArgs {
    const int64_t* slots;
    const uint16_t* pk;
    int8_t* codes; float* scale;
    int rows, Hkv, page_n, page_shift, n_pages;
    int* err;
};

// s + x exactly as the two numbers s (rounded) and what the rounding left out, added to e; two lanes at a time.
__device__ __forceinline__ void two_sum2(uint64_t& s, uint64_t& e, uint64_t x) {
    uint64_t t, b, c, d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(t) : "l"(s), "l"(x));
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(b) : "l"(t), "l"(s));
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(c) : "l"(t), "l"(b));
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(c) : "l"(s), "l"(c));
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(b));
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(c) : "l"(c), "l"(d));
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(e) : "l"(e), "l"(c));
    s = t;
}

constexpr int kSumThreads = 256;
constexpr float kSumLeast = 0x1p-64f, kSumMost = 0x1p126f;

// One warp per (R rows of the step, KV head): a row is its page's last of the step when the next row's slot lies on
// another page, and then the warp sums the page's keys.  A half-warp takes every other token (16 bytes, dims 8 l ..
// 8 l + 7, a lane), 8 tokens a time, the next 8 on their way meanwhile.
// The sums are kept as fp32 pairs (two_sum2), exact to some 48 bits, because a code jumps by one at a border and has to
// be the same however the sum is ordered; 127 S / max is compared with its border in 64 bits only where fp32 leaves it
// open (one element in 5000).  Bound by HBM and, at both ends, latency: the pages of 32K tokens (8 heads, 67 MB)
// take 15 us, 4.5 TB/s over the whole of it; those of 16 decodes 4.4 us, launch and two dependent loads.
template <int R>
__global__ void __launch_bounds__(kSumThreads, 3) page_summaries_kernel(SumsArgs a) {
    const int lane = threadIdx.x & 31, l = lane & 15, odd = lane >> 4;
    const long long unit = (long long)blockIdx.x * (kSumThreads / 32) + (threadIdx.x >> 5);
    const long long chunk = unit / a.Hkv;
    const int h = (int)(unit - chunk * a.Hkv);
    constexpr int kWords = (R + 31) / 32;  // 32 rows a look
    for (int k = 0; k < kWords; ++k) {
        const long long row = chunk * R + 32 * k + lane;
        long long slot = -1;
        bool last = false;
        if (32 * k + lane < R && row < a.rows) {
            slot = a.slots[row];
            const long long after = row + 1 < a.rows ? a.slots[row + 1] : -1;
            if (slot >= (long long)a.n_pages << a.page_shift) {
                slot = -1;
                if (h == 0) atomicOr(a.err, HSQ_DEVERR_PAGE);
            }
            last = slot >= 0 && (after < 0 || (after >> a.page_shift) != (slot >> a.page_shift));
        }
        unsigned todo = __ballot_sync(kFull, last);
        while (todo) {
            const int from = __ffs(todo) - 1;
            todo &= todo - 1;
            const long long at = __shfl_sync(kFull, slot, from);
            const int page = (int)(at >> a.page_shift), n = (int)(at & (a.page_n - 1)) + 1;
            const size_t head = (size_t)page * a.Hkv + h;
            const uint4* src = reinterpret_cast<const uint4*>(a.pk + (head << a.page_shift) * kDim) + odd * 16 + l;
            uint64_t s[4] = {0, 0, 0, 0}, e[4] = {0, 0, 0, 0};
            uint4 v[4];
            auto load = [&](int t0) {
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = t0 + 2 * k + odd < n ? __ldcs(src + (size_t)(t0 + 2 * k) * 16) : make_uint4(0, 0, 0, 0);
            };
            load(0);
#pragma unroll 1
            for (int t0 = 0; t0 < n; t0 += 8) {
                uint4 u[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) u[k] = v[k];
                if (t0 + 8 < n) load(t0 + 8);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        two_sum2(s[i], e[i], (uint64_t)(w[i] << 16) | ((uint64_t)(w[i] & 0xFFFF0000u) << 32));
                }
            }
            float hi[8], lo[8];
            float top = 0.f;
            bool bad = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // the two halves' sums, and the pair brought to hi = their sum rounded
                const uint64_t so = __shfl_xor_sync(kFull, s[i], 16), eo = __shfl_xor_sync(kFull, e[i], 16);
                uint64_t a2 = odd ? so : s[i], b2 = odd ? s[i] : so, r2;  // (in one order, so that both halves get the same)
                asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r2) : "l"(e[i]), "l"(eo));
                two_sum2(a2, r2, b2);
                const float x[2] = {__uint_as_float((uint32_t)a2), __uint_as_float((uint32_t)(a2 >> 32))};
                const float y[2] = {__uint_as_float((uint32_t)r2), __uint_as_float((uint32_t)(r2 >> 32))};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    hi[2 * i + k] = __fadd_rn(x[k], y[k]);
                    lo[2 * i + k] = __fsub_rn(y[k], __fsub_rn(hi[2 * i + k], x[k]));
                    top = fmaxf(top, fabsf(hi[2 * i + k]));
                    bad |= !(fabsf(hi[2 * i + k]) <= kSumMost);
                }
            }
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
            bad = __any_sync(kFull, bad);
            const bool live = !bad && top >= kSumLeast;
            const float by = __fdiv_rn(127.f, live ? top : 1.f);
            int code[8];
            bool open = false;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float y = __fmul_rn(hi[k], by);
                code[k] = live ? __float2int_rn(y) : 0;
                open |= live && fabsf(fabsf(y - rintf(y)) - 0.5f) < 1e-4f;
            }
            if (__any_sync(kFull, open)) {  // (y is off by less than 127 * 2^-22 here)
                float rest = -INFINITY;  // what the largest sum has beyond top
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (fabsf(hi[k]) == top) rest = fmaxf(rest, hi[k] < 0.f ? -lo[k] : lo[k]);
#pragma unroll
                for (int d = 1; d < 16; d <<= 1) rest = fmaxf(rest, __shfl_xor_sync(kFull, rest, d));
                const double m = (double)top + (double)rest;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float y = __fmul_rn(hi[k], by);
                    if (fabsf(fabsf(y - rintf(y)) - 0.5f) < 1e-4f) code[k] = __double2int_rn(127.0 * ((double)hi[k] + lo[k]) / m);
                }
            }
            if (odd == 0) {
                uint32_t w[2] = {0, 0};
#pragma unroll
                for (int k = 0; k < 8; ++k) w[k >> 2] |= (uint32_t)(code[k] & 0xFF) << (8 * (k & 3));
                reinterpret_cast<uint2*>(a.codes + head * kDim)[l] = make_uint2(w[0], w[1]);
                if (l == 0) a.scale[head] = live ? __fdiv_rn(top, 127.f * (float)n) : bad ? INFINITY : 0.f;
            }
        }
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

hsq_status check_summaries(hsq_ctx* ctx, const hsq_summaries* sums) {
    if (!sums || !sums->codes || !sums->scale) return fail(ctx, HSQ_ERR_INVALID, "sums, sums->codes or sums->scale is NULL");
    if (((uintptr_t)sums->codes & 15u) || ((uintptr_t)sums->scale & 3u))
        return fail(ctx, HSQ_ERR_INVALID, "sums->codes must be 16-byte aligned, sums->scale 4-byte");
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

namespace {

// hsq_page_write (rope NULL) and hsq_page_write_rope
hsq_status page_write(hsq_ctx* ctx, const hsq_pages* pages, const hsq_rope* rope, int rows, const void* q, const void* k,
                      const void* v, int64_t q_stride, int64_t k_stride, int64_t v_stride, hsq_dtype dtype,
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
    size_t rope_floats = 0;
    if (rope) {
        if (!rope->table || ((uintptr_t)rope->table & 15u))
            return hsq::fail(ctx, HSQ_ERR_INVALID, "rope->table must be 16-byte aligned and not NULL");
        if (hsq_rope_table(rope->dims, nullptr, 1.0, rope->max_pos, nullptr, &rope_floats) != HSQ_OK)
            return hsq::fail(ctx, HSQ_ERR_INVALID, "rope->dims must be a multiple of 8 in [8, 128], max_pos in [1, 2^24]");
        if (rope->interleaved != 0 && rope->interleaved != 1) return hsq::fail(ctx, HSQ_ERR_INVALID, "rope->interleaved must be 0 or 1");
    }
    const size_t size = dtype == HSQ_DTYPE_BF16 ? 2 : 4, pool = (size_t)pages->n_pages * Hkv * pages->page_n * 256;
    auto strided = [&](const void* p, int64_t stride, int heads) {
        return hsq::Span{p, ((size_t)(rows - 1) * stride + (size_t)heads * 128) * size};
    };
    const hsq::Span ins[] = {strided(q, q_stride, Hq), strided(k, k_stride, Hkv), strided(v, v_stride, Hkv),
                             {pos, 4 * (size_t)rows}, {slots, 8 * (size_t)rows}, {rope ? rope->table : nullptr, 4 * rope_floats}};
    const hsq::Span outs[] = {{q_out, (size_t)rows * Hq * 256}, {pages->k, pool}, {pages->v, pool}};
    if (hsq::outputs_overlap(ins, outs))
        return hsq::fail(ctx, HSQ_ERR_INVALID, "q_out or the pool's k or v overlaps another argument of hsq_page_write");
    if ((st = hsq::check_device(ctx)) != HSQ_OK) return st;
    const int shift = pages->page_n == 16 ? 4 : pages->page_n == 32 ? 5 : pages->page_n == 64 ? 6 : 7;
    WriteArgs a{q, k, v, q_stride, k_stride, v_stride, pos, slots, static_cast<uint16_t*>(q_out),
                static_cast<uint16_t*>(pages->k), static_cast<uint16_t*>(pages->v), rows, Hq, Hkv, pages->page_n, shift,
                (long long)pages->n_pages * pages->page_n, 0, 0, 0, rope ? rope->table : nullptr, rope ? rope->dims : 0,
                rope ? rope->max_pos : 0, ctx->d_err};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const Tables tb = make_tables(ctx);
    // one vector a half-warp until the GPU's warps (32 a SM) are all in use, then as many as fit its registers
    const bool few = vectors <= 64LL * ctx->num_sms;
    const bool bf = dtype == HSQ_DTYPE_BF16;
    if (!rope) launch_write<kOwnRope>(a, bf, few, tb, s);
    else if (rope->interleaved) launch_write<kPairRope>(a, bf, few, tb, s);
    else launch_write<kHalfRope>(a, bf, few, tb, s);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? HSQ_OK : hsq::cuda_fail(ctx, e, "page_write");
}

}  // namespace

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
    return page_write(ctx, pages, nullptr, rows, q, k, v, q_stride, k_stride, v_stride, dtype, pos, slots, q_out, stream);
}

hsq_status hsq_page_write_rope(hsq_ctx* ctx, const hsq_pages* pages, const hsq_rope* rope, int rows, const void* q,
                               const void* k, const void* v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                               hsq_dtype dtype, const int32_t* pos, const int64_t* slots, void* q_out, hsq_stream_t stream) {
    if (!rope) return hsq::fail(ctx, HSQ_ERR_INVALID, "rope is NULL");
    return page_write(ctx, pages, rope, rows, q, k, v, q_stride, k_stride, v_stride, dtype, pos, slots, q_out, stream);
}

hsq_status hsq_page_summaries(hsq_ctx* ctx, const hsq_pages* pages, const hsq_summaries* sums, int rows,
                              const int64_t* slots, hsq_stream_t stream) {
    hsq_status st = hsq::check_pages(ctx, pages, true);
    if (st != HSQ_OK) return st;
    if ((st = hsq::check_summaries(ctx, sums)) != HSQ_OK) return st;
    if (!slots) return hsq::fail(ctx, HSQ_ERR_INVALID, "slots is NULL");
    if (rows < 1 || rows >= kMaxLen) return hsq::fail(ctx, HSQ_ERR_INVALID, "rows must be in [1, 2^30)");
    const int Hkv = ctx->cfg.n_kv_heads, P = pages->page_n;
    const size_t heads = (size_t)pages->n_pages * Hkv;
    const hsq::Span ins[] = {{slots, 8 * (size_t)rows}, {pages->k, heads * P * 256}};
    const hsq::Span outs[] = {{sums->codes, heads * 128}, {sums->scale, heads * 4}};
    if (hsq::outputs_overlap(ins, outs))
        return hsq::fail(ctx, HSQ_ERR_INVALID, "the summaries overlap another argument of hsq_page_summaries");
    if ((st = hsq::check_device(ctx)) != HSQ_OK) return st;
    const int shift = P == 16 ? 4 : P == 32 ? 5 : P == 64 ? 6 : 7;
    SumsArgs a{slots, static_cast<const uint16_t*>(pages->k), sums->codes, sums->scale, rows, Hkv, P, shift, pages->n_pages,
               ctx->d_err};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // a row a warp until the GPU's warps (64 a SM) are in use twice over, then 64: a prompt's rows fill pages of up to 128
    const long long units = (long long)rows * Hkv;
    const bool few = units <= 128LL * ctx->num_sms;
    const long long warps = few ? units : (long long)((rows + 63) / 64) * Hkv;
    const unsigned ctas = (unsigned)((warps + kSumThreads / 32 - 1) / (kSumThreads / 32));
    if (few) page_summaries_kernel<1><<<ctas, kSumThreads, 0, s>>>(a);
    else page_summaries_kernel<64><<<ctas, kSumThreads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? HSQ_OK : hsq::cuda_fail(ctx, e, "page_summaries");
}

}  // extern "C"
