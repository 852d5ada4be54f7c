// Selection of pages by a cheap score (hsq_page_select).
//
// For row i of request b and KV head h, with cq the 8-bit codes of the sum of the head's query rows and
// codes, scale the summary of page p:  score_p = (sum_d cq_d codes_pd) scale_p.  The sum is a whole number below 2^21,
// exact in every order of summation, and the product one rounding, so the selection does not depend on how the work is
// divided.  Taken are the first pages, the row's last ones, and the best of the others, ties to the lower page.
#include <cooperative_groups.h>

#include <algorithm>

#include "hsq_ctx.h"
#include "hsq_paged.cuh"

namespace {

using namespace hsq_paged;
namespace cg = cooperative_groups;

struct SelectArgs {
    const uint16_t* q;
    const int32_t *q_start, *lens, *table, *prefix;
    const int8_t* codes; const float* scale;
    int32_t* sel;
    int rows, B, width, prefix_pages, max_new, n_pages, page_n, page_shift, Hq, Hkv, r, top, first, recent;
    int* err;
};

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

// ---------------------------------------------------------------------------------------
// Rows one by one (decode, proposals): a cluster of CTAs for each (row, KV head).  Its CTAs score a share of the pages each,
// eight lanes a page (16 bytes each, so a warp's load is four whole lines), and leave the keys in the first CTA's
// shared memory, which selects.
// ---------------------------------------------------------------------------------------

constexpr int kRowThreads = 512;

__global__ void __launch_bounds__(kRowThreads) page_select_rows_kernel(const __grid_constant__ SelectArgs a) {
    extern __shared__ uint32_t s_keys[];
    __shared__ SelectSmem ss;
    __shared__ uint32_t s_q[32];
    __shared__ int s_row[3];
    __shared__ int s_out[HSQ_MAX_BETA];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    cg::cluster_group cluster = cg::this_cluster();
    const int S = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int unit = blockIdx.x / S, h = unit % a.Hkv, row = unit / a.Hkv;
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");
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
    if (blockIdx.x == 0) bad |= offsets_bad(a.q_start, a.B, a.rows, kRowThreads);
    __syncthreads();
    asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");  // every CTA of the cluster runs: remote stores may start
    const bool live = s_row[2];
    const int b = s_row[0], c = a.prefix_pages + ((s_row[1] + a.page_n - 1) >> a.page_shift);
    const int G = c - a.first - a.recent, beta = a.top - a.first - a.recent;
    const bool score = live && c > a.top && beta > 0;
    if (score) {
        uint32_t* keys = cluster.map_shared_rank(s_keys, 0);
        const uint4 cq = reinterpret_cast<const uint4*>(s_q)[lane & 7];
        const int g1 = (int)((long long)G * (rank + 1) / S);
        for (int i0 = (int)((long long)G * rank / S) + warp * 32; i0 < g1; i0 += kRowThreads) {
            const int i = i0 + lane, p = a.first + i;
            int id = -1;
            if (i < g1) {
                id = p < a.prefix_pages ? a.prefix[p] : a.table[(size_t)b * a.width + p - a.prefix_pages];
                if (id < 0 || id >= a.n_pages) {
                    id = -1;
                    bad |= HSQ_DEVERR_PAGE;
                }
            }
            const float scale = id >= 0 ? a.scale[(size_t)id * a.Hkv + h] : 0.f;
            uint4 m[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {  // four pages at a time
                const int of = __shfl_sync(kFull, id, 4 * k + (lane >> 3));
                m[k] = make_uint4(0, 0, 0, 0);
                if (of >= 0) m[k] = __ldg(reinterpret_cast<const uint4*>(a.codes + ((size_t)of * a.Hkv + h) * 128 + 16 * (lane & 7)));
            }
            int mine = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                int dot = __dp4a((int)m[k].x, (int)cq.x, 0);
                dot = __dp4a((int)m[k].y, (int)cq.y, dot);
                dot = __dp4a((int)m[k].z, (int)cq.z, dot);
                dot = __dp4a((int)m[k].w, (int)cq.w, dot);
#pragma unroll
                for (int d = 1; d < 8; d <<= 1) dot += __shfl_xor_sync(kFull, dot, d);
                const int got = __shfl_sync(kFull, dot, 8 * (lane & 3));
                if ((lane >> 2) == k) mine = got;
            }
            if (i < g1) keys[i] = id >= 0 ? score_key(mine, scale) : 0u;
        }
    }
    cluster.sync();  // the keys are in the first CTA; no remote access follows
    if (rank == 0 && live) {
        int32_t* out = a.sel + ((size_t)row * a.Hkv + h) * a.top;
        if (c <= a.top) {
            for (int i = tid; i < a.top; i += kRowThreads) out[i] = i < c ? i : -1;
        } else {
            if (score) {
                select_top_beta<kRowThreads>(s_keys, G, beta, s_out, ss);
                __syncthreads();
            }
            // the first pages, the selected ones and the last ones (which move up where fewer could be selected)
            for (int i = tid; i < a.first; i += kRowThreads) out[i] = i;
            const bool got = tid < beta && s_out[tid] >= 0;
            if (got) out[a.first + tid] = a.first + s_out[tid];
            const int n = a.first + __syncthreads_count(got);
            for (int i = tid; i < a.recent; i += kRowThreads) out[n + i] = c - a.recent + i;
            for (int i = n + a.recent + tid; i < a.top; i += kRowThreads) out[i] = -1;
        }
    }
    if (bad) atomicOr(a.err, bad);
}
static_assert(kRowThreads >= HSQ_MAX_BETA, "an entry a thread");

// ---------------------------------------------------------------------------------------
// Rows by tiles of 16 of one request (prompts' chunks): a CTA for each (tile, KV head) goes over the pages in chunks of 1024.
//   Scores by tensor-core products of whole numbers in fp16 (exact: |code| <= 127, sums below 2^21 in fp32): 16 rows (A, in
//   registers) x 8 pages (B).  The dims are taken in an order that gives a lane 32 neighbouring bytes of a page's codes.
//   Selection by a warp a row, the chunk's keys in its registers beside the best so far: from the largest key down by doubled
//   steps until enough keys lie above, then halving until exactly as many do (or keys tie).
// ---------------------------------------------------------------------------------------

constexpr int kTileThreads = 256, kTileRow = 16, kChunk = 1024, kPitch = kChunk + 4, kCandRegs = HSQ_MAX_BETA / 32;

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&x)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};\n"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(b0), "r"(b1));
}

// Four int8 codes as two pairs of fp16: 1024 + (code + 128) has the biased code as its last bits, less 1152 it is the code.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    w ^= 0x80808080u;
    const uint32_t x = __byte_perm(w, 0x64646464u, 0x4140), y = __byte_perm(w, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(x), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(y), "r"(0x64806480u));
}

__global__ void __launch_bounds__(kTileThreads) page_select_tiles_kernel(const __grid_constant__ SelectArgs a) {
    extern __shared__ uint32_t s_dyn[];
    uint32_t* s_key = s_dyn;                                // [16][kPitch] the chunk's keys
    const int beta = a.top - a.first - a.recent;
    uint32_t* s_best = s_key + kTileRow * kPitch;           // [16][beta] the best so far, in the pages' order: key,
    int* s_page = reinterpret_cast<int*>(s_best + kTileRow * max(beta, 0));  // page
    __shared__ uint32_t s_q[kTileRow][32];
    __shared__ int s_scan[kTileThreads / 32];
    __shared__ int s_at[5];   // request, first row, rows, rows before it in the request's own count, own tokens held
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int unit = blockIdx.x / a.Hkv, h = blockIdx.x - unit * a.Hkv;
    int bad = 0;
    if (tid == 0) s_at[2] = 0;
    __syncthreads();
    int before = 0;
    for (int b0 = 0; b0 < a.B && before <= unit; b0 += kTileThreads) {
        const int b = b0 + tid;
        int s = 0, n = 0, l = 0, held = 0;
        if (b < a.B) {
            const int e = a.q_start[b + 1];
            s = a.q_start[b];
            l = a.lens[b];
            if (s < 0 || e < s || e > a.rows || e - s > a.max_new) bad |= HSQ_DEVERR_LEN;
            else n = e - s;
            held = min(max(l, 0), a.width << a.page_shift);
            if (held != l || l < n) bad |= HSQ_DEVERR_LEN;
        }
        const int tiles = (n + kTileRow - 1) / kTileRow;
        int total;
        const int at = before + block_scan_1<kTileThreads>(tiles, s_scan, total);
        if (at <= unit && unit < at + tiles) {
            const int j = (unit - at) * kTileRow;
            s_at[0] = b;
            s_at[1] = s + j;
            s_at[2] = min(kTileRow, n - j);
            s_at[3] = max(l, 0) - n + j;
            s_at[4] = held;
        }
        before += total;
        __syncthreads();
    }
    __syncthreads();
    if (bad) atomicOr(a.err, bad);
    const int b = s_at[0], first_row = s_at[1], rows = s_at[2], ahead = s_at[3], held = s_at[4];
    if (rows == 0) return;
    bad = 0;
    auto pages_of = [&](int j) {
        return a.prefix_pages + ((min(max(ahead + j + 1, 0), held) + a.page_n - 1) >> a.page_shift);
    };
    const int last = pages_of(rows - 1) - a.recent;  // pages in [first, last) are scored
    // codes of the rows' queries
    for (int j = warp; j < kTileRow; j += kTileThreads / 32)
        s_q[j][lane] = j < rows ? query_codes(a.q + ((size_t)(first_row + j) * a.Hq + h * a.r) * 128, a.r) : 0u;
    __syncthreads();
    if (beta > 0 && pages_of(rows - 1) > a.top) {
        uint32_t qf[8][4];  // k step s of lane t: dims 32 t + 4 s .. + 3 of rows g and g + 8
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            codes_f16(s_q[g][8 * t + k], qf[k][0], qf[k][2]);
            codes_f16(s_q[g + 8][8 * t + k], qf[k][1], qf[k][3]);
        }
        int have[2] = {0, 0};  // best so far of the warp's rows 2 warp, 2 warp + 1
        for (int c0 = a.first; c0 < last; c0 += kChunk) {
            const int c1 = min(last, c0 + kChunk);
            // scores: a warp takes 8 pages at a time (lanes 4 g + t: page g)
            for (int p0 = c0 + 8 * warp; p0 < c1; p0 += kTileThreads / 4) {
                const int p = p0 + g;
                int id = -1;
                if (p < c1) {
                    id = p < a.prefix_pages ? a.prefix[p] : a.table[(size_t)b * a.width + p - a.prefix_pages];
                    if (id < 0 || id >= a.n_pages) {
                        id = -1;
                        bad |= HSQ_DEVERR_PAGE;
                    }
                }
                uint4 m0 = make_uint4(0, 0, 0, 0), m1 = m0;
                float scale = 0.f;
                if (id >= 0) {
                    const uint4* src = reinterpret_cast<const uint4*>(a.codes + ((size_t)id * a.Hkv + h) * 128 + 32 * t);
                    m0 = __ldg(src);
                    m1 = __ldg(src + 1);
                    scale = __ldg(a.scale + (size_t)id * a.Hkv + h);
                }
                float d[4] = {0.f, 0.f, 0.f, 0.f};
                const uint32_t w[8] = {m0.x, m0.y, m0.z, m0.w, m1.x, m1.y, m1.z, m1.w};
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    uint32_t lo, hi;
                    codes_f16(w[k], lo, hi);
                    mma_f16(d, qf[k], lo, hi);
                }
                // d[e]: row g + 8 (e >> 1), page p0 + 2 t + (e & 1)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float sc = __shfl_sync(kFull, scale, 4 * (2 * t + e));
                    const int of = __shfl_sync(kFull, id, 4 * (2 * t + e));
                    const int col = p0 - c0 + 2 * t + e;
                    s_key[g * kPitch + col] = of >= 0 ? score_key((int)d[e], sc) : 0u;
                    s_key[(g + 8) * kPitch + col] = of >= 0 ? score_key((int)d[e + 2], sc) : 0u;
                }
            }
            __syncthreads();
#pragma unroll 1
            for (int rr = 0; rr < 2; ++rr) {
                const int j = 2 * warp + rr, c = j < rows ? pages_of(j) : 0;
                if (j >= rows || c <= a.top) continue;
                const int G = min(c - a.recent, c1) - c0;  // keys of the chunk that count for the row
                uint32_t* best = s_best + j * beta;
                int* page = s_page + j * beta;
                const int nb = have[rr];
                uint32_t k[kChunk / 32], o[kCandRegs];
#pragma unroll
                for (int i = 0; i < kChunk / 32; ++i) k[i] = 32 * i + lane < G ? s_key[j * kPitch + 32 * i + lane] : 0u;
#pragma unroll
                for (int i = 0; i < kCandRegs; ++i) o[i] = 32 * i < nb && 32 * i + lane < nb ? best[32 * i + lane] : 0u;
                const int used = (nb + 31) / 32;
                auto count = [&](uint32_t v) {  // keys >= v
                    int n = 0;
#pragma unroll
                    for (int i = 0; i < kChunk / 32; ++i) n += k[i] >= v;
#pragma unroll
                    for (int i = 0; i < kCandRegs; ++i)
                        if (i < used) n += o[i] >= v;
                    return __reduce_add_sync(kFull, n);
                };
                uint32_t lo = 1, top = 0;
                int n_lo = count(1);
                int ties = 0;  // of the keys equal to lo, those to be taken (all where count says so)
                if (n_lo > beta) {
#pragma unroll
                    for (int i = 0; i < kChunk / 32; ++i) top = max(top, k[i]);
#pragma unroll
                    for (int i = 0; i < kCandRegs; ++i) top = max(top, o[i]);
                    uint32_t hi = __reduce_max_sync(kFull, top);  // fewer than beta keys lie at or above hi + 1
                    // (one past the largest: none)
                    uint64_t above = (uint64_t)hi + 1;
                    int n_above = 0;
                    for (uint32_t step = 1u << 21; n_lo != beta; step = step < (1u << 31) ? step << 1 : step) {
                        const uint32_t v = above > (uint64_t)step + 1 ? (uint32_t)(above - step) : 1u;
                        const int n = v == 1 ? n_lo : count(v);
                        if (n >= beta) {
                            lo = v;
                            n_lo = n;
                            break;
                        }
                        above = v;
                        n_above = n;
                    }
                    while (n_lo != beta && above - lo > 1) {
                        const uint32_t v = lo + (uint32_t)((above - lo) >> 1);
                        const int n = count(v);
                        if (n >= beta) {
                            lo = v;
                            n_lo = n;
                        } else {
                            above = v;
                            n_above = n;
                        }
                    }
                    ties = n_lo == beta ? 1 << 30 : beta - n_above;
                } else {
                    ties = 1 << 30;
                }
                // those taken, in the pages' order: the best so far (lower pages), then the chunk's
                int n = 0, eq = 0;
                const unsigned lt = (1u << lane) - 1u;
                auto put = [&](uint32_t key, int pg, bool copy) {
                    const bool e = key == lo;
                    const unsigned be = __ballot_sync(kFull, e);
                    const bool in = key > lo || (e && eq + __popc(be & lt) < ties);
                    const unsigned bi = __ballot_sync(kFull, in);
                    if (in && copy) {
                        best[n + __popc(bi & lt)] = key;
                        page[n + __popc(bi & lt)] = pg;
                    }
                    n += __popc(bi);
                    eq += __popc(be);
                };
                __syncwarp();
#pragma unroll 1
                for (int i = 0; i < used; ++i) {
                    const int at = 32 * i + lane;
                    const uint32_t key = at < nb ? best[at] : 0u;
                    const int pg = at < nb ? page[at] : 0;
                    __syncwarp();
                    put(key, pg, true);
                    __syncwarp();
                }
#pragma unroll
                for (int i = 0; i < kChunk / 32; ++i)
                    if (32 * i < G) put(k[i], c0 + 32 * i + lane, true);
                have[rr] = n;
            }
            __syncthreads();
        }
        // what follows reads the warp's own rows only
#pragma unroll 1
        for (int rr = 0; rr < 2; ++rr) {
            const int j = 2 * warp + rr;
            if (j >= rows || pages_of(j) <= a.top) continue;
            int32_t* out = a.sel + ((size_t)(first_row + j) * a.Hkv + h) * a.top;
            for (int i = lane; i < have[rr]; i += 32) out[a.first + i] = s_page[j * beta + i];
            const int c = pages_of(j), n = a.first + have[rr];
            for (int i = lane; i < a.first; i += 32) out[i] = i;
            for (int i = lane; i < a.recent; i += 32) out[n + i] = c - a.recent + i;
            for (int i = n + a.recent + lane; i < a.top; i += 32) out[i] = -1;
        }
    }
    for (int j = warp; j < rows; j += kTileThreads / 32) {
        const int c = pages_of(j);
        int32_t* out = a.sel + ((size_t)(first_row + j) * a.Hkv + h) * a.top;
        if (c <= a.top) {
            for (int i = lane; i < a.top; i += 32) out[i] = i < c ? i : -1;
        } else if (beta == 0) {
            for (int i = lane; i < a.top; i += 32) out[i] = i < a.first ? i : c - a.recent + i - a.first;
        }
    }
    if (bad) atomicOr(a.err, bad);
}

// Requests of up to this many rows go row by row (where no request has more).
constexpr int kFewRows = 8;

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
    cudaStream_t st_ = reinterpret_cast<cudaStream_t>(stream);
    void* args[] = {&a};
    cudaError_t e;
    if (max_new <= kFewRows) {
        const size_t smem = 4 * (size_t)(np + width);
        int S = 1;
        while (S < 8 && (long long)rows * Hkv * S < 2LL * ctx->num_sms && np + width >= 512 * S) S *= 2;
        if ((e = hsq::raise_smem_limit((const void*)page_select_rows_kernel, ctx->device, smem)) == cudaSuccess)
            e = launch_cluster((const void*)page_select_rows_kernel, (unsigned)(rows * Hkv * S), kRowThreads, S, smem, st_, false, args);
    } else {
        const int beta = top - first - recent;
        const size_t smem = 4 * (size_t)kTileRow * (kPitch + 2 * beta);
        const long long units = rows / kTileRow + std::min(B, rows);
        if ((e = hsq::raise_smem_limit((const void*)page_select_tiles_kernel, ctx->device, smem)) == cudaSuccess)
            e = launch((const void*)page_select_tiles_kernel, (int)(units * Hkv), kTileThreads, smem, st_, false, args);
    }
    return e == cudaSuccess ? HSQ_OK : hsq::cuda_fail(ctx, e, "page_select");
}

}  // extern "C"
