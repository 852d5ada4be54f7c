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

// Order-preserving key of the score dot * scale (dot: a whole number), never 0, which stands for a page that cannot be selected:
// 0 and -0 alike (the sum with 0 makes both 0), -inf lowest, and the NaN that a product gives (0x7FFFFFFF) above all.
__device__ __forceinline__ uint32_t score_key(float dot, float scale) {
    const uint32_t u = __float_as_uint(__fmaf_rn(dot, scale, 0.f));
    return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}

constexpr int kBins = 256;

// The tiles' keys are the score's bits, as whole numbers with a sign: what is not below 0 is in order as it stands (NaN on top), and
// most rows take nothing else; for the others `ordered` puts all in order.  kNoKey stands for a page that cannot be selected (no
// score is -0, a whole number times a scale being 0 or not below the scale).
constexpr int kNoKey = (int)0x80000000;
__device__ __forceinline__ int score_bits(float dot, float scale) { return __float_as_int(__fmaf_rn(dot, scale, 0.f)); }
__device__ __forceinline__ int ordered(int v) { return v == kNoKey ? v : v ^ ((v >> 31) & 0x7FFFFFFF); }
// The same bins as score_bin's, and bin 1 for no key, as the last byte of a word that starts with 0x4B0000.
__device__ __forceinline__ uint32_t bits_bin(int v, float per) {
    return __float_as_uint(fminf(fmaxf(fmaf(__int_as_float(v), per, 8388609.f), 8388609.f), 8388608.f + (kBins - 1)));
}

// The bin of a key where the largest, `most`, has a positive score: bins 1 .. 255 of equal width in the score from 0 to the largest
// (what lies below goes to bin 1), rounded to a whole number in the last bits of 2^23 + it, which takes no conversion; 0 for no key.
// Monotone in the key.  (A product that is no number, of an infinite largest score or one whose 254th part is past fp32's range, goes to
// bin 1 with all that lies at or below it.)
__device__ __forceinline__ int score_bin(uint32_t key, float per) {
    const int x = __float_as_int(fmaxf(fmaf(key_to_float(key), per, 8388609.f), 8388609.f)) - 0x4B000000;
    return key == 0u ? 0 : min(x, kBins - 1);
}

// By a warp: the bin of the need-th key from the top of a histogram (lane l adds up the bins 255 - 8 l .. 248 - 8 l; bin 0 counts for
// none, and there are need of the others); need becomes the number to be taken of it.
__device__ __forceinline__ int locate_bin(const int* hist, int& need, int& in_bin) {
    const int lane = threadIdx.x & 31;
    const int4 h1 = reinterpret_cast<const int4*>(hist)[kBins / 4 - 1 - 2 * lane];
    const int4 h0 = reinterpret_cast<const int4*>(hist)[kBins / 4 - 2 - 2 * lane];
    const int hv[8] = {h1.w, h1.z, h1.y, h1.x, h0.w, h0.z, h0.y, lane == 31 ? 0 : h0.x};
    const int sum = ((hv[0] + hv[1]) + (hv[2] + hv[3])) + ((hv[4] + hv[5]) + (hv[6] + hv[7]));
    int run = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(kFull, run, d);
        if (lane >= d) run += x;
    }
    const unsigned reach = __ballot_sync(kFull, run >= need);
    run -= sum;
    int bin = 0, above = 0, in = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (run < need && run + hv[i] >= need) {
            bin = kBins - 1 - 8 * lane - i;
            above = run;
            in = hv[i];
        }
        run += hv[i];
    }
    const int from = __ffs(reach) - 1;
    need -= __shfl_sync(kFull, above, from);
    in_bin = __shfl_sync(kFull, in, from);
    return __shfl_sync(kFull, bin, from);
}

// By a warp: the need-th of up to 32 candidates from the top, and how many of those equal to it are to be taken (all: 1 << 30).
template <class T>
__device__ __forceinline__ T rank_candidates(const T* cand, int count, int need, int& ties) {
    const int lane = threadIdx.x & 31;
    const T x = lane < count ? cand[lane] : T(0);
    int gt = 0, eq = 0;
    for (int i = 0; i < count; ++i) {
        const T y = __shfl_sync(kFull, x, i);
        gt += y > x;
        eq += y == x;
    }
    const int who = __ffs(__ballot_sync(kFull, lane < count && gt < need && gt + eq >= need)) - 1;
    gt = __shfl_sync(kFull, gt, who);
    eq = __shfl_sync(kFull, eq, who);
    ties = gt + eq > need ? need - gt : 1 << 30;
    return __shfl_sync(kFull, x, who);
}

// ---------------------------------------------------------------------------------------
// Rows one by one (decode, proposals): a cluster of CTAs for each (row, KV head).  Its CTAs score a share of the pages each,
// eight lanes a page (16 bytes each, so a warp's load is four whole lines), and leave the keys in the first CTA's
// shared memory, which selects.
// 16 decodes of 520 to 2048 pages, 8 heads: 12.4 us; 4 of some 4000 pages: 9.7.  Bound by latency: of a CTA's cycles 1 to 2
// thousand are the row's lookup, 4 to 7 the scores, 1 to 2 the cluster's barrier, the rest the selection.
// ---------------------------------------------------------------------------------------

constexpr int kRowThreads = 512, kRowWarps = kRowThreads / 32;

struct RowSmem {
    alignas(16) int hist[kBins];
    uint32_t cand[32];
    int cands;
    uint4 count[2][kRowWarps];  // counts at seven pivots, two to a word
    uint32_t word[2][kRowWarps];
};

// The whole CTA's selection of the beta largest of the keys s_keys[0 .. G) (0: none; beta >= 1, at least one barrier since they were
// written): the pages first + i of those taken go to out in ascending order; returns their number.
// K keys a thread in registers; warp w has the 32 K from 32 K w on, in steps of 32.  A histogram of the scores tells the bin
// that holds the beta-th key, and up to 32 keys in it are ranked one against the other.  Where more share the bin, or no score is
// positive, passes of counting find it (each some 0.5 us: as the only way 13.8 us in place of 12.4 for 16 decodes of up
// to 2048 pages, 12.6 in place of 9.7 for 4 of 4096).  A pass counts the keys at or above seven pivots with one barrier:
// first at doubling distances below the largest key, then in turn close around where the count should be met and at the
// eighths of the span that holds the beta-th, until exactly beta lie above or the span is one key (whose ties go to the
// lower pages).
template <int K>
__device__ int select_row(const uint32_t* s_keys, int G, int beta, int first, int32_t* out, RowSmem& sm) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, at = warp * 32 * K + lane;
    uint32_t k[K];
    uint32_t top = 0;
    int n = 0;
#pragma unroll
    for (int i = 0; i < K; ++i) {
        k[i] = at + 32 * i < G ? s_keys[at + 32 * i] : 0u;
        top = max(top, k[i]);
        n += k[i] != 0u;
    }
    top = __reduce_max_sync(kFull, top);
    n = __reduce_add_sync(kFull, n);
    if (lane == 0) {
        sm.word[0][warp] = top;
        sm.word[1][warp] = n;
    }
    if (threadIdx.x < kBins) sm.hist[threadIdx.x] = 0;
    if (threadIdx.x == 0) sm.cands = 0;
    __syncthreads();
    top = __reduce_max_sync(kFull, lane < kRowWarps ? sm.word[0][lane] : 0u);
    n = __reduce_add_sync(kFull, lane < kRowWarps ? (int)sm.word[1][lane] : 0);
    // At least beta keys (or all there are) lie at or above lo, n_above < beta at or above lo + span.  (32 bits throughout: the
    // span of all keys is top - 1 + 1.)
    uint32_t lo = 1, span = top;
    int n_lo = n, n_above = 0, turn = 0, ties = 1 << 30;  // ties: of the keys equal to lo, those to be taken
    bool found = n <= beta;
    if (!found && key_to_float(top) > 0.f) {
        const float per = 254.f / key_to_float(top);
#pragma unroll
        for (int i = 0; i < K; ++i)
            if (k[i] != 0u) atomicAdd(sm.hist + score_bin(k[i], per), 1);
        __syncthreads();
        int need = beta, in_bin = 0;
        const int bin = locate_bin(sm.hist, need, in_bin);  // (every warp the same)
        if (in_bin <= 32) {
#pragma unroll
            for (int i = 0; i < K; ++i)
                if (k[i] != 0u && score_bin(k[i], per) == bin) sm.cand[atomicAdd(&sm.cands, 1)] = k[i];
            __syncthreads();
            lo = rank_candidates(sm.cand, in_bin, need, ties);
            found = true;
        }
    }
    if (!found) {
        bool doubling = true, even = false;
        uint32_t step = 1u << 20;
#pragma unroll 1
        while (n_lo != beta && span > 1) {
            uint32_t v[7];  // as distances from lo, descending
            if (doubling) {
#pragma unroll
                for (int i = 0; i < 7; ++i) v[i] = span > step << i && step << i >> i == step ? span - (step << i) : 0u;
            } else if (even) {
                const uint32_t whole = span >> 3, rest = span & 7;
#pragma unroll
                for (int i = 0; i < 7; ++i) v[i] = whole * (7 - i) + (rest * (7 - i) >> 3);
            } else {  // close around where the count should be met if the keys were spread evenly
                const float width = (float)span, at = width * __fdividef((float)(n_lo - beta) + 0.5f, (float)(n_lo - n_above));
#pragma unroll
                for (int i = 0; i < 7; ++i) v[i] = min(max(__float2uint_rz(fmaf(width, (float)(3 - i) * (1.f / 24.f), at)), 1u), span - 1);
            }
            even = !doubling && !even;
#pragma unroll
            for (int i = 0; i < 7; ++i) v[i] += lo;
            uint32_t c[4] = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < K; ++i)
#pragma unroll
                for (int j = 0; j < 7; ++j) c[j >> 1] += k[i] >= v[j] ? (j & 1 ? 1u << 16 : 1u) : 0u;
#pragma unroll
            for (int j = 0; j < 4; ++j) c[j] = __reduce_add_sync(kFull, c[j]);
            if (lane == 0) sm.count[turn][warp] = make_uint4(c[0], c[1], c[2], c[3]);
            __syncthreads();
            const uint4 x = lane < kRowWarps ? sm.count[turn][lane] : make_uint4(0, 0, 0, 0);
            turn ^= 1;
            c[0] = __reduce_add_sync(kFull, x.x);
            c[1] = __reduce_add_sync(kFull, x.y);
            c[2] = __reduce_add_sync(kFull, x.z);
            c[3] = __reduce_add_sync(kFull, x.w);
            bool met = false;
            uint32_t above = lo + span;  // (0: past the last key there can be)
#pragma unroll
            for (int j = 0; j < 7; ++j) {
                const int m = (int)(j & 1 ? c[j >> 1] >> 16 : c[j >> 1] & 0xFFFFu);
                if (!met) {
                    if (m >= beta) {
                        lo = v[j];
                        n_lo = m;
                        met = true;
                    } else {
                        above = v[j];
                        n_above = m;
                    }
                }
            }
            span = above - lo;
            if (met) doubling = false;
            else step <<= 7;
        }
        if (n_lo > beta) ties = beta - n_above;
    }
    int gt = 0, eq = 0;
#pragma unroll
    for (int i = 0; i < K; ++i) {
        gt += __popc(__ballot_sync(kFull, k[i] > lo));
        eq += __popc(__ballot_sync(kFull, k[i] == lo));
    }
    __syncthreads();  // (the words and counts above have been read)
    if (lane == 0) {
        sm.word[0][warp] = gt;
        sm.word[1][warp] = eq;
    }
    __syncthreads();
    int g0 = 0, e0 = 0, g_all = 0, e_all = 0;  // before the warp; in all
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) {
        const int x = (int)sm.word[0][w], y = (int)sm.word[1][w];
        g0 += w < warp ? x : 0;
        e0 += w < warp ? y : 0;
        g_all += x;
        e_all += y;
    }
    const unsigned lt = (1u << lane) - 1u;
    if (gt | eq) {
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const bool is_g = k[i] > lo, is_e = k[i] == lo;
            const unsigned bg = __ballot_sync(kFull, is_g), be = __ballot_sync(kFull, is_e);
            const int e = e0 + __popc(be & lt);
            if (is_g || (is_e && e < ties)) out[g0 + __popc(bg & lt) + min(e, ties)] = first + at + 32 * i;
            g0 += __popc(bg);
            e0 += __popc(be);
        }
    }
    return g_all + min(e_all, ties);
}

template <int K>  // keys a thread that the first CTA selects from, at most
__global__ void __launch_bounds__(kRowThreads, K <= 16 ? 2 : 1) page_select_rows_kernel(const __grid_constant__ SelectArgs a) {
    extern __shared__ uint32_t s_keys[];
    __shared__ RowSmem s_sel;
    __shared__ uint32_t s_q[32];
    __shared__ int s_row[3];
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
    if (blockIdx.x == 0) bad |= requests_bad(a.q_start, a.lens, a.B, a.rows, a.width << a.page_shift, kRowThreads);
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
        auto id_of = [&](int i) {
            const int p = a.first + i;
            return i >= g1 ? -1 : p < a.prefix_pages ? a.prefix[p] : a.table[(size_t)b * a.width + p - a.prefix_pages];
        };
        int i0 = (int)((long long)G * rank / S) + warp * 32, ahead = id_of(i0 + lane);
        for (; i0 < g1; i0 += kRowThreads) {
            const int i = i0 + lane;
            int id = ahead;
            ahead = id_of(i + kRowThreads);  // (one step ahead)
            if (i < g1 && (id < 0 || id >= a.n_pages)) {
                id = -1;
                bad |= HSQ_DEVERR_PAGE;
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
            if (i < g1) keys[i] = id >= 0 ? score_key((float)mine, scale) : 0u;
        }
    }
    cluster.sync();  // the keys are in the first CTA; no remote access follows
    if (rank == 0 && live) {
        int32_t* out = a.sel + ((size_t)row * a.Hkv + h) * a.top;
        if (c <= a.top) {
            for (int i = tid; i < a.top; i += kRowThreads) out[i] = i < c ? i : -1;
        } else {
            // the first pages, the selected ones and the last ones (which move up where fewer could be selected)
            for (int i = tid; i < a.first; i += kRowThreads) out[i] = i;
            int n = a.first;
            if (score) {
                if (K > 4 && G <= 4 * kRowThreads) n += select_row<4>(s_keys, G, beta, a.first, out + a.first, s_sel);
                else if (K > 8 && G <= 8 * kRowThreads) n += select_row<8>(s_keys, G, beta, a.first, out + a.first, s_sel);
                else if (K > 16 && G <= 16 * kRowThreads) n += select_row<16>(s_keys, G, beta, a.first, out + a.first, s_sel);
                else n += select_row<K>(s_keys, G, beta, a.first, out + a.first, s_sel);
            }
            for (int i = tid; i < a.recent; i += kRowThreads) out[n + i] = c - a.recent + i;
            for (int i = n + a.recent + tid; i < a.top; i += kRowThreads) out[i] = -1;
        }
    }
    if (bad) atomicOr(a.err, bad);
}
static_assert(64 * kRowThreads >= HSQ_MAX_SELECT_PAGES, "the keys fit the registers");

// ---------------------------------------------------------------------------------------
// Rows by tiles of 16 of one request (prompts' chunks): a CTA for each (tile, KV head) goes over the pages in chunks of 1024.
//   Scores by tensor-core products of whole numbers in fp16 (exact: |code| <= 127, sums below 2^21 in fp32): 16 rows (A, in
//   registers) x 8 pages (B).  The dims are taken in an order that gives a lane 16 neighbouring bytes of a page's codes twice.
//   Selection by a warp a row: a histogram of the row's keys, the ranks of those in the bin that holds the last to be
//   taken, and the taken ones in order from masks of 32 neighbours a lane.
// 2048 rows x 8 heads over 1024 pages, 64 taken: 64 us (with a CTA a row 375; with the keys in order from the start 67).  Bound by
// issue slots (60 %) and the latency of the codes' loads; with one page taken it is 4 us less.
// ---------------------------------------------------------------------------------------

constexpr int kTileThreads = 512, kTileRow = kTileThreads / 32, kChunk = 1024;
// A row's keys: 32 neighbours (a lane's) and two words between, so that lanes side by side read and rows side by side are written without bank
// conflicts.
constexpr int kLanePitch = 34, kPitch = kChunk / 32 * kLanePitch + 8;
static_assert(kTileRow == 16, "a warp a row, 16 rows a product");

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

__global__ void __launch_bounds__(kTileThreads, 2) page_select_tiles_kernel(const __grid_constant__ SelectArgs a) {
    extern __shared__ int s_dyn[];
    int* s_key = s_dyn;                                     // [16][kPitch] the chunk's keys
    const int beta = a.top - a.first - a.recent;
    int* s_best = s_key + kTileRow * kPitch;                // [16][beta] the best so far, in the pages' order: key,
    int* s_page = s_best + kTileRow * max(beta, 0);         // page
    __shared__ uint32_t s_q[kTileRow][32];
    __shared__ alignas(16) int s_id[kChunk];
    __shared__ alignas(16) float s_scale[kChunk];
    __shared__ alignas(16) int s_hist[kTileThreads / 32][kBins + 4];  // (and the number of candidates)
    __shared__ int s_cand[kTileThreads / 32][32];
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
    s_q[warp][lane] = warp < rows ? query_codes(a.q + ((size_t)(first_row + warp) * a.Hq + h * a.r) * 128, a.r) : 0u;
    __syncthreads();
    if (beta > 0 && pages_of(rows - 1) > a.top) {
        uint32_t qf[8][4];  // step k of lane t: dims 16 t + 4 k .. + 3, from k = 4 on 64 + 16 t + 4 (k - 4) .., of rows g and g + 8
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int w = (k < 4 ? 4 * t : 12 + 4 * t) + k;
            codes_f16(s_q[g][w], qf[k][0], qf[k][2]);
            codes_f16(s_q[g + 8][w], qf[k][1], qf[k][3]);
        }
        int have = 0;  // best so far of the warp's row
        for (int c0 = a.first; c0 < last; c0 += kChunk) {
            const int c1 = min(last, c0 + kChunk);
            bool gone = false;
            for (int i = tid; i < c1 - c0; i += kTileThreads) {
                const int p = c0 + i;
                int id = p < a.prefix_pages ? a.prefix[p] : a.table[(size_t)b * a.width + p - a.prefix_pages];
                if (id < 0 || id >= a.n_pages) {
                    id = -1;
                    bad |= HSQ_DEVERR_PAGE;
                }
                gone |= id < 0;
                s_id[i] = id;
                s_scale[i] = id >= 0 ? __ldg(a.scale + (size_t)id * a.Hkv + h) : 0.f;
            }
            gone = __syncthreads_or(gone);
            // scores: a warp takes 8 pages at a time (lanes 4 g + t: page g), twice over with the loads first
            for (int p0 = 8 * warp; p0 < c1 - c0; p0 += 2 * kTileThreads / 4) {
                uint4 m[2][2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int p = p0 + u * (kTileThreads / 4) + g, id = p < c1 - c0 ? s_id[p] : -1;
                    m[u][0] = m[u][1] = make_uint4(0, 0, 0, 0);
                    if (id >= 0) {
                        const uint4* src = reinterpret_cast<const uint4*>(a.codes + ((size_t)id * a.Hkv + h) * 128 + 16 * t);
                        m[u][0] = __ldg(src);
                        m[u][1] = __ldg(src + 4);
                    }
                }
                float d[2][4];  // [u][e]: row g + 8 (e >> 1), page p0 + 128 u + 2 t + (e & 1)
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e) d[u][e] = 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint4 w = m[u][k >> 2];
                        uint32_t lo, hi;
                        codes_f16((k & 3) == 0 ? w.x : (k & 3) == 1 ? w.y : (k & 3) == 2 ? w.z : w.w, lo, hi);
                        mma_f16(d[u], qf[k], lo, hi);
                    }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int col = p0 + u * (kTileThreads / 4) + 2 * t;
                    if (col >= c1 - c0) continue;
                    const float2 sc = *reinterpret_cast<const float2*>(s_scale + col);  // (columns behind the last page are not looked at)
                    int* to = s_key + g * kPitch + col + 2 * (col >> 5);
                    *reinterpret_cast<int2*>(to) = make_int2(score_bits(d[u][0], sc.x), score_bits(d[u][1], sc.y));
                    *reinterpret_cast<int2*>(to + 8 * kPitch) = make_int2(score_bits(d[u][2], sc.x), score_bits(d[u][3], sc.y));
                }
            }
            __syncthreads();
            if (gone) {
                for (int i = lane; i < c1 - c0; i += 32)
                    if (s_id[i] < 0) s_key[warp * kPitch + i + 2 * (i >> 5)] = kNoKey;
                __syncwarp();
            }
            const int j = warp, c = j < rows ? pages_of(j) : 0;
            if (c > a.top) {
                const int G = min(c - a.recent, c1) - c0;  // keys of the chunk that count for the row
                int* best = s_best + j * beta;
                int* page = s_page + j * beta;
                int* row_keys = s_key + j * kPitch;
                int* mine = row_keys + lane * kLanePitch;  // the lane's 32
                const int nb = have, used = (nb + 31) >> 5;
                for (int i = max(G, 0) + lane; i < kChunk; i += 32) row_keys[i + 2 * (i >> 5)] = kNoKey;
                __syncwarp();
                // every key: the chunk's, then the best so far
                auto each = [&](auto&& f) {
#pragma unroll 1
                    for (int i = 0; i < 32; ++i) f(mine[i]);
#pragma unroll 1
                    for (int i = 0; i < used; ++i) f(32 * i + lane < nb ? best[32 * i + lane] : kNoKey);
                };
                // The key lo above which fewer than beta keys lie, at or above which beta or more (or all there are).  A histogram
                // of the scores tells the bin that holds the beta-th; up to 32 keys in it are ranked one against the other.  Where
                // more share it, or scores not above 0 are taken, histograms of the keys' bits lead there, each over a bin of the last.
                int lo = kNoKey + 1;
                int ties = 1 << 30;  // of the keys equal to lo, those to be taken (all)
                int need = beta;     // of the keys in play
                int* hist = s_hist[warp];
                auto clear = [&] {
#pragma unroll
                    for (int i = 0; i < kBins / 128; ++i) reinterpret_cast<int4*>(hist)[32 * i + lane] = make_int4(0, 0, 0, 0);
                    if (lane == 0) hist[kBins] = 0;  // candidates
                    __syncwarp();
                };
                auto locate = [&](int& in_bin) {
                    __syncwarp();
                    return locate_bin(hist, need, in_bin);
                };
                auto rank = [&](int in_bin) {  // lo and ties from the candidates
                    __syncwarp();
                    lo = rank_candidates(s_cand[warp], in_bin, need, ties);
                };
                auto keep = [&](int v) { s_cand[warp][atomicAdd(hist + kBins, 1)] = v; };
                // First by the score, for rows that take scores above 0 alone.  The bins of a lane's keys stay in registers, four to
                // a word, for the second look.
                int most = kNoKey;
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    const int2 v = *reinterpret_cast<const int2*>(mine + i);
                    most = max(most, max(v.x, v.y));
                }
#pragma unroll 1
                for (int i = 0; i < used; ++i) most = max(most, 32 * i + lane < nb ? best[32 * i + lane] : kNoKey);
                most = __reduce_max_sync(kFull, most);
                bool found = false;
                int in_bin = 0;
                if (most > 0 && most <= 0x7F800000) {  // (else the largest is no number, or none is above 0)
                    const float per = 254.f / __int_as_float(most);
                    uint32_t bins[kChunk / 128];
                    clear();
#pragma unroll
                    for (int w = 0; w < kChunk / 128; ++w) {
                        const int2 v0 = *reinterpret_cast<const int2*>(mine + 4 * w), v1 = *reinterpret_cast<const int2*>(mine + 4 * w + 2);
                        const uint32_t x[4] = {bits_bin(v0.x, per), bits_bin(v0.y, per), bits_bin(v1.x, per), bits_bin(v1.y, per)};
#pragma unroll
                        for (int i = 0; i < 4; ++i) atomicAdd(hist + (x[i] & 0xFFu), 1);
                        bins[w] = __byte_perm(__byte_perm(x[0], x[1], 0x0040), __byte_perm(x[2], x[3], 0x0040), 0x5410);
                    }
#pragma unroll 1
                    for (int i = 0; i < used; ++i)
                        if (32 * i + lane < nb) atomicAdd(hist + (bits_bin(best[32 * i + lane], per) & 0xFFu), 1);
                    const int bin = locate(in_bin);
                    if (bin > 1 && in_bin <= 32) {
                        const uint32_t four = 0x01010101u * (uint32_t)bin;
#pragma unroll
                        for (int w = 0; w < kChunk / 128; ++w) {
                            uint32_t hit = __vcmpeq4(bins[w], four) & 0x01010101u;
                            while (hit) {
                                const int i = (__ffs(hit) - 1) >> 3;
                                keep(mine[4 * w + i]);
                                hit &= hit - 1;
                            }
                        }
#pragma unroll 1
                        for (int i = 0; i < used; ++i) {
                            const int v = 32 * i + lane < nb ? best[32 * i + lane] : kNoKey;
                            if (v != kNoKey && (int)(bits_bin(v, per) & 0xFFu) == bin) keep(v);
                        }
                        rank(in_bin);
                        found = true;
                    }
                }
                if (!found) {
                    // Crowded, or scores not above 0: in order, by the keys' bits.
                    need = beta;
                    int klo = 0x7FFFFFFF, khi = kNoKey, there = 0;
#pragma unroll 1
                    for (int i = 0; i < 32; ++i) mine[i] = ordered(mine[i]);
                    each([&](int v) {
                        if (v != kNoKey) {
                            klo = min(klo, v);
                            khi = max(khi, v);
                            ++there;
                        }
                    });
                    there = __reduce_add_sync(kFull, there);
                    while (there >= beta) {  // (else all are taken)
                        klo = __reduce_min_sync(kFull, klo);
                        khi = __reduce_max_sync(kFull, khi);
                        // (the number to be taken is at most the number in play)
                        const int shift = max(32 - __clz((uint32_t)khi - (uint32_t)klo) - 7, 0);  // 128 bins, from 1 on
                        clear();
                        each([&](int v) {
                            if (v != kNoKey && v >= klo && v <= khi) atomicAdd(hist + 1 + (((uint32_t)v - (uint32_t)klo) >> shift), 1);
                        });
                        const int which = locate(in_bin);
                        int l = 0x7FFFFFFF, u = kNoKey;
                        const bool few = in_bin <= 32;
                        each([&](int v) {
                            if (v != kNoKey && v >= klo && v <= khi && 1 + (int)(((uint32_t)v - (uint32_t)klo) >> shift) == which) {
                                if (few) keep(v);
                                l = min(l, v);
                                u = max(u, v);
                            }
                        });
                        if (few) {
                            rank(in_bin);
                            break;
                        }
                        klo = __reduce_min_sync(kFull, l);
                        khi = __reduce_max_sync(kFull, u);
                        if (klo == khi) {  // one key over and over
                            lo = klo;
                            if (in_bin > need) ties = need;
                            break;
                        }
                    }
                }
                // those taken, in the pages' order: the best so far (lower pages), then the chunk's
                int n = 0, eq = 0;
                const unsigned lt = (1u << lane) - 1u;
#pragma unroll 1
                for (int i = 0; i < used; ++i) {
                    const int at = 32 * i + lane;
                    const int key = at < nb ? best[at] : kNoKey;
                    const int pg = at < nb ? page[at] : 0;
                    __syncwarp();
                    const unsigned be = __ballot_sync(kFull, key == lo);
                    const bool in = key > lo || (key == lo && eq + __popc(be & lt) < ties);
                    eq += __popc(be);
                    const unsigned bi = __ballot_sync(kFull, in);
                    if (in) {
                        best[n + __popc(bi & lt)] = key;
                        page[n + __popc(bi & lt)] = pg;
                    }
                    n += __popc(bi);
                    __syncwarp();
                }
                uint32_t in = 0;  // of the lane's 32
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    const int2 v = *reinterpret_cast<const int2*>(mine + i);
                    in |= (v.x >= lo ? 1u << i : 0u) | (v.y >= lo ? 2u << i : 0u);
                }
                if (ties != 1 << 30) {  // only so many of those equal to lo
                    uint32_t even = 0;
                    for (uint32_t x = in; x; x &= x - 1) even |= mine[__ffs(x) - 1] == lo ? x & (0u - x) : 0u;
                    int e = __popc(even);
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) {
                        const int x = __shfl_up_sync(kFull, e, d);
                        if (lane >= d) e += x;
                    }
                    e += eq - __popc(even);  // before the lane's first
                    for (; even; even &= even - 1)
                        if (e++ >= ties) in &= ~(even & (0u - even));
                }
                int at = __popc(in), all;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int x = __shfl_up_sync(kFull, at, d);
                    if (lane >= d) at += x;
                }
                all = __shfl_sync(kFull, at, 31);
                at += n - __popc(in);
                for (; in; in &= in - 1, ++at) {
                    const int i = __ffs(in) - 1;
                    best[at] = mine[i];
                    page[at] = c0 + 32 * lane + i;
                }
                n += all;
                __syncwarp();
                have = n;
            }
            __syncthreads();
        }
        // (the warp's own row)
        const int c = warp < rows ? pages_of(warp) : 0;
        if (c > a.top) {
            int32_t* out = a.sel + ((size_t)(first_row + warp) * a.Hkv + h) * a.top;
            for (int i = lane; i < have; i += 32) out[a.first + i] = s_page[warp * beta + i];
            const int n = a.first + have;
            for (int i = lane; i < a.first; i += 32) out[i] = i;
            for (int i = lane; i < a.recent; i += 32) out[n + i] = c - a.recent + i;
            for (int i = n + a.recent + lane; i < a.top; i += 32) out[i] = -1;
        }
    }
    if (warp < rows) {
        const int c = pages_of(warp);
        int32_t* out = a.sel + ((size_t)(first_row + warp) * a.Hkv + h) * a.top;
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
        while (S < 8 && (long long)rows * Hkv * 2 * S <= 2LL * ctx->num_sms && np + width >= 512 * S) S *= 2;
        const void* fn = np + width <= 4 * kRowThreads ? (const void*)page_select_rows_kernel<4>
                         : np + width <= 8 * kRowThreads ? (const void*)page_select_rows_kernel<8>
                         : np + width <= 16 * kRowThreads ? (const void*)page_select_rows_kernel<16> : (const void*)page_select_rows_kernel<64>;
        if ((e = hsq::raise_smem_limit(fn, ctx->device, smem)) == cudaSuccess)
            e = launch_cluster(fn, (unsigned)(rows * Hkv * S), kRowThreads, S, smem, st_, false, args);
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
