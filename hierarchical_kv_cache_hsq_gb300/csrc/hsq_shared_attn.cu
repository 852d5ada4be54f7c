// Attention of a batch whose requests share a prefix (hsq_shared_attn).
//
// For row i of request b (token j of its n new ones) and query head jq of KV head
// h: one softmax, scale 1/sqrt(128), over the prefix's tokens and the request's own
// tokens s <= len - n + j.  A softmax over the union of two key sets is the
// weighted sum of the softmaxes over each: with m, l, o the maximum, the sum of
// exp(x - m) and the sum of exp(x - m) v of a part,
//     out = sum_p exp(m_p - M) o_p / sum_p exp(m_p - M) l_p,   M = max_p m_p,
// so the prefix is read once for all rows of the batch, each request's own pages
// once for its rows, and the parts are joined at the end.
//
// Rows.  The r = Hq / Hkv query heads of a KV head and the rows of the batch
// make one row index (token * r + head), so a tile of 128 rows holds
// floor(128 / r) tokens of ANY requests for the prefix: the tensor cores see full
// tiles in a decode step too.
//
// Three kernels, at most two of them in a call besides the prefix's:
//   prefix  shared_tc_kernel<false>: pairs of 128-row tiles x the prefix's
//           128-key tiles on the tensor cores, the whole (KV head, pair, key tile)
//           space cut into equal runs, one per CTA (one CTA per SM); every run
//           leaves its parts (m, l, o in fp32) in the workspace;
//   own     shared_few_kernel for requests of few rows (n r <= 16, the decode step): one
//           cluster per (request, KV head), warps stream keys and values from
//           the pages straight into mma.sync fragments (bound by HBM: 16 rows are too
//           few for a 128-row tile to matter);
//           shared_tc_kernel<true> for requests with more rows: one CTA per
//           (request, KV head, pair of row tiles), causal.
//   Both own kernels read the prefix's parts of their rows, join them with their own and
//   write the result.  They are launched with programmatic serialization: their own keys are
//   read while the prefix kernel finishes, its parts only after griddepcontrol.wait.
//
// Rounding: q, k and v are bf16, products exact, sums fp32; the softmax weights are rounded to
// bf16 for the product with the values (an error of 2^-9 of each weight at most, random over
// the keys, where the output's own rounding is 2^-9 of the result), l sums
// them before that rounding.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "hsq_ctx.h"
#include "hsq_device.cuh"
#include "hsq_tc.cuh"

namespace {

using namespace hsq_tc;

constexpr int kFewRows = 16;                    // rows (tokens x r) of a request up to which the few-rows kernel takes it
constexpr int kTileRows = 128, kTileKeys = 128;
constexpr float kRaise = 8.f;                   // log2 units a logit may exceed the running maximum by before o is rescaled
constexpr float kTileSum = 65536.f;             // sum of a tile's 128 weights from which the maximum is taken anew

struct SharedArgs {
    const uint16_t *q, *pk, *pv;
    const int32_t *q_start, *lens, *table, *prefix;
    uint16_t* out; float* lse;
    int rows, B, width, prefix_len, max_new, n_pages, page_n, page_shift, Hq, Hkv, r;
    int tpt;       // tokens of a row tile: 128 / r
    int runs;      // CTAs of the prefix kernel
    float* part_o;   // [slot][2 streams][128 rows][128]
    float2* part_ml; // [slot][2 streams][128 rows]: maximum (of q.k, unscaled), sum
    int* err;
};

// Request b's rows and own tokens, checked: rows [first, first + n), own tokens [0, len).
struct Request { int first, n, len; };

__device__ __forceinline__ Request request_of(const SharedArgs& a, int b, int& bad) {
    Request r;
    const int s = a.q_start[b], e = a.q_start[b + 1];
    r.first = s;
    r.n = e - s;
    if (s < 0 || e < s || e > a.rows || r.n > a.max_new) {
        bad |= HSQ_DEVERR_LEN;
        r.first = r.n = 0;
    }
    const int len = a.lens[b];
    const long long cap = (long long)a.width << a.page_shift;
    r.len = (int)min((long long)max(len, 0), cap);
    if (len != r.len || r.len < r.n) bad |= HSQ_DEVERR_LEN;
    return r;
}

// ---- the prefix's work: key tiles of (KV head, pair of row tiles), cut into equal runs ----

struct PrefixPlan {
    int tiles, pairs, steps;  // row tiles in use, pairs of them, key tiles
    long long work;           // Hkv * pairs * steps
};

__device__ __forceinline__ PrefixPlan prefix_plan(const SharedArgs& a) {
    PrefixPlan p;
    const int live = min(max(a.q_start[a.B], 0), a.rows);
    p.tiles = (live + a.tpt - 1) / a.tpt;
    p.pairs = (p.tiles + 1) >> 1;
    p.steps = (a.prefix_len + kTileKeys - 1) / kTileKeys;
    p.work = (long long)a.Hkv * p.pairs * p.steps;
    return p;
}

// run c covers the steps [c work / runs, (c + 1) work / runs); an item's segment in run c keeps its
// parts in slot item + c (segments in order raise one of the two by one, so slots are unique)
__device__ __forceinline__ long long run_begin(const PrefixPlan& p, int runs, int c) { return p.work * c / runs; }
__device__ __forceinline__ int run_of(const PrefixPlan& p, int runs, long long w) {
    return (int)(((w + 1) * runs - 1) / p.work);
}

// The parts of one row (token, head jj of KV head h): indices [at + k * step], k < n, of part_ml rows
struct RowParts { size_t at; size_t step; int n; };

__device__ __forceinline__ RowParts row_parts(const SharedArgs& a, const PrefixPlan& p, int h, int token, int jj) {
    const int tile = token / a.tpt, pair = tile >> 1, stream = tile & 1;
    const int row = (token - tile * a.tpt) * a.r + jj;
    const long long item = (long long)h * p.pairs + pair, w0 = item * p.steps;
    const int c0 = run_of(p, a.runs, w0), c1 = run_of(p, a.runs, w0 + p.steps - 1);
    // a pair of one tile has its key tiles dealt to both streams
    const bool split = tile == p.tiles - 1 && !(tile & 1);
    RowParts x;
    x.at = ((size_t)(item + c0) * 2 + stream) * kTileRows + row;
    x.step = split ? kTileRows : 2 * kTileRows;
    x.n = (c1 - c0 + 1) * (split ? 2 : 1);
    return x;
}

// One arrival for the whole warp, after every lane's writes.
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

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

// ---------------------------------------------------------------------------------------
// Tensor-core kernel.  One CTA per SM, 12 warps: softmax warps 0-3 (stream 0) and 4-7
// (stream 1), warp 8 loads, warp 9 issues the MMAs (10 and 11 only give their registers away:
// 168 a thread at launch, then 184 for the softmax warps, whose row of 128 logits
// lives in registers, and 136 for the others).  A stream is a 128-row query tile with
// its S / P and O in tensor memory.  The two streams either hold two row tiles and share every
// key tile (so keys and values are loaded once for 256 rows), or, when only one row tile is
// left, hold the same rows and take the key tiles in turn.  While one stream's softmax
// runs, the tensor cores work for the other.
//   shared memory: ring of five 32 KB tiles K0 V0 K1 V1 ... (TMA, 128-byte swizzle), two Q tiles;
//   tensor memory: S of stream s at columns 128 s (P, bf16, over its first 64), O at 256 + 128 s.
// ---------------------------------------------------------------------------------------

constexpr int kTcThreads = 384, kStages = 5;
constexpr uint32_t kTileBytes = 128 * 128 * 2, kHalfBytes = kTileBytes / 2;
constexpr uint32_t kOffQ = kStages * kTileBytes, kOffBars = kOffQ + 2 * kTileBytes;
// barriers: full[5] | empty[5] | q_full[2] | s_full[2] | p_full[2] | o_full[2] | tail | x_full
constexpr int kTcBars = 2 * kStages + 10;
constexpr uint32_t kOffMask = kOffBars + 8 * (kTcBars + 1);        // [8] pages of a key tile that lie in the pool
constexpr uint32_t kTcSmem = kOffMask + 32 + 16 + 1024;      // + TMEM address, alignment

// A place in the ring of stages, and the parity of its barriers' phase.
struct Ring {
    uint32_t stage, phase;
    __device__ __forceinline__ void advance(uint32_t by) {
        stage += by;
        if (stage >= kStages) {
            stage -= kStages;
            phase ^= 1;
        }
    }
};

// One run of key tiles [n0, n1) of an item.
struct Segment {
    int h, item;
    int tok0, tok1;    // first token of each stream's tile
    int toks0, toks1;  // its tokens
    int n0, n1, end0, end1;
    bool split;
    int klen;          // keys in all
    const int32_t* ids;  // page ids
};

// keys that token `t` of the request sees (own), or all (prefix)
template <bool kOwn>
__device__ __forceinline__ int key_limit(const Request& rq, int klen, int t) {
    return kOwn ? min(klen, rq.len - rq.n + (t - rq.first) + 1) : klen;
}

template <bool kOwn>
__global__ void __launch_bounds__(kTcThreads, 1)
    shared_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                     const __grid_constant__ CUtensorMap mv, const __grid_constant__ SharedArgs a) {
    extern __shared__ uint8_t tc_raw[];
    const uint32_t raw = smem_addr(tc_raw), base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = tc_raw + (base - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t full = base + kOffBars, empty = full + 8 * kStages, q_full = empty + 8 * kStages;
    const uint32_t s_full = q_full + 16, p_full = s_full + 16, o_full = p_full + 16, tail = o_full + 16, x_full = tail + 8;
    volatile uint32_t* s_mask = reinterpret_cast<volatile uint32_t*>(gbase + kOffMask);
    volatile uint32_t* s_tmem = reinterpret_cast<volatile uint32_t*>(gbase + kOffMask + 32);
    int bad = 0;

    // ---- what this CTA works on ----
    Request rq{0, 0, 0};
    PrefixPlan plan = prefix_plan(a);
    long long w = 0, w_end = 0;
    int unit = 0;
    const int32_t* own_ids = nullptr;
    bool have = true;
    if (kOwn) {
        // pair ids: request b's start at q_start[b] / (2 tpt) + b, which leaves room for all of them; the last ids first
        // (later tokens see more keys)
        const int two = 2 * a.tpt, id = (int)(gridDim.y - 1 - blockIdx.y);
        int below = 0;
        for (int b0 = 0; b0 < a.B; b0 += kTcThreads) {
            const int b = b0 + tid;
            below += __syncthreads_count(b < a.B && max(a.q_start[b], 0) / two + b <= id);
        }
        const int b = max(below - 1, 0);
        rq = request_of(a, b, bad);
        unit = id - (max(a.q_start[b], 0) / two + b);
        have = below > 0 && rq.n * a.r > kFewRows && unit * two < rq.n;
        own_ids = a.table + (size_t)b * a.width;
    } else {
        w = run_begin(plan, a.runs, blockIdx.x);
        w_end = run_begin(plan, a.runs, blockIdx.x + 1);
        have = w < w_end;
    }
    if (!kOwn) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (!have) {
        if (kOwn) {
            asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
            asm volatile("griddepcontrol.wait;" ::: "memory");  // (a grid that ends has seen its predecessor end)
        }
        return;
    }

    // the next segment; false when there is none
    auto next = [&](long long& w, Segment& s) {
        if (w >= w_end) return false;
        if (kOwn) {
            s.h = blockIdx.x;
            s.item = 0;
            const int left = rq.n - unit * 2 * a.tpt;  // tokens from this pair's first on
            s.split = left <= a.tpt;
            s.toks0 = min(left, a.tpt);
            s.toks1 = s.split ? s.toks0 : min(left - a.tpt, a.tpt);
            s.tok0 = rq.first + unit * 2 * a.tpt;
            s.tok1 = s.split ? s.tok0 : s.tok0 + a.tpt;
            s.klen = max(0, key_limit<true>(rq, rq.len, s.tok1 + s.toks1 - 1));
            s.ids = own_ids;
            s.n0 = 0;
            s.n1 = (s.klen + kTileKeys - 1) / kTileKeys;
            const int l0 = max(0, key_limit<true>(rq, s.klen, s.tok0 + s.toks0 - 1));
            s.end0 = (l0 + kTileKeys - 1) / kTileKeys;
            s.end1 = s.n1;
            w = w_end;
        } else {
            s.item = (int)(w / plan.steps);
            s.h = s.item / plan.pairs;
            const int pair = s.item - s.h * plan.pairs;
            s.split = 2 * pair + 1 == plan.tiles;
            const int live = min(max(a.q_start[a.B], 0), a.rows);
            s.tok0 = 2 * pair * a.tpt;
            s.tok1 = s.split ? s.tok0 : s.tok0 + a.tpt;
            s.toks0 = min(a.tpt, live - s.tok0);
            s.toks1 = min(a.tpt, live - s.tok1);
            s.klen = a.prefix_len;
            s.ids = a.prefix;
            s.n0 = (int)(w - (long long)s.item * plan.steps);
            s.n1 = (int)min((long long)plan.steps, s.n0 + (w_end - w));
            s.end0 = s.end1 = s.n1;
            w += s.n1 - s.n0;
        }
        return true;
    };
    if (kOwn) w_end = 1;
    // key tiles that stream s takes in a segment
    auto tiles_of = [](const Segment& s, int st) {
        if (!s.split) return (st ? s.end1 : s.end0) - s.n0;
        return (s.n1 - s.n0 + 1 - st) >> 1;
    };

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full + 8 * i, 1);
            mbar_init(s_full + 8 * i, 1);
            mbar_init(p_full + 8 * i, 4);
            mbar_init(o_full + 8 * i, 1);
        }
        mbar_init(tail, 1);
        mbar_init(x_full, 4);
        mbar_init_fence();
    }
    if (warp == 9) {
        tmem_alloc(smem_addr((const void*)s_tmem), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    bool failed = false;
    Segment s;

    // (128 x 168 x 3 registers at launch: 2 x 128 x 184 + 128 x 136)
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 136;\n");
        if (warp == 8) {
            // ---- loads: per key tile the K pages, then the V pages (lane i: page i of the tile) ----
            Ring ring{0, 1};  // (a fresh barrier lets a wait for parity 1 pass: the stages start empty)
            uint32_t step = 0, tail_par = 0;
            const uint32_t page_bytes = (uint32_t)a.page_n * 256u, half_page = (uint32_t)a.page_n * 128u;
            while (next(w, s)) {
#pragma unroll 1
                for (int n = s.n0; n < s.n1; ++n, ++step) {
                    const int nk = min(kTileKeys, s.klen - n * kTileKeys), np = (nk + a.page_n - 1) >> a.page_shift;
                    int id = -1;
                    if (lane < np) id = s.ids[((n * kTileKeys) >> a.page_shift) + lane];
                    const bool in = lane < np && id >= 0 && id < a.n_pages;
                    const uint32_t mask = __ballot_sync(kFull, in);
                    if (mask != (1u << np) - 1u) bad |= HSQ_DEVERR_PAGE;
                    // (a page outside the pool is read past the map's extent: zeros, masked in the softmax)
                    const int y = in ? (id * a.Hkv + s.h) << a.page_shift : (a.n_pages * a.Hkv) << a.page_shift;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        const uint32_t stage = base + ring.stage * kTileBytes, bar = full + 8 * ring.stage;
                        mbar_wait_fast(empty + 8 * ring.stage, ring.phase, failed);
                        failed = __any_sync(kFull, failed);
                        // The values of a tile that does not end on a multiple of 16 keys: the rows up to there
                        // hold what the page holds; their weights are 0, so they have to be finite.  Cleared
                        // here before the tile is handed over.
                        const bool ragged = kv && (nk & 15);
                        const uint32_t lands = ragged ? tail : bar;
                        if (lane == 0) {
                            if (!kv) s_mask[step & 7] = mask;
                            mbar_expect_tx(lands, np * page_bytes);
                        }
                        __syncwarp();
                        if (lane < np) {
                            const void* map = kv ? &mv : &mk;
                            tma_2d(stage + lane * half_page, map, 0, y, lands);
                            tma_2d(stage + lane * half_page + kHalfBytes, map, 64, y, lands);
                        }
                        if (ragged) {
                            mbar_wait_fast(tail, tail_par, failed);
                            failed = __any_sync(kFull, failed);
                            tail_par ^= 1;
                            const int z = (16 - (nk & 15)) * 16;  // 16-byte chunks in both halves
                            for (int i = lane; i < z; i += 32)
                                *reinterpret_cast<uint4*>(gbase + (stage - base) + ((i >> 3) & 1) * kHalfBytes +
                                                          (nk + (i >> 4)) * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
                            fence_async_smem();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(bar);
                        }
                        ring.advance(1);
                    }
                    if (failed) break;
                }
                if (failed) break;
            }
            if (failed) {  // see the copies in flight land before the CTA ends
                for (int i = 0; i < kStages; ++i) mbar_wait(full + 8 * i, i < (int)ring.stage ? ring.phase ^ 1 : ring.phase);
            }
        } else if (warp == 9 && elect_one()) {
            // ---- MMAs, one thread ----
            // Straight code: per pair of key tiles three waits, each one poll; the tensor pipe takes an MMA every 64
            // cycles and holds only one or two more, so what the thread does in between shows.
            const uint32_t q_bytes = (uint32_t)a.tpt * a.r * 256u;
            constexpr uint32_t idO = idesc_bf16_f32_bmn(128, 128), idFull = idesc_bf16_f32(128, 128);
            Ring kr{0, 0}, vr{1, 0};
            uint32_t q_par = 0, p_par = 0;  // a bit for each stream
            auto load_q = [&](int st, int tok) {
                const uint32_t dst = base + kOffQ + st * kTileBytes, bar = q_full + 8 * st;
                mbar_expect_tx(bar, q_bytes);
                tma_3d(dst, &mq, 0, s.h * a.r, tok, bar);
                tma_3d(dst + kHalfBytes, &mq, 64, s.h * a.r, tok, bar);
            };
            auto load_both = [&] {
                if (tiles_of(s, 0) > 0) load_q(0, s.tok0);
                if (tiles_of(s, 1) > 0) load_q(1, s.tok1);
            };
            auto scores = [&](int st, uint32_t idS) {  // S = Q K^T of the tile at kr
                const uint32_t dS = tmem + 128 * st;
                const uint64_t dq = sw128_desc(base + kOffQ + st * kTileBytes), dk = sw128_desc(base + kr.stage * kTileBytes);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t o = ((k >> 2) * kHalfBytes + (k & 3) * 32) >> 4;
                    mma_bf16(dS, dq + o, dk + o, idS, k > 0);
                }
                mma_commit(s_full + 8 * st);
            };
            auto product = [&](int st, uint32_t begun) {  // O += P V of the whole tile at vr
                const uint32_t pa = tmem + 128 * st, dO = pa + 256;
                const uint64_t dv = sw128_mn_desc(base + vr.stage * kTileBytes, kHalfBytes);
                mbar_wait_fast(p_full + 8 * st, (p_par >> st) & 1, failed);
                p_par ^= 1u << st;
                tc_fence_after();
                mma_bf16_ts(dO, pa, dv, idO, begun);
#pragma unroll
                for (int k = 1; k < 8; ++k) mma_bf16_ts(dO, pa + 8 * k, dv + k * (2048 >> 4), idO, 1);
            };
            auto product_last = [&](int st, int ks16, uint32_t begun) {  // the same of an item's last tile: ks16 groups of 16 keys
                const uint32_t pa = tmem + 128 * st, dO = pa + 256;
                const uint64_t dv = sw128_mn_desc(base + vr.stage * kTileBytes, kHalfBytes);
                mbar_wait_fast(p_full + 8 * st, (p_par >> st) & 1, failed);
                p_par ^= 1u << st;
                tc_fence_after();
#pragma unroll 1
                for (int k = 0; k < ks16; ++k) mma_bf16_ts(dO, pa + 8 * k, dv + k * (2048 >> 4), idO, begun | (k > 0));
            };
            bool more = next(w, s);
            if (more) load_both();
            while (more) {
                const int n_last = s.n1 - 1, nk_last = s.klen - n_last * kTileKeys;
                const uint32_t id_last = nk_last < kTileKeys ? idesc_bf16_f32(128, (nk_last + 15) & ~15) : idFull;
                const int ks_last = min(8, (nk_last + 15) >> 4);
                if (tiles_of(s, 0) > 0) { mbar_wait_fast(q_full, q_par & 1, failed); q_par ^= 1; }
                if (tiles_of(s, 1) > 0) { mbar_wait_fast(q_full + 8, (q_par >> 1) & 1, failed); q_par ^= 2; }
                if (!s.split) {
                    const int n0 = s.n0, n1 = s.n1, end0 = s.end0;
                    if (n1 > n0) {
                        mbar_wait_fast(full + 8 * kr.stage, kr.phase, failed);
                        if (n0 < end0) scores(0, n0 == n_last ? id_last : idFull);
                        scores(1, n0 == n_last ? id_last : idFull);
                        mma_commit(empty + 8 * kr.stage);
                        kr.advance(2);
                        int n = n0 + 1;
                        const int both = min(end0, n_last);
#pragma unroll 1
                        for (; n < both; ++n) {  // P V of tile n - 1 and S of tile n, all tiles whole
                            mbar_wait_fast(full + 8 * kr.stage, kr.phase, failed);
                            mbar_wait_fast(full + 8 * vr.stage, vr.phase, failed);
                            product(0, n > n0 + 1);
                            scores(0, idFull);
                            product(1, n > n0 + 1);
                            mma_commit(empty + 8 * vr.stage);
                            vr.advance(2);
                            scores(1, idFull);
                            mma_commit(empty + 8 * kr.stage);
                            kr.advance(2);
                        }
#pragma unroll 1
                        for (; n < n1; ++n) {  // stream 0 ends before stream 1, or the last tile
                            const uint32_t idS = n == n_last ? id_last : idFull;
                            mbar_wait_fast(full + 8 * kr.stage, kr.phase, failed);
                            mbar_wait_fast(full + 8 * vr.stage, vr.phase, failed);
                            if (n <= end0) product_last(0, 8, n > n0 + 1);
                            if (n < end0) scores(0, idS);
                            product_last(1, 8, n > n0 + 1);
                            mma_commit(empty + 8 * vr.stage);
                            vr.advance(2);
                            scores(1, idS);
                            mma_commit(empty + 8 * kr.stage);
                            kr.advance(2);
                        }
                        mbar_wait_fast(full + 8 * vr.stage, vr.phase, failed);
                        if (end0 == n1) product_last(0, ks_last, n_last > n0);
                        if (end0 > n0) mma_commit(o_full);
                        product_last(1, ks_last, n_last > n0);
                        mma_commit(o_full + 8);
                        mma_commit(empty + 8 * vr.stage);
                        vr.advance(2);
                    }
                } else {
#pragma unroll 1
                    for (int n = s.n0; n < s.n1 + 2; ++n) {
                        const int st = (n - s.n0) & 1, np = n - 2;
                        if (np >= s.n0) {
                            mbar_wait_fast(full + 8 * vr.stage, vr.phase, failed);
                            product_last(st, np == n_last ? ks_last : 8, np > s.n0 + 1);
                            mma_commit(empty + 8 * vr.stage);
                            vr.advance(2);
                            if (n >= s.n1) mma_commit(o_full + 8 * st);
                        }
                        if (n < s.n1) {
                            mbar_wait_fast(full + 8 * kr.stage, kr.phase, failed);
                            scores(st, n == n_last ? id_last : idFull);
                            mma_commit(empty + 8 * kr.stage);
                            kr.advance(2);
                        }
                    }
                }
                if (failed) break;
                more = next(w, s);
                if (more) load_both();  // (every S of the segment is done: its P has been seen)
            }
            if (failed) {  // query tiles in flight land before the CTA ends
                mbar_wait(q_full, q_par & 1, 1 << 12);
                mbar_wait(q_full + 8, (q_par >> 1) & 1, 1 << 12);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;\n");
        // ---- softmax: thread = row of its stream's tile ----
        const int st = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t tS = tmem + lanes + 128 * st, tO = tmem + lanes + 256 + 128 * st;
        uint32_t s_par = 0, o_par = 0;
        int step0 = 0;
        while (next(w, s)) {
            const int own_token = row / a.r;
            const bool live = own_token < (st ? s.toks1 : s.toks0);
            const bool idle = 32 * (warp & 3) >= (st ? s.toks1 : s.toks0) * a.r;  // (warp-uniform) no row of this warp in use
            const int lim = live ? key_limit<kOwn>(rq, s.klen, (st ? s.tok1 : s.tok0) + own_token) : 0;
            const int lim_min = key_limit<kOwn>(rq, s.klen, (st ? s.tok1 : s.tok0));
            float m = -INFINITY, l = 0.f;
#pragma unroll 1
            for (int n = s.n0 + (s.split ? st : 0); n < (st ? s.end1 : s.end0); n += s.split ? 2 : 1) {
                mbar_wait_fast(s_full + 8 * st, s_par, failed);
                s_par ^= 1;
                if (!idle) {
                    // The running maximum need not be one: any m that keeps the sums in range gives the same
                    // result, p and l being floating point.  So the row's maximum is looked for in its first tile and
                    // where the tile's sum shows that the logits have outgrown m by far; every other tile goes without
                    // (a third of the softmax's time).
                    tc_fence_after();
                    const int nk = min(kTileKeys, s.klen - n * kTileKeys), np = (nk + a.page_n - 1) >> a.page_shift;
                    const uint32_t mask = s_mask[(step0 + n - s.n0) & 7];
                    if ((n + 1) * kTileKeys > lim_min || mask != (1u << np) - 1u) {
                        // keys past the row's limit or of no page: hidden in S itself, so that the code below (and the
                        // instruction cache) knows whole tiles only
#pragma unroll 1
                        for (int c0 = 0; c0 < 128; c0 += 32) {
                            float x[32];
                            tmem_ld32(tS + c0, x);
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (n * kTileKeys + c0 + c >= lim || !((mask >> ((c0 + c) >> a.page_shift)) & 1u)) x[c] = -INFINITY;
                            tmem_st32(tS + c0, x);
                        }
                    }
                    float t;
                    uint32_t p[2][32];
                    bool look = __any_sync(kFull, live && m == -INFINITY);
#pragma unroll 1
                    while (true) {
                        float x[2][64];
                        if (look) {
                            float m4[4] = {m, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                            for (int c0 = 0; c0 < 128; c0 += 64) {
                                tmem_ld64(tS + c0, x[0]);
#pragma unroll
                                for (int c = 0; c < 64; c += 2)
                                    m4[(c >> 1) & 3] = fmaxf(fmaxf(m4[(c >> 1) & 3], x[0][c]), x[0][c + 1]);
                            }
                            const float mn = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                            const float alpha = m == -INFINITY ? 0.f : ex2_approx((m - mn) * kLogitScaleLog2);
                            m = mn;
                            l *= alpha;
                            if (n >= s.n0 + (s.split ? 2 : 1)) {  // O holds the tiles before (S of this tile follows their P V)
#pragma unroll 1
                                for (int c0 = 0; c0 < 128; c0 += 32) {
                                    float o[32];
                                    tmem_ld32(tO + c0, o);
#pragma unroll
                                    for (int c = 0; c < 32; ++c) o[c] *= alpha;
                                    tmem_st32(tO + c0, o);
                                }
                            }
                        }
                        const float off = m == -INFINITY ? 0.f : -m * kLogitScaleLog2;
                        const uint64_t off2 = pack2(off, off), scale2 = pack2(kLogitScaleLog2, kLogitScaleLog2);
                        uint64_t l2[2] = {0, 0};
                        tmem_ld64(tS, x[0]);
                        tmem_ld64_nowait(tS + 64, x[1]);
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            if (hf) tmem_ld64_wait(x[1]);
#pragma unroll
                            for (int c = 0; c < 64; c += 2) {
                                float e0, e1;
                                unpack2(fma2(pack2(x[hf][c], x[hf][c + 1]), scale2, off2), e0, e1);
                                e0 = ex2_approx(e0);
                                e1 = ex2_approx(e1);
                                l2[(c >> 1) & 1] = add2(l2[(c >> 1) & 1], pack2(e0, e1));
                                p[hf][c >> 1] = pack_bf16(e0, e1);
                            }
                        }
                        float lo, hi;
                        unpack2(add2(l2[0], l2[1]), lo, hi);
                        t = lo + hi;
                        if (look || !__any_sync(kFull, live && !(t < kTileSum))) break;
                        look = true;
                    }
                    tmem_st32_nowait(tS, p[0]);
                    tmem_st32_nowait(tS + 32, p[1]);
                    l += t;
                    tmem_st_wait();
                    tc_fence_before();
                    warp_arrive(p_full + 8 * st);
                } else {
                    warp_arrive(p_full + 8 * st);
                }
            }
            const bool any = tiles_of(s, st) > 0;
            if (any) {
                mbar_wait_fast(o_full + 8 * st, o_par, failed);
                o_par ^= 1;
            }
            // (the join writes to the ring: the other stream's products first)
            if (kOwn && tiles_of(s, 1 - st) > 0) mbar_wait_fast(o_full + 8 * (1 - st), 0, failed);
            failed = __any_sync(kFull, failed);
            if (failed) break;
            tc_fence_after();
            if (!kOwn) {
                const size_t at = ((size_t)(s.item + blockIdx.x) * 2 + st) * kTileRows + row;
                if (live) a.part_ml[at] = make_float2(m, l);
                if (any && !idle) {
#pragma unroll 1
                    for (int c0 = 0; c0 < 128; c0 += 32) {
                        float o[32];
                        tmem_ld32(tO + c0, o);
                        if (live) {
                            float4* dst = reinterpret_cast<float4*>(a.part_o + at * 128 + c0);
#pragma unroll
                            for (int c = 0; c < 32; c += 4) dst[c >> 2] = make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]);
                        }
                    }
                }
            } else {
                // Join: the two streams of a split pair, then the prefix's parts.  A thread has its row's statistics; the
                // sums go through shared memory (the ring is at rest), where the warp takes its 32 rows one after
                // another, a lane four dims, so that parts are read and results written in whole lines (thread by
                // thread, row by row, this took 25 us of a CTA's 35).
                constexpr int kPitch = 132;  // floats: 16-byte columns of 8 rows fall into different banks
                float* mine = reinterpret_cast<float*>(gbase) + warp * 32 * kPitch;
                const float* other = mine + 4 * 32 * kPitch;
                float2* xml = reinterpret_cast<float2*>(gbase + 8 * 32 * kPitch * 4);
                float M = m, L = l, w_me = 1.f, w_ot = 0.f;
                auto put = [&](float scale) {
#pragma unroll 1
                    for (int c0 = 0; c0 < 128; c0 += 32) {
                        float o[32];
                        if (any) tmem_ld32(tO + c0, o);
#pragma unroll
                        for (int c = 0; c < 32; c += 4)
                            *reinterpret_cast<float4*>(mine + lane * kPitch + c0 + c) =
                                any && scale > 0.f ? make_float4(o[c] * scale, o[c + 1] * scale, o[c + 2] * scale, o[c + 3] * scale)
                                                   : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                };
                if (s.split) {
                    if (st == 1) {
                        xml[row] = make_float2(m, l);
                        put(1.f);
                        warp_arrive(x_full);
                        break;
                    }
                    mbar_wait_fast(x_full, 0, failed);
                    failed = __any_sync(kFull, failed);
                    if (failed) break;
                    const float2 ot = xml[row];
                    M = fmaxf(m, ot.x);
                    w_me = m == -INFINITY ? 0.f : ex2_approx((m - M) * kLogitScaleLog2);
                    w_ot = ot.x == -INFINITY ? 0.f : ex2_approx((ot.x - M) * kLogitScaleLog2);
                    L = l * w_me + ot.y * w_ot;
                }
                asm volatile("griddepcontrol.wait;" ::: "memory");
                const int token = (st ? s.tok1 : s.tok0) + own_token, jj = row - own_token * a.r;
                RowParts rp{0, 0, 0};
                if (live && plan.work > 0) rp = row_parts(a, plan, s.h, token, jj);
                float Mall = M;
                for (int k = 0; k < rp.n; ++k) Mall = fmaxf(Mall, __ldcg(&a.part_ml[rp.at + k * rp.step]).x);
                const float wm = M == -INFINITY ? 0.f : ex2_approx((M - Mall) * kLogitScaleLog2);
                w_me *= wm;
                w_ot *= wm;
                L *= wm;
                for (int k = 0; k < rp.n; ++k) {
                    const float2 ml = __ldcg(&a.part_ml[rp.at + k * rp.step]);
                    if (ml.y > 0.f) L += ml.y * ex2_approx((ml.x - Mall) * kLogitScaleLog2);
                }
                const float inv = L > 0.f ? 1.0f / L : 0.f;
                const size_t to = (size_t)token * a.Hq + s.h * a.r + jj;
                if (live && a.lse) a.lse[to] = L > 0.f ? Mall * kRsqrtD + logf(L) : -INFINITY;
                put(w_me);
                __syncwarp();
                const int count = min(32, (st ? s.toks1 : s.toks0) * a.r - 32 * (warp & 3));  // rows of this warp in use
#pragma unroll 1
                for (int i0 = 0; i0 < count; i0 += 4) {
                    float4 x[4];
                    int n[4], most = 0;
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int i = i0 + u;  // (rows past count: computed from what lies there, not written)
                        x[u] = *reinterpret_cast<const float4*>(mine + i * kPitch + 4 * lane);
                        const float wo = __shfl_sync(kFull, w_ot, i);
                        if (wo > 0.f) {
                            const float4 y = *reinterpret_cast<const float4*>(other + i * kPitch + 4 * lane);
                            x[u] = make_float4(fmaf(y.x, wo, x[u].x), fmaf(y.y, wo, x[u].y), fmaf(y.z, wo, x[u].z), fmaf(y.w, wo, x[u].w));
                        }
                        n[u] = __shfl_sync(kFull, rp.n, i);
                        most = max(most, n[u]);
                    }
#pragma unroll 1
                    for (int k = 0; k < most; ++k) {
                        float2 ml[4];
                        float4 v[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const size_t at = __shfl_sync(kFull, (unsigned long long)(rp.at + k * rp.step), i0 + u);
                            ml[u] = make_float2(0.f, 0.f);
                            v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (k < n[u]) {
                                ml[u] = __ldcg(&a.part_ml[at]);
                                v[u] = __ldcg(reinterpret_cast<const float4*>(a.part_o + at * 128) + lane);
                            }
                        }
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const float Mu = __shfl_sync(kFull, Mall, i0 + u);
                            if (ml[u].y > 0.f) {
                                const float wp = ex2_approx((ml[u].x - Mu) * kLogitScaleLog2);
                                x[u] = make_float4(fmaf(v[u].x, wp, x[u].x), fmaf(v[u].y, wp, x[u].y), fmaf(v[u].z, wp, x[u].z),
                                                   fmaf(v[u].w, wp, x[u].w));
                            }
                        }
                    }
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const float iu = __shfl_sync(kFull, inv, i0 + u);
                        const size_t tu = __shfl_sync(kFull, (unsigned long long)to, i0 + u);
                        if (i0 + u < count)
                            *reinterpret_cast<uint2*>(a.out + tu * 128 + 4 * lane) =
                                make_uint2(pack_bf16(x[u].x * iu, x[u].y * iu), pack_bf16(x[u].z * iu, x[u].w * iu));
                    }
                }
            }
            tc_fence_before();  // (O has been read: the next segment's first P releases it)
            step0 += s.n1 - s.n0;
        }
    }
    if (failed) bad |= HSQ_DEVERR_WAIT;
    if (bad) atomicOr(a.err, bad);
    tc_fence_before();
    __syncthreads();
    if (kOwn) {
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        asm volatile("griddepcontrol.wait;" ::: "memory");  // (every thread: a grid that ends has seen its predecessor end)
    }
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------------------
// Few rows: one cluster per (request, KV head), NT tiles of 8 rows (tokens x heads).  The
// cluster's warps take groups of 16 keys in turn; a warp's fragments come straight from the
// pages in 16-byte loads, without shared memory or barriers:
//   S^T (16 keys x 8 rows) = K (A operand, 16 x 16) Q^T: the product over the 128 dims
//     may take them in any order, so lane (g, t) reads dims [32 j + 8 t, + 8) of keys g and
//     g + 8 (j = 0..3) and feeds two k-steps from each load; Q is read the same way;
//   O^T (dims x 8 rows) += V^T (A) P^T (B): lane (g, t) reads dims [64 c + 8 g, + 8) of keys
//     2t, 2t + 1, 2t + 8, 2t + 9 and interleaves pairs of keys with byte permutes; row g
//     of MMA i is dim 8 g + i, row g + 8 dim 64 + 8 g + i.  P^T comes from S^T by two 8 x 8
//     transposes (movmatrix).
// So 16 rows cost two MMAs where 8 cost one, and a warp's bytes in flight are its
// registers: the next group's keys are on their way while this one's values arrive.
// Bound by HBM.
// ---------------------------------------------------------------------------------------

constexpr int kFewWarps = 4, kFewThreads = 32 * kFewWarps;

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};\n"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}

template <int NT>
__global__ void __launch_bounds__(kFewThreads) shared_few_kernel(const __grid_constant__ SharedArgs a) {
    constexpr int kRows = 8 * NT;
    __shared__ float s_o[kFewWarps][kRows][128];
    __shared__ float2 s_ml[kFewWarps][kRows];
    __shared__ float2 s_cta[kRows];
    __shared__ float4 s_x[kFewWarps][32];
    namespace cg = cooperative_groups;
    cg::cluster_group cl = cg::this_cluster();
    const int rank = blockIdx.x, splits = gridDim.x, h = blockIdx.y, b = blockIdx.z;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    int bad = 0;
    const Request rq = request_of(a, b, bad);
    const int rows = rq.n * a.r;
    if (rows == 0 || rows > kFewRows) {  // (the same for the whole cluster)
        if (bad && tid == 0) atomicOr(a.err, bad);
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    const int32_t* ids = a.table + (size_t)b * a.width;
    const int groups = (rq.len + 15) >> 4, stride = splits * kFewWarps;

    uint32_t qf[NT][8][2];
    int lim[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int row = 8 * nt + g;
        const bool in = row < rows;
        const uint16_t* src = a.q + ((size_t)(rq.first + (in ? row / a.r : 0)) * a.Hq + h * a.r + (in ? row % a.r : 0)) * 128 + 8 * t;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint4 x = in ? *reinterpret_cast<const uint4*>(src + 32 * j) : make_uint4(0, 0, 0, 0);
            qf[nt][2 * j][0] = x.x;
            qf[nt][2 * j][1] = x.y;
            qf[nt][2 * j + 1][0] = x.z;
            qf[nt][2 * j + 1][1] = x.w;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int rr = 8 * nt + 2 * t + e;
            lim[nt][e] = rr < rows ? min(rq.len, rq.len - rq.n + rr / a.r + 1) : 0;
        }
    }
    float o[NT][8][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
    }
    // offset of key 16 s in the pool, or -1 (no page there)
    auto place = [&](int s) -> long long {
        if (s >= groups) return -1;
        const int id = ids[(16 * s) >> a.page_shift];
        if (id < 0 || id >= a.n_pages) {
            bad |= HSQ_DEVERR_PAGE;
            return -1;
        }
        return ((((long long)id * a.Hkv + h) << a.page_shift) + ((16 * s) & (a.page_n - 1))) * 128;
    };
    uint4 kf[2][4];
    // keys past the length (and of no page) read as zero, so that nothing stale enters a product
    auto load_k = [&](int s, long long at) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const bool in = at >= 0 && 16 * s + g + 8 * e < rq.len;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                kf[e][j] = in ? __ldcs(reinterpret_cast<const uint4*>(a.pk + at + (g + 8 * e) * 128 + 32 * j + 8 * t))
                              : make_uint4(0, 0, 0, 0);
        }
    };
    int s = rank * kFewWarps + warp;
    long long at = place(s);
    if (s < groups) load_k(s, at);
#pragma unroll 1
    for (; s < groups; s += stride) {
        const long long ahead = place(s + stride);
        uint4 vf[4][2];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int key = 2 * t + (e & 1) + 8 * (e >> 1);
            const bool in = at >= 0 && 16 * s + key < rq.len;
#pragma unroll
            for (int c = 0; c < 2; ++c)
                vf[e][c] = in ? __ldcs(reinterpret_cast<const uint4*>(a.pv + at + key * 128 + 64 * c + 8 * g))
                              : make_uint4(0, 0, 0, 0);
        }
        float x[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                mma_16816(x[nt], kf[0][j].x, kf[1][j].x, kf[0][j].y, kf[1][j].y, qf[nt][2 * j][0], qf[nt][2 * j][1]);
                mma_16816(x[nt], kf[0][j].z, kf[1][j].z, kf[0][j].w, kf[1][j].w, qf[nt][2 * j + 1][0], qf[nt][2 * j + 1][1]);
            }
        if (s + stride < groups) load_k(s + stride, ahead);
        bool raise = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {  // key g + 8 (e >> 1), row 2 t + (e & 1)
                if (at < 0 || 16 * s + g + 8 * (e >> 1) >= lim[nt][e & 1]) x[nt][e] = -INFINITY;
                raise |= x[nt][e] * kLogitScaleLog2 > m[nt][e & 1] * kLogitScaleLog2 + kRaise;
            }
        if (__any_sync(kFull, raise)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(m[nt][e], fmaxf(x[nt][e], x[nt][e + 2]));
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, d));
                    const float alpha = mx == -INFINITY ? 1.f : ex2_approx((m[nt][e] - mx) * kLogitScaleLog2);
                    m[nt][e] = mx;
                    l[nt][e] *= alpha;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        o[nt][i][e] *= alpha;
                        o[nt][i][e + 2] *= alpha;
                    }
                }
        }
        uint32_t pf[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float off = m[nt][e & 1] == -INFINITY ? 0.f : m[nt][e & 1] * kLogitScaleLog2;
                p[e] = ex2_approx(fmaf(x[nt][e], kLogitScaleLog2, -off));
                l[nt][e & 1] += p[e];
            }
            pf[nt][0] = transpose_8x8(pack_bf16(p[0], p[1]));
            pf[nt][1] = transpose_8x8(pack_bf16(p[2], p[3]));
        }
        const uint32_t* v[4][2];
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int c = 0; c < 2; ++c) v[e][c] = reinterpret_cast<const uint32_t*>(&vf[e][c]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t sel = (i & 1) ? 0x7632u : 0x5410u;
            const uint32_t a0 = __byte_perm(v[0][0][i >> 1], v[1][0][i >> 1], sel);
            const uint32_t a1 = __byte_perm(v[0][1][i >> 1], v[1][1][i >> 1], sel);
            const uint32_t a2 = __byte_perm(v[2][0][i >> 1], v[3][0][i >> 1], sel);
            const uint32_t a3 = __byte_perm(v[2][1][i >> 1], v[3][1][i >> 1], sel);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_16816(o[nt][i], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
        }
        at = ahead;
    }

    // ---- join: the CTA's warps, the cluster's CTAs, the prefix's parts ----
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[nt][e] += __shfl_xor_sync(kFull, l[nt][e], d);
            const int row = 8 * nt + 2 * t + e;
            if (g == 0) s_ml[warp][row] = make_float2(m[nt][e], l[nt][e]);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float4* dst = reinterpret_cast<float4*>(&s_o[warp][row][64 * c + 8 * g]);
                dst[0] = make_float4(o[nt][0][e + 2 * c], o[nt][1][e + 2 * c], o[nt][2][e + 2 * c], o[nt][3][e + 2 * c]);
                dst[1] = make_float4(o[nt][4][e + 2 * c], o[nt][5][e + 2 * c], o[nt][6][e + 2 * c], o[nt][7][e + 2 * c]);
            }
        }
    }
    if (bad) atomicOr(a.err, bad);
    __syncthreads();
    for (int row = 0; row < rows; ++row) {  // thread = dim
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) M = fmaxf(M, s_ml[w][row].x);
        float L = 0.f, x = 0.f;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) {
            const float2 ml = s_ml[w][row];
            if (ml.y > 0.f) {
                const float c = ex2_approx((ml.x - M) * kLogitScaleLog2);
                L = fmaf(ml.y, c, L);
                x = fmaf(s_o[w][row][tid], c, x);
            }
        }
        s_o[0][row][tid] = x;  // (this thread alone reads and writes the column)
        if (tid == 0) s_cta[row] = make_float2(M, L);
    }
    if (splits > 1) cl.sync(); else __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // This CTA's rows (every splits-th), one warp a row, or two or four warps where there are
    // that few rows: lane k holds the weights of parts k, k + 32, ..., then the warp adds
    // the parts up, a lane four dims.  Loads do not wait for one another but for that one step.
    const PrefixPlan plan = prefix_plan(a);
    const int mine = (rows - rank + splits - 1) / splits;                  // (rows > rank, or none)
    const int per = mine == 1 ? kFewWarps : mine == 2 ? kFewWarps / 2 : 1;  // warps a row
    for (int i0 = 0; i0 < mine; i0 += kFewWarps / per) {
        const int i = i0 + warp / per, sub = warp % per;
        const bool live = i < mine;
        const int row = rank + (live ? i : 0) * splits, token = rq.first + row / a.r, jj = row % a.r;
        RowParts rp{0, 0, 0};
        if (live && plan.work > 0) rp = row_parts(a, plan, h, token, jj);
        // parts: the cluster's CTAs 0 .. splits - 1, then the prefix's
        const int n = live ? splits + rp.n : 0;
        float M = -INFINITY;
        for (int k = lane; k < n; k += 32)
            M = fmaxf(M, k < splits ? cl.map_shared_rank(s_cta, k)[row].x : __ldcg(&a.part_ml[rp.at + (k - splits) * rp.step]).x);
#pragma unroll
        for (int d = 16; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, d));
        float L = 0.f;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k0 = 0; k0 < n; k0 += 32) {
            float wt = 0.f;  // weight of part k0 + lane
            if (k0 + lane < n) {
                const int k = k0 + lane;
                const float2 ml = k < splits ? cl.map_shared_rank(s_cta, k)[row] : __ldcg(&a.part_ml[rp.at + (k - splits) * rp.step]);
                if (ml.y > 0.f) {
                    wt = ex2_approx((ml.x - M) * kLogitScaleLog2);
                    L = fmaf(ml.y, wt, L);
                }
            }
            const int stop = min(32, n - k0);
#pragma unroll 8
            for (int e = sub; e < stop; e += per) {
                const float wk = __shfl_sync(kFull, wt, e);
                const int k = k0 + e;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (wk > 0.f)
                    v = k < splits ? *reinterpret_cast<const float4*>(cl.map_shared_rank(&s_o[0][row][4 * lane], k))
                                   : __ldcg(reinterpret_cast<const float4*>(a.part_o + (rp.at + (k - splits) * rp.step) * 128) + lane);
                x.x = fmaf(v.x, wk, x.x);
                x.y = fmaf(v.y, wk, x.y);
                x.z = fmaf(v.z, wk, x.z);
                x.w = fmaf(v.w, wk, x.w);
            }
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) L += __shfl_xor_sync(kFull, L, d);
        if (per > 1) {
            s_x[warp][lane] = x;
            __syncthreads();
            for (int w = 1; w < per; ++w) {
                const float4 v = s_x[warp - sub + (sub + w) % per][lane];
                x.x += v.x;
                x.y += v.y;
                x.z += v.z;
                x.w += v.w;
            }
        }
        if (live && sub == 0) {
            const size_t to = (size_t)token * a.Hq + h * a.r + jj;
            const float inv = L > 0.f ? 1.0f / L : 0.f;
            *reinterpret_cast<uint2*>(a.out + to * 128 + 4 * lane) =
                make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
            if (a.lse && lane == 0) a.lse[to] = L > 0.f ? M * kRsqrtD + logf(L) : -INFINITY;
        }
    }
    if (splits > 1) cl.sync();  // (the others may still read this CTA's part)
}

// ---- host side --------------------------------------------------------------------------

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
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
bool encode_rows(CUtensorMap* map, void* p, uint64_t rows, uint32_t box_rows) {
    const cuuint64_t dims[2] = {128, rows}, strides[1] = {256};
    const cuuint32_t box[2] = {64, box_rows}, es[2] = {1, 1};
    return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// queries [rows][Hq][128]: a box is `tokens` tokens x the r heads of a KV head x 64 columns
bool encode_q(CUtensorMap* map, const void* p, uint64_t rows, uint64_t Hq, uint32_t r, uint32_t tokens) {
    const cuuint64_t dims[3] = {128, Hq, rows}, strides[2] = {256, 256 * Hq};
    const cuuint32_t box[3] = {64, r, tokens}, es[3] = {1, 1, 1};
    return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, es,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// workspace: part_o, then part_ml, of Hkv * pairs + runs slots
struct Parts { long long slots; size_t o_bytes, bytes; int runs; };

Parts parts_of(const hsq_ctx* ctx, int rows, int prefix_len) {
    Parts p{0, 0, 256, 0};
    if (prefix_len == 0) return p;
    const int tpt = kTileRows / ctx->r, tiles = (rows + tpt - 1) / tpt, pairs = (tiles + 1) / 2;
    const long long items = (long long)ctx->cfg.n_kv_heads * pairs;
    const long long work = items * ((prefix_len + kTileKeys - 1) / kTileKeys);
    p.runs = (int)std::min<long long>(ctx->num_sms, work);
    p.slots = items + p.runs;
    p.o_bytes = (size_t)p.slots * 2 * kTileRows * 128 * 4;
    p.bytes = p.o_bytes + (size_t)p.slots * 2 * kTileRows * 8;
    return p;
}

cudaError_t launch(const void* fn, dim3 grid, int threads, size_t smem, cudaStream_t st, int cluster, bool after,
                   void** args) {
    cudaLaunchConfig_t lc{};
    lc.gridDim = grid;
    lc.blockDim = dim3(threads);
    lc.dynamicSmemBytes = smem;
    lc.stream = st;
    cudaLaunchAttribute at[2];
    int n = 0;
    if (cluster > 1) {
        at[n].id = cudaLaunchAttributeClusterDimension;
        at[n].val.clusterDim.x = cluster;
        at[n].val.clusterDim.y = at[n].val.clusterDim.z = 1;
        ++n;
    }
    if (after) {
        at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    lc.attrs = at;
    lc.numAttrs = n;
    return cudaLaunchKernelExC(&lc, fn, args);
}

}  // namespace

extern "C" {

hsq_status hsq_shared_attn_workspace_size(const hsq_ctx* ctx, int rows, int B, int prefix_len, int max_new,
                                          size_t* bytes) {
    if (!ctx || !bytes) return hsq::fail(nullptr, HSQ_ERR_INVALID, "ctx or bytes is NULL");
    if (rows < 1 || B < 1 || prefix_len < 0 || max_new < 1)
        return hsq::fail(nullptr, HSQ_ERR_INVALID, "rows, B and max_new must be positive, prefix_len not negative");
    *bytes = parts_of(ctx, rows, prefix_len).bytes;
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
    const Parts parts = parts_of(ctx, rows, prefix_len);
    if (workspace_bytes < parts.bytes)
        return hsq::fail(ctx, HSQ_ERR_INVALID, "workspace smaller than hsq_shared_attn_workspace_size");
    if ((st = hsq::check_device(ctx)) != HSQ_OK) return st;
    const int r = ctx->r, Hkv = ctx->cfg.n_kv_heads, tpt = kTileRows / r;
    SharedArgs a{};
    a.q = static_cast<const uint16_t*>(q);
    a.pk = static_cast<const uint16_t*>(pages->k);
    a.pv = static_cast<const uint16_t*>(pages->v);
    a.q_start = q_start; a.lens = lens; a.table = table; a.prefix = prefix;
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse_opt;
    a.rows = rows; a.B = B; a.width = width; a.prefix_len = prefix_len; a.max_new = max_new;
    a.n_pages = pages->n_pages; a.page_n = pages->page_n;
    a.page_shift = pages->page_n == 16 ? 4 : pages->page_n == 32 ? 5 : pages->page_n == 64 ? 6 : 7;
    a.Hq = ctx->cfg.n_q_heads; a.Hkv = Hkv; a.r = r; a.tpt = tpt; a.runs = parts.runs;
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + parts.o_bytes);
    a.err = ctx->d_err;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool many = (long long)max_new * r > kFewRows;
    CUtensorMap mq, mk, mv;
    if (prefix_len > 0 || many) {
        if (!encode_fn()) return hsq::fail(ctx, HSQ_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
        const uint64_t n = (uint64_t)pages->n_pages * Hkv * pages->page_n;
        if (!encode_q(&mq, q, rows, a.Hq, r, tpt) || !encode_rows(&mk, pages->k, n, pages->page_n) ||
            !encode_rows(&mv, pages->v, n, pages->page_n))
            return hsq::fail(ctx, HSQ_ERR_CUDA, "cuTensorMapEncodeTiled refused a tensor map");
    }
    cudaError_t e = cudaSuccess;
    bool after = false;
    void* tc_args[] = {&mq, &mk, &mv, &a};
    void* few_args[] = {&a};
    if (prefix_len > 0) {
        const void* fn = (const void*)shared_tc_kernel<false>;
        if ((e = hsq::raise_smem_limit(fn, ctx->device, kTcSmem)) != cudaSuccess)
            return hsq::cuda_fail(ctx, e, "cudaFuncSetAttribute(shared_attn)");
        e = launch(fn, dim3(parts.runs), kTcThreads, kTcSmem, s, 1, false, tc_args);
        if (e != cudaSuccess) return hsq::cuda_fail(ctx, e, "shared_attn prefix");
        after = true;
    }
    if (many) {
        const void* fn = (const void*)shared_tc_kernel<true>;
        if ((e = hsq::raise_smem_limit(fn, ctx->device, kTcSmem)) != cudaSuccess)
            return hsq::cuda_fail(ctx, e, "cudaFuncSetAttribute(shared_attn)");
        const int ids = rows / (2 * tpt) + B;
        if (ids > 65535) return hsq::fail(ctx, HSQ_ERR_INVALID, "too many rows");
        e = launch(fn, dim3(Hkv, ids), kTcThreads, kTcSmem, s, 1, after, tc_args);
        if (e != cudaSuccess) return hsq::cuda_fail(ctx, e, "shared_attn rows");
        after = true;
    }
    int splits = 1;
    while (splits < 8 && (long long)B * Hkv * splits < 3 * ctx->num_sms &&
           (long long)width * pages->page_n > 16LL * kFewWarps * 4 * splits)
        splits *= 2;
    const void* fn = many || max_new * r > 8 ? (const void*)shared_few_kernel<2> : (const void*)shared_few_kernel<1>;
    e = launch(fn, dim3(splits, Hkv, B), kFewThreads, 0, s, splits, after, few_args);
    if (e != cudaSuccess) return hsq::cuda_fail(ctx, e, "shared_attn few");
    return HSQ_OK;
}

}  // extern "C"
