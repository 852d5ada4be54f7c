// Attention of a batch whose requests share a prefix (hsq_shared_attn).
//
// For row i of request b (token j of its n new ones) and query head jq of KV head
// h: one softmax, scale 1/sqrt(128), over the prefix's tokens and the request's own
// tokens s <= len - n + j (of those that its table holds).  A softmax over the union of key sets is the weighted
// sum of the softmaxes over each: with m, l, o a reference exponent, the sum of
// exp(x - m) and the sum of exp(x - m) v of a part,
//     out = sum_p exp(m_p - M) o_p / sum_p exp(m_p - M) l_p,   M = max_p m_p,
// so a pass over the prefix serves rows of any requests, a pass over a request's own pages all of
// its rows, and the parts are joined at the end.
//
// Rows.  The r = Hq / Hkv query heads of a KV head and the rows of the batch make
// one row index (token * r + head): a tile of 128 rows holds floor(128 / r) tokens
// of ANY requests for the prefix, so the tensor cores see full tiles in a decode
// step too.
//
// Work.  A request is short when its new tokens fit one tile (n <= 128 / r: decode,
// proposals), else long (a prompt's chunk).  Four kinds of items:
//   A  (KV head, pair of row tiles of the short requests' tokens, packed): the prefix;
//   B  (short request of more than 16 rows, n r > 16, KV head): its own tokens;
//   C  (long request, KV head, pair of its row tiles): the prefix, then its own
//      tokens up to the pair's last;
//   D  (request of up to 16 rows, KV head): its own tokens, by single warps.
// An item is a run of key tiles (D: of groups of 16 keys) with a cost each.  The SMs (a
// persistent CTA each) are dealt to A and to the rest by their costs; each side's items
// one after another make a line of cost, cut into as many equal runs as it has CTAs.  So
// some SMs work on A, bound by the tensor cores, while others stream D's pages, bound
// by HBM, and both are in use throughout.  A's line is the prefix's keys, head by head; up
// to four pairs of row tiles have a line (a lane) each, cut alike, so that CTAs side by side read
// the same key tiles at the same time and HBM gives them once; more pairs go over the prefix one after
// another, as every pair of a long request's row tiles does.
//
// Three kernels, the later two launched with programmatic serialization (their set-up
// runs while the one before ends):
//   shared_plan_kernel   checks the lengths, adds up the line (one CTA);
//   shared_tc_kernel     the items' tiles on the tensor cores; a C item that no cut
//                        divides is written at once, everything else leaves its parts (m, l, o in
//                        fp32) in the workspace;
//   shared_join_kernel   joins the parts.
//
// Rounding: q, k and v are bf16, products exact, sums fp32; the softmax weights are
// rounded to bf16 for the product with the values (an error of 2^-8 of each weight
// at most, random over the keys, where the output's own rounding is up to 2^-8 of the
// result); l sums them before that rounding.  Against 64 bits the result is off by 0.0018 to
// 0.0023 of its size, where rounding the exact one gives 0.0017.  (Two bf16 terms for each weight, as the
// prefill has them, would be half as many products again on the pipe that bounds the prompts.)
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "hsq_ctx.h"
#include "hsq_device.cuh"
#include "hsq_paged.cuh"
#include "hsq_tc.cuh"

namespace {

using namespace hsq_tc;
using namespace hsq_paged;

constexpr int kTileRows = 128, kTileKeys = 128;
constexpr float kTileSum = 65536.f;  // sum of a tile's 128 weights from which the maximum is taken anew
// Cost of a key tile, per key: of A for two row tiles (tensor cores) and for one (tensor cores and loads), of C, of
// B (loads); and what an item of B or A costs beside its tiles, in keys (its epilogue; the start of its loads).  Set by
// timing; one up or down, in us: pairs 112.8 / 107.6 / 109.0 (9, 10, 11) and D's groups below 114.3 / 107.6 / 116.4 (3, 4,
// 5) for 128 requests over a prefix of 32K; one tile 97.5 instead of 91.9 (9, 8) for 8 requests with a chunk of 1000
// among them; C 93.8 / 92.0 / 91.3 (6, 7, 8) for those and 361 / 359 / 359.5 for four prompts of 1024; A's items
// without the 128 keys 38.1 instead of 36.4 for 16 requests over 8K.  (Runs of one build differ by 3 %.)  They do not
// know the head ratio or the rows of a few-rows item.
constexpr int kCostPair = 10, kCostOne = 8, kCostLong = 7, kCostOwn = 6, kItemKeys = 96, kItemKeysA = 128;
// D: requests of up to kFewRows rows; a group is 16 keys of one warp, kFewWarps warps share a CTA's run
constexpr int kFewRows = 16, kFewWarps = 8, kCostFew = 4, kFewItemKeys = 64;

struct PlanHead {
    long long lane_a;                // A: length of a lane's line, and of one KV head's part of it
    long long head_a;
    long long work, work_c, work_t;  // the others' line: [C | B | D], work_t where D begins
    int lanes, cuts_a, runs_a;       // A: lanes (1: the pairs one after another), runs of each, CTAs
    int tokens, tiles, pairs;        // of the short requests
    int dense;                       // 1: the short requests' tokens are the rows [base, base + tokens)
    int base;
    int runs;                        // the others' CTAs: runs_a and up
    long long each_a, each_w;        // lane_a / cuts_a, work / runs
    int rest_a, rest_w;              // and their remainders
};  // (no run is shorter than a tile, so that every run inside an item holds one)

struct SharedArgs {
    const int32_t *q_start, *lens, *table, *prefix;
    const uint16_t* q;
    uint16_t* out; float* lse;
    int rows, B, width, prefix_len, prefix_tiles, max_new, n_pages, page_n, page_shift, Hq, Hkv, r;
    int tpt;   // tokens of a row tile: 128 / r
    int runs;  // CTAs of the main kernel: an SM each
    int own_rows;  // most rows of a B item
    int tokens_cap;  // most tokens that short requests can have
    // workspace
    PlanHead* head;
    // [B][2] first row, rows, own tokens (no more than its table holds), short tokens before it | own tokens before its first
    // row (row j sees the first min(own tokens, that + j + 1)), tokens of the B requests before it
    int4* req;
    int* of;                // [short tokens] their requests
    long long *c_at, *b_at, *d_at; // [B + 1] cost of the C, B and D items before request b
    int* cut;               // [runs][16 ints] the C item that run c is the second to work on (see CutRecord)
    // parts: o [slot][2 streams][128 dims][rows], ml [slot][2 streams][rows] (maximum of q.k, unscaled; sum).  A slot of A and C has
    // 128 rows, one of B as many as its item: they lie one item behind another, and own_rows further for each run (see own_slot).
    float *a_o, *b_o, *c_o;
    float2 *a_ml, *b_ml, *c_ml;
    // D's: o [slot][rows][128], ml [slot][rows]
    float* d_o;
    float2* d_ml;
    int few_rows;  // 8 or 16
    int polls;     // of a wait, before it has run out
    int fault;     // HSQ_FAULT_WAIT_*: the roles of the main kernel that give up at a certain wait (0 but in tests)
    int* err;
};

// n / d (n >= 0, d > 0) where the quotient is below 2^16: in float within one of it, then exactly.  (A 64-bit division
// is some hundred instructions; the lookups here and in the join have a dozen of them.)
__device__ __forceinline__ int small_quotient(long long n, long long d) {
    const int q = (int)__fdividef((float)n, (float)d);
    const long long rest = n - q * d;
    return q + (rest >= d) - (rest < 0);
}

// A line cut into equal runs: the run that holds place w, and where run i begins (floor(line i / runs), from the
// quotient and the remainder of line / runs).
__device__ __forceinline__ int run_of(long long line, int runs, long long w) { return small_quotient((w + 1) * runs - 1, line); }
__device__ __forceinline__ long long run_begin(long long each, int rest, int runs, int i) {
    i = min(i, runs);
    return each * i + (unsigned)(rest * i) / (unsigned)runs;
}
__device__ __forceinline__ long long a_begin(const PlanHead& p, int i) { return run_begin(p.each_a, p.rest_a, p.cuts_a, i); }
__device__ __forceinline__ long long w_begin(const PlanHead& p, int i) { return run_begin(p.each_w, p.rest_w, p.runs, i); }

__device__ __forceinline__ long long few_cost(int len) { return (long long)(((len + 15) >> 4) * 16 + kFewItemKeys) * kCostFew; }

// D: the warp (of all CTAs' warps) that takes the group at place x: a CTA's share of D is cut into eight equal parts
// (into as many as it has groups, the last ones of the eight, where D begins inside its run)
struct FewShare { long long lo, hi; int parts; };
__device__ __forceinline__ FewShare few_share(const PlanHead& p, int i) {  // i: of the others' runs
    FewShare s;
    s.lo = max(w_begin(p, i), p.work_t);
    s.hi = w_begin(p, i + 1);
    s.parts = max(1, (int)min((long long)kFewWarps, max(s.hi - s.lo, 0LL) / (16u * kCostFew)));
    return s;
}
// where part j begins: floor(length j / parts)
__device__ __forceinline__ long long few_begin(const FewShare& s, int j) {
    const long long n = s.hi - s.lo;  // (fewer parts than kFewWarps: the length is small)
    return s.lo + (s.parts == kFewWarps ? n * j / kFewWarps : (long long)((unsigned)n * j / (unsigned)s.parts));
}
__device__ __forceinline__ int few_warp_of(const PlanHead& p, long long x) {
    const int i = run_of(p.work, p.runs, x);
    const FewShare s = few_share(p, i);
    return i * kFewWarps + kFewWarps - s.parts + small_quotient((x - s.lo + 1) * s.parts - 1, s.hi - s.lo);
}

// virtual keys of unit u of a long request (never fewer than the real ones): its cost is kCostLong a key
__device__ __forceinline__ long long unit_base(const SharedArgs& a, int ahead) {
    return (long long)a.prefix_tiles * kTileKeys + max(ahead, 0);
}
// virtual keys of an item of A (0: there is none)
__device__ __forceinline__ long long a_keys(const SharedArgs& a) {
    return a.prefix_tiles ? (long long)a.prefix_tiles * kTileKeys + kItemKeysA : 0;
}
// Rows before the part of a B item (KV head h of a request of n tokens, `before` tokens of B requests before it) that run i leaves:
// from one part to the next either the item goes on by one, or the run does.
__device__ __forceinline__ int own_slot(const SharedArgs& a, int before, int n, int h, int i) {
    return (before * a.Hkv + h * n) * a.r + i * a.own_rows;
}
// cost of the units before u (u < number of units), D tokens each
__device__ __forceinline__ long long units_before(long long base, int D, long long u) {
    return kCostLong * (u * base + D * (u * (u + 1) / 2));
}

// ---------------------------------------------------------------------------------------
// Plan: one CTA scans the requests.
// ---------------------------------------------------------------------------------------

constexpr int kPlanThreads = 512;

__global__ void __launch_bounds__(kPlanThreads) shared_plan_kernel(const __grid_constant__ SharedArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ long long s_w[4][kPlanThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int bad = 0, disorder = 0;
    long long before[4] = {0, 0, 0, 0};  // short tokens (and, from bit 32 on, those of B requests), C, B and D cost
    for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int first = 0, n = 0, len = 0, ahead = 0, l = 0;
        bool wrong = false;
        if (b < a.B) {
            const int s = a.q_start[b], e = a.q_start[b + 1];
            l = a.lens[b];
            first = s;
            n = e - s;
            wrong = s < 0 || e < s || e > a.rows || n > a.max_new;
        }
        // (no row may belong to two requests: the workspace has room for each row once)
        if (disorder |= __syncthreads_or(wrong)) {
            for (int c = 0; c < b && b < a.B; ++c) wrong |= a.q_start[c] > first && a.q_start[c] <= a.rows;
        }
        if (wrong) {
            bad |= HSQ_DEVERR_LEN;
            first = n = 0;
        }
        if (b < a.B) {
            len = (int)min((long long)max(l, 0), (long long)a.width << a.page_shift);
            if (len != l || len < n) bad |= HSQ_DEVERR_LEN;
            ahead = min(max(l, 0) - n, len);  // (by the length given: a table too short for it hides keys, but moves no row)
        }
        const bool brief = n <= a.tpt;
        long long x[4] = {brief ? n : 0, 0, 0, 0}, own[4];
        if (n > 0 && brief && len > 0) {
            if (n * a.r > kFewRows) {
                x[2] = (long long)a.Hkv * (len + kItemKeys) * kCostOwn;
                x[0] |= (long long)n << 32;
            } else {
                x[3] = a.Hkv * few_cost(len);
            }
        }
        if (!brief) {
            const int D = 2 * a.tpt, units = (n + D - 1) / D;
            const long long base = unit_base(a, ahead);
            x[1] = a.Hkv * (units_before(base, D, units - 1) + kCostLong * (base + n));
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            own[k] = x[k];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long u = __shfl_up_sync(kFull, x[k], o);
                if (lane >= o) x[k] += u;
            }
            if (lane == 31) s_w[k][warp] = x[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // (warps past the last request have nothing to add)
            long long t = before[k], mine = 0;
            for (int w = 0; w < min(kPlanThreads / 32, (a.B - b0 + 31) / 32); ++w) {
                if (w == warp) mine = t;
                t += s_w[k][w];
            }
            before[k] = t;
            x[k] += mine - own[k];
        }
        if (b < a.B) {
            a.req[2 * b] = make_int4(first, n, len, (int)x[0]);
            a.req[2 * b + 1] = make_int4(ahead, (int)(x[0] >> 32), 0, 0);
            for (int i = 0; i < (int)own[0]; ++i) a.of[(int)x[0] + i] = b;
            a.c_at[b] = x[1];
            a.b_at[b] = x[2];
            a.d_at[b] = x[3];
        }
        __syncthreads();
    }
    if (bad) atomicOr(a.err, bad);
    const int any_bad = __syncthreads_or(bad);
    if (tid == 0) {
        PlanHead h;
        h.tokens = (int)before[0];
        h.tiles = (h.tokens + a.tpt - 1) / a.tpt;
        h.pairs = (h.tiles + 1) >> 1;
        const long long keys = a_keys(a);
        const long long full = h.tiles >> 1, one = h.tiles & 1;
        // Lanes for up to four pairs.  With lanes and with one line, us: 2 pairs 108.2 / 108.2 (128 requests over 32K), 81.1 / 81.5
        // (over 2K), verification 46.9 / 47.1; 3 pairs 53.7 / 53.7; 4 pairs 67.4 / 68.0 (128 x 8 heads over 8K); 61 requests of 5 heads,
        // whose second lane is half empty, 44.2 / 40.5.  Eight lanes would gain for 8 pairs over a long prefix (240 / 257 over 32K, 107.9 /
        // 109.3 over 8K) and lose over a short one (89.8 / 88.1 over 1K).
        h.lanes = h.pairs <= 4 ? max(h.pairs, 1) : 1;
        // (lanes are cut alike, so a pair of one tile counts as a whole one there)
        h.head_a = h.pairs == 0 ? 0 : h.lanes == 1 ? keys * (full * kCostPair + one * kCostOne) : keys * kCostPair;
        h.lane_a = a.Hkv * h.head_a;
        h.work_c = before[1];
        h.work_t = h.work_c + before[2];
        h.work = h.work_t + before[3];
        h.base = a.q_start[0];
        h.dense = !any_bad && before[1] == 0;
        const long long work_a = a.Hkv * keys * (full * kCostPair + one * kCostOne), all = work_a + h.work;
        // CTAs for A, a multiple of the lanes; at least one for what there is of either
        int ga = 0;
        if (work_a > 0) {
            ga = (int)((work_a * a.runs / h.lanes + all / 2) / all) * h.lanes;
            ga = max(h.lanes, min(ga, (a.runs - (h.work > 0)) / h.lanes * h.lanes));
        }
        const int rate = (h.tiles > 1 ? kCostPair : kCostOne) * kTileKeys;
        h.cuts_a = (int)min((long long)(ga / h.lanes), h.lane_a / rate);
        h.runs_a = h.cuts_a * h.lanes;
        const int most = max(max(kCostLong, kCostOwn), kCostFew) * kTileKeys;
        h.runs = h.work > 0 ? (int)max(1LL, min((long long)(a.runs - ga), h.work / most)) : 0;
        h.each_a = h.cuts_a ? h.lane_a / h.cuts_a : 0;
        h.rest_a = h.cuts_a ? (int)(h.lane_a - h.each_a * h.cuts_a) : 0;
        h.each_w = h.runs ? h.work / h.runs : 0;
        h.rest_w = h.runs ? (int)(h.work - h.each_w * h.runs) : 0;
        *a.head = h;
        a.c_at[a.B] = before[1];
        a.b_at[a.B] = before[2];
        a.d_at[a.B] = before[3];
    }
}

// ---------------------------------------------------------------------------------------
// Main kernel.  One CTA per SM, 12 warps: softmax warps 0-3 (stream 0) and 4-7 (stream 1),
// warp 8 walks the run and loads keys and values, warp 9 issues the MMAs (one elected thread), warp 10 loads
// the queries, warp 11 fetches tensor maps and page ids ahead (168 registers a thread at launch, then 176 for the
// softmax warps, whose row of logits lives in registers, and 152 for the others; at the time four prompts 349 us, with 168 for
// all 357, with 184 and 136, where the warps of 136 spill, 357).  NT: D's tiles of 8 rows, 1 where max_new * r <= 8, else 2, which
// decode runs too (16 requests 37.1 and 37.3 us, 128 over 32K 107.5 and 128.6).
// A stream is a 128-row query tile with its S / P and O in tensor memory.  The two streams
// either hold two row tiles and share every key tile (so keys and values are loaded once
// for 256 rows), or (split) hold the same rows and take the key tiles in turn.  While
// one stream's softmax runs, the tensor cores work for the other.
//   shared memory: a ring of three K tiles and one of two V tiles, 32 KB each (TMA, 128-byte swizzle; in
//     one ring of five a key tile had to wait for the P V of three tiles before), two Q tiles;
//   tensor memory: S of stream s at columns 128 s (P, bf16, over its first 64), O at 256 + 128 s.
// What it reaches: four prompts of 1024 over a prefix of 8192 (32/8 heads, 0.58 TFLOP) 345 us of the call's 357
// to 366 (384 for seconds on end, under the power limit), 1.7 PFLOP/s, the tensor pipe 75 % of the time active; bound by the pipe and by what a key tile costs beside it (a
// 128 x 128 x 16 MMA takes 64 cycles in any of the forms used here, so a key tile of two row tiles 2048, 1.07 us at 1.9
// GHz; it takes 1.4).  128 requests over 32K: 98 us for 500 MB, 5.1 TB/s, bound by HBM with some 25 us
// of start and end.  Few requests (16 over 8K, 79 MB, 27 us): bound by the latencies of start, first loads and end.
// ---------------------------------------------------------------------------------------

constexpr int kTcThreads = 384, kKeyStages = 3, kValueStages = 2, kStages = kKeyStages + kValueStages, kQueue = 4;
constexpr uint32_t kTileBytes = 128 * 128 * 2, kHalfBytes = kTileBytes / 2;
constexpr uint32_t kOffQ = kStages * kTileBytes, kOffBars = kOffQ + 2 * kTileBytes;
// barriers: full[5] | empty[5] | q_full[2] | q_empty[2] | s_full[2] | p_full[2] | o_full[2] | tail | drain | seg_full[4] | seg_empty[4]
constexpr int kTcBars = 2 * kStages + 12 + 2 * kQueue;
static_assert(kTcBars % 2 == 0, "segments lie on 16-byte boundaries");
constexpr uint32_t kOffMask = kOffBars + 8 * kTcBars;  // [8] pages of a key tile that lie in the pool
constexpr uint32_t kOffSeg = kOffMask + 32;                  // [4] segments of the run
constexpr uint32_t kSegBytes = 96;
constexpr uint32_t kOffFew = kOffSeg + kQueue * kSegBytes + 16;  // (+ TMEM address) D's barriers, three a warp
constexpr uint32_t kTcSmem = kOffFew + 8 * 8 * 3 + 1024;         // + alignment
constexpr int kSegReaders = 10;                              // 8 softmax warps, the MMA thread, the query loader

// The key tiles [n0, n1) of an item that lie in this CTA's run.
enum : int { kEnd = -1, kPrefixItem = 0, kOwnItem = 1, kWholeItem = 2, kCutItem = 3 };
struct alignas(16) Segment {
    int kind, h;
    int tok0, tok1, toks0, toks1;  // each stream's tile: first token (A: of the packed ones), tokens
    int n0, n1, end0, end1;        // a stream works on [n0, end)
    int split;
    int ptiles;                    // the item's tiles that are the prefix's
    int olen, obase, first;        // own keys; token t sees min(olen, obase + t - first) of them
    int b, slot;
    int flip;                      // split: the stream of the first tile
    int pad[2];
};

__device__ __forceinline__ int tiles_of(const Segment& s, int st) {
    return s.split ? (s.n1 - s.n0 + 1 - (st ^ s.flip)) >> 1 : (st ? s.end1 : s.end0) - s.n0;
}
// keys of tile n that are loaded
__device__ __forceinline__ int keys_of(const SharedArgs& a, const Segment& s, int n) {
    return min(kTileKeys, n < s.ptiles ? a.prefix_len - n * kTileKeys : s.olen - (n - s.ptiles) * kTileKeys);
}

// What the join has to know of a C item that run c is the second to work on.
struct CutRecord { int valid, h, tok0, tok1, toks0, toks1, c0, c1; };

using KeyRing = Ring<kKeyStages>;      // stages 0, 1, 2 of `full` and `empty`
using ValueRing = Ring<kValueStages>;  // stages 3, 4

// Walks the CTA's run of the line (a whole warp, uniformly).
struct Walker {
    const SharedArgs& a;
    const PlanHead& p;
    long long at, end;      // the run, of A's lane or of the others' line
    long long w0;           // where the current item begins
    int zone, b, h, u, n, len, first, ahead, before;  // the item: A (h, u = pair), C (b, h, unit u), B (b, h)
    int lane, run;          // A: the CTA's lane and run; else the run
    long long cost;         // the item's
    bool more;

    __device__ __forceinline__ void load_request() {
        const int4 q = a.req[2 * b], e = a.req[2 * b + 1];
        first = q.x;
        n = q.y;
        len = q.z;
        ahead = e.x;
        before = e.y;
    }
    __device__ __forceinline__ int units() const { return (n + 2 * a.tpt - 1) / (2 * a.tpt); }
    __device__ __forceinline__ int a_rate() const { return p.lanes == 1 && u == p.pairs - 1 && (p.tiles & 1) ? kCostOne : kCostPair; }
    __device__ __forceinline__ void set_cost() {
        if (zone == 0) {
            cost = a_keys(a) * a_rate();
        } else if (zone == 1) {
            const long long base = unit_base(a, ahead);
            cost = kCostLong * (base + min(n, (u + 1) * 2 * a.tpt));
        } else {
            cost = (long long)(len + kItemKeys) * kCostOwn;
        }
    }
    // the item that holds place x of the line
    __device__ void locate(long long x) {
        if (zone == 0) {
            const long long pair = a_keys(a) * kCostPair;
            h = small_quotient(x, p.head_a);
            u = p.lanes > 1 ? lane : min((int)((x - h * p.head_a) / pair), p.pairs - 1);
            w0 = h * p.head_a + (p.lanes > 1 ? 0 : u * pair);
        } else if (x >= p.work_t) {
            more = false;
            return;
        } else if (x < p.work_c) {
            zone = 1;
            b = warp_find(a.c_at, a.B, x);
            load_request();
            const int D = 2 * a.tpt;
            const long long base = unit_base(a, ahead), at_b = a.c_at[b], z = x - at_b;
            const long long per = units_before(base, D, units() - 1) + kCostLong * (base + n);  // a KV head's
            h = small_quotient(z, per);
            const long long rem = z - h * per;
            // units_before(u) <= rem: the quadratic's root (as 2 c / (sqrt(b^2 + 2 D c) + b), which cancels nothing), then exactly
            const float bq = (float)base + 0.5f * D, c = (float)rem / kCostLong;
            u = (int)(2.f * c / (sqrtf(bq * bq + 2.f * D * c) + bq));
            u = min(max(u, 0), units() - 1);
            while (u > 0 && units_before(base, D, u) > rem) --u;
            while (u + 1 < units() && units_before(base, D, u + 1) <= rem) ++u;
            w0 = at_b + h * per + units_before(base, D, u);
        } else {
            zone = 2;
            const long long y = x - p.work_c;
            b = warp_find(a.b_at, a.B, y);
            load_request();
            set_cost();
            h = small_quotient(y - a.b_at[b], cost);
            w0 = p.work_c + a.b_at[b] + h * cost;
        }
        set_cost();
    }
    __device__ void start(int c) {
        zone = c < p.runs_a ? 0 : 1;
        if (zone == 0) {
            lane = c % p.lanes;
            run = c / p.lanes;
            at = a_begin(p, run);
            end = a_begin(p, run + 1);
        } else {
            run = c - p.runs_a;
            at = end = 0;
            if (run < p.runs) {
                at = w_begin(p, run);
                end = min(w_begin(p, run + 1), p.work_t);
            }
        }
        more = at < end;
        if (more) locate(at);
    }
    __device__ void step() {  // to the next item
        const long long w1 = w0 + cost;
        if (w1 >= end) {
            more = false;
            return;
        }
        if (zone == 0) {
            if (p.lanes > 1 || u + 1 == p.pairs) {
                ++h;
                u = p.lanes > 1 ? lane : 0;
            } else {
                ++u;
            }
            w0 = w1;
            set_cost();
            return;
        }
        if (zone == 1 && u + 1 < units()) { ++u; w0 = w1; set_cost(); return; }
        if (zone == 1 && h + 1 < a.Hkv) { ++h; u = 0; w0 = w1; set_cost(); return; }
        if (zone == 2 && h + 1 < a.Hkv) { ++h; w0 = w1; return; }
        locate(w1);
    }
    // The item's tiles in the run; false when none begins there (tile k lies at w0 + 128 k rate).
    __device__ bool segment(Segment& s, CutRecord& cut) {
        const int rate = (zone == 0 ? a_rate() : zone == 1 ? kCostLong : kCostOwn) * kTileKeys;
        auto tiles_from = [&](long long x) {  // ceil(x / rate), x > 0: divisions by constants
            const unsigned long long y = x + rate - 1;
            return (long long)(zone == 1 ? y / (kCostLong * kTileKeys) : zone == 2 ? y / (kCostOwn * kTileKeys)
                               : rate == kCostPair * kTileKeys ? y / (kCostPair * kTileKeys) : y / (kCostOne * kTileKeys));
        };
        s.h = h;
        s.b = b;
        s.obase = s.first = 0;
        int tiles;
        if (zone == 0) {
            s.kind = kPrefixItem;
            s.split = u == p.pairs - 1 && (p.tiles & 1);
            s.tok0 = 2 * u * a.tpt;
            s.tok1 = s.split ? s.tok0 : s.tok0 + a.tpt;
            s.toks0 = min(a.tpt, p.tokens - s.tok0);
            s.toks1 = min(a.tpt, p.tokens - s.tok1);
            s.ptiles = tiles = a.prefix_tiles;
            s.olen = 0;
            s.end0 = s.end1 = tiles;
        } else if (zone == 1) {
            const int left = n - u * 2 * a.tpt;  // tokens from this pair's first on
            s.split = 0;
            s.toks0 = left > a.tpt ? a.tpt : 0;   // (a single tile goes to stream 1)
            s.toks1 = left > a.tpt ? min(left - a.tpt, a.tpt) : left;
            s.tok0 = first + u * 2 * a.tpt;
            s.tok1 = s.tok0 + s.toks0;
            s.ptiles = a.prefix_tiles;
            s.first = first;
            s.obase = ahead + 1;
            s.olen = min(len, max(0, s.obase + s.tok1 + s.toks1 - 1 - first));
            tiles = s.ptiles + (s.olen + kTileKeys - 1) / kTileKeys;
            const int l0 = min(s.olen, max(0, s.obase + s.tok0 + s.toks0 - 1 - first));
            s.end0 = s.toks0 ? s.ptiles + (l0 + kTileKeys - 1) / kTileKeys : 0;
            s.end1 = tiles;
        } else {
            s.kind = kOwnItem;
            s.split = 1;
            s.tok0 = s.tok1 = s.first = first;
            s.toks0 = s.toks1 = n;
            s.ptiles = 0;
            s.obase = ahead + 1;
            s.olen = len;
            s.end0 = s.end1 = tiles = (len + kTileKeys - 1) / kTileKeys;
        }
        s.n0 = at <= w0 ? 0 : (int)tiles_from(at - w0);
        s.n1 = w0 + (long long)tiles * rate <= end ? tiles : (int)min((long long)tiles, tiles_from(end - w0));
        if (tiles == 0) {  // (C only: rows that see nothing are written all the same, where the item begins)
            if (at > w0) return false;
            s.n0 = s.n1 = 0;
        } else if (s.n0 >= s.n1) {
            return false;
        }
        s.end0 = min(max(s.end0, s.n0), s.n1);
        s.end1 = min(max(s.end1, s.n0), s.n1);
        if (zone == 0) {  // (segments of a lane in order raise item or run by one: each slot has one)
            s.slot = ((p.lanes > 1 ? h : h * p.pairs + u) + run) * p.lanes + lane;
        } else if (zone == 2) {
            s.slot = own_slot(a, before, n, h, run);
        } else {
            s.kind = s.n0 == 0 && s.n1 == tiles ? kWholeItem : kCutItem;
            s.slot = 2 * run + (s.n0 == 0);  // the run's first segment, or its last
            if (s.kind == kCutItem && s.n0 > 0) {
                const int c0 = run_of(p.work, p.runs, w0);
                if (c0 == run - 1)
                    cut = CutRecord{1, h, s.tok0, s.tok1, s.toks0, s.toks1, c0, run_of(p.work, p.runs, w0 + (long long)(tiles - 1) * rate)};
            }
        }
        return true;
    }
};

// ---- D: few rows, single warps -----------------------------------------------------------
// NT tiles of 8 rows (tokens x heads).  A warp takes groups of 16 keys one after another, loaded three groups
// ahead (TMA, 128-byte swizzle) into 24 KB of the ring that the CTA's other work no longer needs, on from one
// item to the next.
//   S^T (16 keys x 8 rows) = K (A operand, by ldmatrix) Q^T (B);
//   O^T (128 dims x 8 rows) += V^T (A, by transposing ldmatrix) P^T (B); P^T comes from S^T by two 8 x 8
//     transposes (movmatrix).
// So no lane exchanges logits but for a new maximum, and up to 192 KB an SM are in flight.  Bound by HBM.  (On
// the tensor cores' path a request of 4 rows costs what one of 128 does: 1.4 us a 128-key tile and as much
// an item, and 128 requests over 32K took 171 us instead of 142; with the fragments loaded straight into registers, 8 KB a warp in flight, a group took 1.8 us.)

constexpr int kFewStages = 3;
constexpr uint32_t kFewStageBytes = 16 * 256 * 2, kFewWarpBytes = kFewStages * kFewStageBytes;
static_assert(kFewWarps * kFewWarpBytes <= kOffBars, "the warps' stages fit the ring and the query tiles");

// Walks a warp's share of D, item by item: groups [s, s1) of (request b, KV head h).
struct FewWalk {
    const SharedArgs& a;
    const PlanHead& p;
    long long at, end, w0;
    int b, h, s, s1, first, n, len, ahead;
    bool more;

    __device__ __forceinline__ void find(long long x) {
        b = warp_find(a.d_at, a.B, x - p.work_t);
        const int4 q = a.req[2 * b];
        ahead = a.req[2 * b + 1].x;
        first = q.x;
        n = q.y;
        len = q.z;
        const long long z = x - p.work_t - a.d_at[b], cost = few_cost(len);
        h = small_quotient(z, cost);
        w0 = x - z + h * cost;
    }
    __device__ __forceinline__ void take() {  // the item's groups, or the next item's that has some
        constexpr int rate = 16 * kCostFew;
        while (true) {
            const int groups = (len + 15) >> 4;
            s = at <= w0 ? 0 : (int)((at - w0 + rate - 1) / rate);
            s1 = w0 + (long long)groups * rate <= end ? groups : (int)min((long long)groups, (end - w0 + rate - 1) / rate);
            if (s < s1) return;
            if (!step()) return;
        }
    }
    __device__ __forceinline__ bool step() {
        const long long w1 = w0 + few_cost(len);
        if (w1 >= end) return more = false;
        if (h + 1 < a.Hkv) {
            ++h;
            w0 = w1;
        } else {
            find(w1);
        }
        return true;
    }
    __device__ __forceinline__ void next_item() {
        if (step()) take();
    }
};

template <int NT>
__device__ __forceinline__ void few_rows(const SharedArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, const PlanHead& p,
                                         int run, int warp, uint32_t stages, uint8_t* stages_g, uint32_t bars, bool& failed,
                                         int& bad) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if (run < 0 || run >= p.runs) return;
    const FewShare share = few_share(p, run);
    if (share.hi <= share.lo) return;
    const int sub = warp - (kFewWarps - share.parts);
    if (sub < 0) return;
    FewWalk ask{a, p};  // what is loaded next
    ask.at = few_begin(share, sub);
    ask.end = few_begin(share, sub + 1);
    ask.more = ask.at < ask.end;
    if (!ask.more) return;
    ask.find(ask.at);
    ask.take();
    if (!ask.more) return;
    FewWalk now = ask;  // what is worked on
    Ring<kFewStages> in{0, 0}, out{0, 0};
    uint32_t missing = 0;  // a bit for each stage: its page is not in the pool
    auto id_of = [&] { return a.table[(size_t)ask.b * a.width + ((16 * ask.s) >> a.page_shift)]; };
    int id = id_of();
    auto load = [&] {  // the next group into stage in
        if (!ask.more) return;
        const bool have = id >= 0 && id < a.n_pages;
        if (!have) bad |= HSQ_DEVERR_PAGE;
        missing = (missing & ~(1u << in.stage)) | (have ? 0u : 1u << in.stage);
        if (lane == 0) {
            const uint32_t dst = stages + in.stage * kFewStageBytes, bar = bars + 8 * in.stage;
            // (a page outside the pool is read past the map's extent: zeros, masked below)
            const int y = have ? ((id * a.Hkv + ask.h) << a.page_shift) + ((16 * ask.s) & (a.page_n - 1)) : (a.n_pages * a.Hkv) << a.page_shift;
            mbar_expect_tx(bar, kFewStageBytes);
            tma_2d(dst, &mk, 0, y, bar);
            tma_2d(dst + 2048, &mk, 64, y, bar);
            tma_2d(dst + 4096, &mv, 0, y, bar);
            tma_2d(dst + 6144, &mv, 64, y, bar);
        }
        __syncwarp();
        in.advance();
        if (++ask.s == ask.s1) ask.next_item();
        if (ask.more) id = id_of();
    };
    for (int i = 0; i < kFewStages; ++i) load();
    failed |= (a.fault & HSQ_FAULT_WAIT_FEW) != 0;
    // lane's row of the 8 x 8 matrices that ldmatrix takes: K: keys (lane & 15), chunks 2 kk + (lane >> 4);
    // V: keys (lane & 7) + 8 (lane >> 4), chunks 2 i + ((lane >> 3) & 1)
    const uint32_t k_row = (lane & 15) * 128, k_x = lane & 7, k_c = lane >> 4;
    const uint32_t v_row = ((lane & 7) + 8 * (lane >> 4)) * 128, v_c = (lane >> 3) & 1;
    while (now.more && !failed) {
        const int rows = now.n * a.r;
        uint32_t qf[NT][8][2];
        int lim[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = 8 * nt + g;
            const bool in_use = row < rows;
            const uint32_t* src = reinterpret_cast<const uint32_t*>(
                a.q + ((size_t)(now.first + (in_use ? row / a.r : 0)) * a.Hq + now.h * a.r + (in_use ? row % a.r : 0)) * 128 + 2 * t);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                qf[nt][kk][0] = in_use ? src[8 * kk] : 0u;
                qf[nt][kk][1] = in_use ? src[8 * kk + 4] : 0u;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int rr = 8 * nt + 2 * t + e;
                lim[nt][e] = rr < rows ? min(now.len, now.ahead + rr / a.r + 1) : 0;
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
#pragma unroll 1
        for (int s = now.s; s < now.s1; ++s) {
            const uint32_t kb = stages + out.stage * kFewStageBytes, vb = kb + 4096;
            mbar_wait_fast(bars + 8 * out.stage, out.phase, failed, a.polls);
            const bool gone = (missing >> out.stage) & 1u;
            const int valid = now.len - 16 * s;  // keys of the group that the request has
            if (valid < 16) {  // the rest of the page is stale: weight 0, but it has to be finite
                for (int i = lane; i < (16 - valid) * 16; i += 32)
                    *reinterpret_cast<uint4*>(stages_g + out.stage * kFewStageBytes + 4096 + ((i >> 3) & 1) * 2048 + (valid + (i >> 4)) * 128 +
                                              (i & 7) * 16) = make_uint4(0, 0, 0, 0);
                fence_async_smem();
                __syncwarp();
            }
            float x[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.f;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                uint32_t k[4];
                ldmatrix(k, kb + (kk >> 2) * 2048 + k_row + ((((2 * kk + k_c) & 7) ^ k_x) << 4));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_16816(x[nt], k, qf[nt][kk][0], qf[nt][kk][1]);
            }
            bool look = failed;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {  // key g + 8 (e >> 1), row 2 t + (e & 1)
                    if (gone || 16 * s + g + 8 * (e >> 1) >= lim[nt][e & 1]) x[nt][e] = -INFINITY;
                    look |= x[nt][e] * kLogitScaleLog2 > m[nt][e & 1] * kLogitScaleLog2 + 8.f;  // (the first key raises from -inf)
                }
            if (__any_sync(kFull, look)) {
                failed = __any_sync(kFull, failed);
                if (failed) break;  // (a stage whose copy may still be under way is not asked for again)
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
                float pr[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float off = m[nt][e & 1] == -INFINITY ? 0.f : m[nt][e & 1] * kLogitScaleLog2;
                    pr[e] = ex2_approx(fmaf(x[nt][e], kLogitScaleLog2, -off));
                    l[nt][e & 1] += pr[e];
                }
                pf[nt][0] = transpose_8x8(pack_bf16(pr[0], pr[1]));
                pf[nt][1] = transpose_8x8(pack_bf16(pr[2], pr[3]));
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t v[4];
                ldmatrix_trans(v, vb + (i >> 2) * 2048 + v_row + ((((2 * i + v_c) & 7) ^ k_x) << 4));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_16816(o[nt][i], v, pf[nt][0], pf[nt][1]);
            }
            __syncwarp();  // (every lane has read the stage)
            out.advance();
            load();
        }
        if (failed) break;
        const size_t slot = (size_t)now.b * a.Hkv + now.h + run * kFewWarps + warp;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[nt][e] += __shfl_xor_sync(kFull, l[nt][e], d);
                const int row = 8 * nt + 2 * t + e;
                if (row < rows) {
                    const size_t to = slot * (8 * NT) + row;
                    if (g == 0) a.d_ml[to] = make_float2(m[nt][e], l[nt][e]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        a.d_o[to * 128 + 16 * i + g] = o[nt][i][e];
                        a.d_o[to * 128 + 16 * i + 8 + g] = o[nt][i][e + 2];
                    }
                }
            }
        now.next_item();
    }
    if (failed)  // see the copies in flight (one a stage at most) land before the CTA ends
        for (int i = 0; i < kFewStages; ++i)
            mbar_wait(bars + 8 * i, i < (int)in.stage ? in.phase : in.phase ^ 1, 1 << 12);
}

template <int NT>
__global__ void __launch_bounds__(kTcThreads, 1)
    shared_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                     const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mk16,
                     const __grid_constant__ CUtensorMap mv16, const __grid_constant__ SharedArgs a) {
    extern __shared__ uint8_t tc_raw[];
    const uint32_t raw = smem_addr(tc_raw), base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = tc_raw + (base - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t full = base + kOffBars, empty = full + 8 * kStages, q_full = empty + 8 * kStages, q_empty = q_full + 16;
    const uint32_t s_full = q_empty + 16, p_full = s_full + 16, o_full = p_full + 16, tail = o_full + 16;
    const uint32_t drain = tail + 8, seg_full = drain + 8, seg_empty = seg_full + 8 * kQueue;
    volatile uint32_t* s_mask = reinterpret_cast<volatile uint32_t*>(gbase + kOffMask);
    volatile uint32_t* s_tmem = reinterpret_cast<volatile uint32_t*>(gbase + kOffSeg + kQueue * kSegBytes);
    int bad = 0;

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full + 8 * i, 1);
            mbar_init(q_empty + 8 * i, 1);
            mbar_init(s_full + 8 * i, 1);
            mbar_init(p_full + 8 * i, 4);
            mbar_init(o_full + 8 * i, 1);
        }
        mbar_init(tail, 1);
        mbar_init(drain, 1);
        for (int i = 0; i < kQueue; ++i) {
            mbar_init(seg_full + 8 * i, 1);
            mbar_init(seg_empty + 8 * i, kSegReaders);
        }
        for (int i = 0; i < kFewWarps * kFewStages; ++i) mbar_init(base + kOffFew + 8 * i, 1);
        mbar_init_fence();
    }
    if (warp == 9) {
        tmem_alloc(smem_addr((const void*)s_tmem), 512);
        tmem_relinquish();
    }
    if (warp == 11) {
        // what the first copies will need, on its way while the plan is made (the page ids are not the plan kernel's)
        if (lane < 5) {
            const CUtensorMap* map = lane == 0 ? &mq : lane == 1 ? &mk : lane == 2 ? &mv : lane == 3 ? &mk16 : &mv16;
            asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
        }
        const int ahead = (a.prefix_len + a.page_n - 1) >> a.page_shift;
        const long long lines_p = (ahead + 31) / 32, lines = lines_p + ((long long)a.B * a.width + 31) / 32;
        for (long long i = blockIdx.x * 32 + lane, k = 0; i < lines && k < 4; i += gridDim.x * 32, ++k) {
            const int32_t* at = i < lines_p ? a.prefix + 32 * i : a.table + 32 * (i - lines_p);
            asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    bool failed = false;
    Segment s;
    // A wait that runs out sets its warp's `failed`.  From there on the warp arms no barrier, starts no copy and writes no segment
    // (a stage or a queue place may still be in use), sees what it has in flight to its end and stops; the others' waits then run
    // out in turn.  The results are undefined, the error word says so, and the next call finds everything as it should be.
    auto wait = [&](uint32_t bar, uint32_t parity) { mbar_wait_fast(bar, parity, failed, a.polls); };

    // the next segment of the queue, read by one thread or by a warp
    auto receive = [&](Ring<kQueue>& q, bool release) {
        wait(seg_full + 8 * q.stage, q.phase);
        const int4* src = reinterpret_cast<const int4*>(gbase + kOffSeg + q.stage * kSegBytes);
        int4* dst = reinterpret_cast<int4*>(&s);
        if (release) failed = __any_sync(kFull, failed);  // (a warp stays together)
        if (failed) {
            s.kind = kEnd;
            return false;
        }
#pragma unroll
        for (int i = 0; i < (int)(sizeof(Segment) / 16); ++i) dst[i] = src[i];
        if (release) {
            __syncwarp();
            if (lane == 0) mbar_arrive(seg_empty + 8 * q.stage);
        } else {
            mbar_arrive(seg_empty + 8 * q.stage);
        }
        q.advance();
        return s.kind != kEnd;
    };

    // (128 x 168 x 3 registers at launch: 2 x 128 x 176 + 128 x 152)
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 152;\n");
        if (warp == 8) {
            // ---- the run's segments, and per key tile the K pages, then the V pages (lane i: page i of the tile) ----
            asm volatile("griddepcontrol.wait;" ::: "memory");
            // (only now: so the join kernel, when it is scheduled, finds the plan complete)
            asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
            KeyRing kr{0, 1};
            ValueRing vr{0, 1};
            Ring<kQueue> queue{0, 1};  // (a fresh barrier lets a wait for parity 1 pass: the stages start empty)
            uint32_t step = 0, tail_par = 0;
            bool tail_due = false;
            const uint32_t page_bytes = (uint32_t)a.page_n * 256u, half_page = (uint32_t)a.page_n * 128u;
            const PlanHead plan = *a.head;
            Walker walk{a, plan};
            walk.start(blockIdx.x);
            CutRecord cut{0, 0, 0, 0, 0, 0, 0, 0};
            int flip = 0;
            auto send = [&] {
                wait(seg_empty + 8 * queue.stage, queue.phase);
                failed = __any_sync(kFull, failed);
                if (failed) return;
                if (lane == 0) {
                    *reinterpret_cast<Segment*>(gbase + kOffSeg + queue.stage * kSegBytes) = s;
                    mbar_arrive(seg_full + 8 * queue.stage);
                }
                __syncwarp();
                queue.advance();
            };
            // A key tile to load.  It is looked up (segment, page ids) while the one before it is issued: the ids' way
            // from memory would otherwise stand before every tile's own.
            struct Tile { int n, np, nk, id, h, first; };
            bool fresh = true;  // the walker stands on an item not yet taken
            int n_next = 0;
            auto fetch = [&](Tile& u) {
                u.first = 0;
                if (fresh || n_next >= s.n1) {
                    if (!fresh) walk.step();
                    fresh = false;
                    while (walk.more && !walk.segment(s, cut)) walk.step();
                    if (!walk.more) return false;
                    s.flip = s.split ? flip : 0;  // (items of one tile in turn on both streams)
                    if (s.split) flip ^= (s.n1 - s.n0) & 1;
                    n_next = s.n0;
                    u.first = 1;
                }
                u.n = n_next++;
                u.h = s.h;
                u.np = 0;
                if (u.n >= s.n1) return true;  // (an item without a tile)
                const bool pre = u.n < s.ptiles;
                u.nk = keys_of(a, s, u.n);
                u.np = (u.nk + a.page_n - 1) >> a.page_shift;
                u.id = -1;
                if (lane < u.np)
                    u.id = pre ? a.prefix[(u.n * kTileKeys >> a.page_shift) + lane]
                               : a.table[(size_t)s.b * a.width + ((u.n - s.ptiles) * kTileKeys >> a.page_shift) + lane];
                return true;
            };
            Tile now, then;
            bool have = fetch(now);
            while (have && !failed) {
                if (now.first) send();
                have = fetch(then);
                const int np = now.np, nk = now.nk;
                if (np > 0) {
                    const bool in = lane < np && now.id >= 0 && now.id < a.n_pages;
                    const uint32_t mask = __ballot_sync(kFull, in);
                    if (mask != (1u << np) - 1u) bad |= HSQ_DEVERR_PAGE;
                    // (a page outside the pool is read past the map's extent: zeros, masked in the softmax)
                    const int y = in ? (now.id * a.Hkv + now.h) << a.page_shift : (a.n_pages * a.Hkv) << a.page_shift;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        const uint32_t slot = kv ? kKeyStages + vr.stage : kr.stage;
                        const uint32_t stage = base + slot * kTileBytes, bar = full + 8 * slot;
                        wait(empty + 8 * slot, kv ? vr.phase : kr.phase);
                        if (kv) failed |= (a.fault & HSQ_FAULT_WAIT_LOAD) != 0;
                        failed = __any_sync(kFull, failed);
                        if (failed) break;
                        // The values of a tile that does not end on a multiple of 16 keys: the rows up to there
                        // hold what the page holds; their weights are 0, so they have to be finite.  Cleared
                        // here before the tile is handed over.
                        const bool ragged = kv && (nk & 15);
                        const uint32_t lands = ragged ? tail : bar;
                        if (lane == 0) {
                            if (!kv) s_mask[step & 7] = mask == (1u << np) - 1u ? ~0u : mask;
                            mbar_expect_tx(lands, np * page_bytes);
                        }
                        __syncwarp();
                        if (lane < np) {
                            const void* map = kv ? &mv : &mk;
                            tma_2d(stage + lane * half_page, map, 0, y, lands);
                            tma_2d(stage + lane * half_page + kHalfBytes, map, 64, y, lands);
                        }
                        if (ragged) {
                            wait(tail, tail_par);
                            failed = __any_sync(kFull, failed);
                            if (failed) {
                                tail_due = true;
                                break;
                            }
                            tail_par ^= 1;
                            const int z = (16 - (nk & 15)) * 16;  // 16-byte chunks in both halves
                            for (int i = lane; i < z; i += 32)
                                *reinterpret_cast<uint4*>(gbase + (stage - base) + ((i >> 3) & 1) * kHalfBytes +
                                                          (nk + (i >> 4)) * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
                            fence_async_smem();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(bar);
                        }
                        if (kv) vr.advance(); else kr.advance();
                    }
                    ++step;
                }
                now = then;
            }
            s.kind = kEnd;
            send();
            if (lane == 0 && blockIdx.x >= plan.runs_a) *reinterpret_cast<CutRecord*>(a.cut + 16 * walk.run) = cut;
            if (failed) {  // see the copies in flight land before the CTA ends
                for (int i = 0; i < kStages; ++i) {
                    const bool lap = i < kKeyStages ? i < (int)kr.stage : i - kKeyStages < (int)vr.stage;
                    mbar_wait(full + 8 * i, (i < kKeyStages ? kr.phase : vr.phase) ^ (lap ? 1u : 0u), 1 << 12);
                }
                if (tail_due) mbar_wait(tail, tail_par, 1 << 12);
            }
        } else if (warp == 9 && elect_one()) {
            // ---- MMAs, one thread ----
            // Straight code: per pair of key tiles four waits, each one poll; the tensor pipe takes an MMA every 64
            // cycles and holds only one or two more, so what the thread does in between shows.
            constexpr uint32_t idO = idesc_bf16_f32_bmn(128, 128), idFull = idesc_bf16_f32(128, 128);
            KeyRing kr{0, 0};
            ValueRing vr{0, 0};
            Ring<kQueue> queue{0, 0};
            uint32_t q_par = 0, p_par = 0;  // a bit for each stream
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
                const uint64_t dv = sw128_mn_desc(base + (kKeyStages + vr.stage) * kTileBytes, kHalfBytes);
                wait(p_full + 8 * st, (p_par >> st) & 1);
                p_par ^= 1u << st;
                tc_fence_after();
                mma_bf16_ts(dO, pa, dv, idO, begun);
#pragma unroll
                for (int k = 1; k < 8; ++k) mma_bf16_ts(dO, pa + 8 * k, dv + k * (2048 >> 4), idO, 1);
            };
            auto product_n = [&](int st, int ks16, uint32_t begun) {  // the same of a tile of ks16 groups of 16 keys
                const uint32_t pa = tmem + 128 * st, dO = pa + 256;
                const uint64_t dv = sw128_mn_desc(base + (kKeyStages + vr.stage) * kTileBytes, kHalfBytes);
                wait(p_full + 8 * st, (p_par >> st) & 1);
                p_par ^= 1u << st;
                tc_fence_after();
#pragma unroll 1
                for (int k = 0; k < ks16; ++k) mma_bf16_ts(dO, pa + 8 * k, dv + k * (2048 >> 4), idO, begun | (k > 0));
            };
            auto k_wait = [&] { wait(full + 8 * kr.stage, kr.phase); };
            auto v_wait = [&] { wait(full + 8 * (kKeyStages + vr.stage), vr.phase); };
            auto k_done = [&] { mma_commit(empty + 8 * kr.stage); kr.advance(); };
            auto v_done = [&] { mma_commit(empty + 8 * (kKeyStages + vr.stage)); vr.advance(); };
            auto groups = [&](int n) { return (keys_of(a, s, n) + 15) >> 4; };
            // split segments: the product of a stream's tile waits here until the stream's next S, so that the
            // streams go on from one item to the next without a gap (bit 0: there is one, 1: of the segment's first tile
            // of the stream, 2: of its last, from 8 on: its groups of 16 keys)
            uint32_t due0 = 0, due1 = 0;
            auto settle = [&](int st) {
                const uint32_t due = st ? due1 : due0;
                if (!(due & 1)) return;
                v_wait();
                if ((due >> 8) == 8) product(st, !(due & 2));
                else product_n(st, due >> 8, !(due & 2));
                if (__builtin_expect(failed, 0)) return;
                v_done();
                if (due & 4) mma_commit(o_full + 8 * st);
                if (st) due1 = 0; else due0 = 0;
            };
            int turn = 0;  // the stream of the next tile of a split segment: the one whose product is older
            // (after a wait that ran out no stage is handed back: its copy may still be under way)
            auto work = [&] {
                while (receive(queue, false)) {
                    const int n0 = s.n0, n1 = s.n1, end0 = s.end0;
                    if (s.split) {
#pragma unroll 1
                        for (int n = n0; n < n1; ++n) {
                            const int st = (n - n0 + s.flip) & 1;
                            turn = st ^ 1;
                            settle(st);
                            if (n - n0 < 2) {
                                wait(q_full + 8 * st, (q_par >> st) & 1);
                                q_par ^= 1u << st;
                            }
                            const int g = groups(n);
                            k_wait();
                            if (__builtin_expect(failed, 0)) return;
                            scores(st, idesc_bf16_f32(128, 16 * g));
                            k_done();
                            if (n + 2 >= n1) mma_commit(q_empty + 8 * st);  // (the stream's last S of the segment)
                            const uint32_t due = 1u | (n - n0 < 2 ? 2u : 0u) | (n + 2 >= n1 ? 4u : 0u) | ((uint32_t)g << 8);
                            if (st) due1 = due; else due0 = due;
                        }
                        continue;
                    }
                    settle(turn);
                    settle(turn ^ 1);
                    const bool has0 = tiles_of(s, 0) > 0, has1 = tiles_of(s, 1) > 0;
                    if (has0) { wait(q_full, q_par & 1); q_par ^= 1; }
                    if (has1) { wait(q_full + 8, (q_par >> 1) & 1); q_par ^= 2; }
                    if (n1 > n0) {
                        // the tiles that are not whole: the prefix's last and the item's last
                        const int r1 = (a.prefix_len & 127) ? s.ptiles - 1 : -2, both = min(end0, n1 - 1);
                        k_wait();
                        if (__builtin_expect(failed, 0)) return;
                        if (n0 < end0) scores(0, idesc_bf16_f32(128, 16 * groups(n0)));
                        scores(1, idesc_bf16_f32(128, 16 * groups(n0)));
                        k_done();
                        failed |= (a.fault & HSQ_FAULT_WAIT_MMA) != 0;
                        int n = n0 + 1;
                        while (n < n1) {
                            const int to = r1 >= n ? min(both, r1) : both;
                            if (n - 1 != r1) {
#pragma unroll 1
                                for (; n < to; ++n) {  // P V of tile n - 1 and S of tile n, both whole
                                    k_wait();
                                    v_wait();
                                    product(0, n > n0 + 1);
                                    scores(0, idFull);
                                    product(1, n > n0 + 1);
                                    if (__builtin_expect(failed, 0)) return;
                                    v_done();
                                    scores(1, idFull);
                                    k_done();
                                }
                            }
                            if (n < n1) {  // stream 0 at its end, or a tile that is not whole
                                const uint32_t idS = idesc_bf16_f32(128, 16 * groups(n));
                                const int gp = groups(n - 1);
                                k_wait();
                                v_wait();
                                if (n <= end0) product_n(0, gp, n > n0 + 1);
                                if (n < end0) scores(0, idS);
                                product_n(1, gp, n > n0 + 1);
                                if (__builtin_expect(failed, 0)) return;
                                v_done();
                                scores(1, idS);
                                k_done();
                                ++n;
                            }
                        }
                        if (has0) mma_commit(q_empty);
                        mma_commit(q_empty + 8);
                        const int gp = groups(n1 - 1);
                        v_wait();
                        if (end0 == n1) product_n(0, gp, n1 - 1 > n0);
                        if (has0) mma_commit(o_full);
                        product_n(1, gp, n1 - 1 > n0);
                        if (__builtin_expect(failed, 0)) return;
                        mma_commit(o_full + 8);
                        v_done();
                    }
                }
                if (failed) return;
                settle(turn);
                settle(turn ^ 1);
            };
            work();
            if (failed) {  // what is in flight ends before its operands' and results' memory is given up
                mma_commit(drain);
                mbar_wait(drain, 0, 1 << 12);
            }
        } else if (warp == 10) {
            // ---- queries of the segments' streams ----
            asm volatile("griddepcontrol.wait;" ::: "memory");
            Ring<kQueue> queue{0, 0};
            uint32_t q_par = 3;  // (the buffers start empty)
            const uint32_t q_bytes = (uint32_t)a.tpt * a.r * 256u;
            const PlanHead plan = *a.head;
            while (receive(queue, true)) {
#pragma unroll 1
                for (int st = 0; st < 2; ++st) {
                    if (tiles_of(s, st) <= 0) continue;
                    const uint32_t dst = base + kOffQ + st * kTileBytes, bar = q_full + 8 * st;
                    const int tok = st ? s.tok1 : s.tok0, toks = st ? s.toks1 : s.toks0;
                    wait(q_empty + 8 * st, (q_par >> st) & 1);
                    if (st) failed |= (a.fault & HSQ_FAULT_WAIT_QUERY) != 0;
                    failed = __any_sync(kFull, failed);
                    if (failed) break;
                    q_par ^= 1u << st;
                    if (s.kind != kPrefixItem || plan.dense) {  // tokens side by side
                        const int row = s.kind == kPrefixItem ? plan.base + tok : tok;
                        if (lane == 0) {
                            mbar_expect_tx(bar, q_bytes);
                            tma_3d(dst, &mq, 0, s.h * a.r, row, bar);
                            tma_3d(dst + kHalfBytes, &mq, 64, s.h * a.r, row, bar);
                        }
                        __syncwarp();
                    } else {  // the short requests' tokens among others: row by row, into the swizzled layout
#pragma unroll 1
                        for (int i0 = 0; i0 < toks; i0 += 32) {
                            int row = -1;
                            if (i0 + lane < toks) {
                                const int4 q = a.req[2 * a.of[tok + i0 + lane]];
                                row = q.x + tok + i0 + lane - q.w;
                            }
                            const int chunks = min(32, toks - i0) * a.r * 16;
#pragma unroll 4
                            for (int e0 = 0; e0 < chunks; e0 += 32) {
                                const int e = e0 + lane, hr = e >> 4, c = e & 15, i = min(hr / a.r, 31), jj = hr - (hr / a.r) * a.r;
                                const int from = __shfl_sync(kFull, row, i);
                                if (e < chunks) {
                                    const uint4 v = *reinterpret_cast<const uint4*>(a.q + ((size_t)from * a.Hq + s.h * a.r + jj) * 128 + 8 * c);
                                    const int rt = (i0 + i) * a.r + jj;
                                    *reinterpret_cast<uint4*>(gbase + (dst - base) + (c >> 3) * kHalfBytes + rt * 128 +
                                                              (((c & 7) ^ (rt & 7)) << 4)) = v;
                                }
                            }
                        }
                        fence_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar);
                    }
                }
                if (failed) break;
            }
            if (failed)  // query tiles in flight land before the CTA ends
                for (int st = 0; st < 2; ++st) mbar_wait(q_full + 8 * st, (q_par >> st) & 1, 1 << 12);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 176;\n");
        // ---- softmax: thread = row of its stream's tile ----
        const int st = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t tS = tmem + lanes + 128 * st, tO = tmem + lanes + 256 + 128 * st;
        uint32_t s_par = 0, o_par = 0;
        Ring<kQueue> queue{0, 0};
        int step0 = 0;
        const int row_token = row / a.r;
        asm volatile("griddepcontrol.wait;" ::: "memory");
        const PlanHead plan = *a.head;
        // (a run of D alone does not wait for the queue)
        const int other = (int)blockIdx.x - plan.runs_a;
        const bool tiles = other < 0 || (other < plan.runs && w_begin(plan, other) < plan.work_t);
        while (tiles && receive(queue, true)) {
            const int toks = st ? s.toks1 : s.toks0, tok = st ? s.tok1 : s.tok0, stop = st ? s.end1 : s.end0;
            const bool live = row_token < toks;
            const bool idle = 32 * (warp & 3) >= toks * a.r;  // (warp-uniform) no row of this warp in use
            const int own_min = min(s.olen, s.obase + tok - s.first);             // own keys that the tile's first row sees
            const int own_lim = min(s.olen, s.obase + tok - s.first + row_token); // and this row
            float m = -INFINITY, l = 0.f;
#pragma unroll 1
            for (int n = s.n0 + (s.split ? st ^ s.flip : 0); n < stop; n += s.split ? 2 : 1) {
                wait(s_full + 8 * st, s_par);
                s_par ^= 1;
                if (!idle) {
                    // The running maximum need not be one: any m that keeps the sums in range gives the same
                    // result, p and l being floating point.  So the row's maximum is looked for in its first tile and
                    // where the tile's sum shows that the logits have outgrown m by far; every other tile goes without
                    // (a third of the softmax's time).
                    tc_fence_after();
                    const int begin = (n < s.ptiles ? n : n - s.ptiles) * kTileKeys;
                    const uint32_t mask = s_mask[(step0 + n - s.n0) & 7];
                    if (begin + kTileKeys > (n < s.ptiles ? a.prefix_len : own_min) || mask != ~0u) {
                        // keys past the row's limit or of no page: hidden in S itself, so that the code below (and the
                        // instruction cache) knows whole tiles only
                        const int lim = !live ? 0 : (n < s.ptiles ? a.prefix_len : own_lim) - begin;
#pragma unroll 1
                        for (int c0 = 0; c0 < 128; c0 += 32) {
                            float x[32];
                            tmem_ld32(tS + c0, x);
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (c0 + c >= lim || !((mask >> ((c0 + c) >> a.page_shift)) & 1u)) x[c] = -INFINITY;
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
                wait(o_full + 8 * st, o_par);
                o_par ^= 1;
            }
            failed |= (a.fault & HSQ_FAULT_WAIT_SOFTMAX) != 0;
            failed = __any_sync(kFull, failed);
            if (failed) break;
            tc_fence_after();
            if (s.kind == kWholeItem) {  // the result
                const float inv = l == 0.f ? 0.f : 1.0f / l;  // (a sum that is not a number shows in the result)
                const size_t to = (size_t)(tok + row_token) * a.Hq + s.h * a.r + (row - row_token * a.r);
                if (live && a.lse) a.lse[to] = l == 0.f ? -INFINITY : m * kRsqrtD + logf(l);
                if (!idle) {
#pragma unroll 1
                    for (int c0 = 0; c0 < 128; c0 += 32) {
                        float o[32];
                        if (any) tmem_ld32(tO + c0, o);
                        if (live) {
                            uint4* dst = reinterpret_cast<uint4*>(a.out + to * 128 + c0);
#pragma unroll
                            for (int c = 0; c < 32; c += 8)
                                dst[c >> 3] = l == 0.f ? make_uint4(0, 0, 0, 0)
                                                       : make_uint4(pack_bf16(o[c] * inv, o[c + 1] * inv), pack_bf16(o[c + 2] * inv, o[c + 3] * inv),
                                                                    pack_bf16(o[c + 4] * inv, o[c + 5] * inv), pack_bf16(o[c + 6] * inv, o[c + 7] * inv));
                        }
                    }
                }
            } else if (!idle) {  // a part: dims apart, rows side by side, so that a warp writes whole lines
                const int pitch = s.kind == kOwnItem ? toks * a.r : kTileRows;
                const size_t at = (size_t)s.slot * (s.kind == kOwnItem ? 2 : 2 * kTileRows) + st * pitch;  // rows before it
                float* o_to = (s.kind == kPrefixItem ? a.a_o : s.kind == kOwnItem ? a.b_o : a.c_o) + at * 128 + row;
                float2* ml_to = (s.kind == kPrefixItem ? a.a_ml : s.kind == kOwnItem ? a.b_ml : a.c_ml) + at + row;
                if (live) *ml_to = make_float2(m, l);
                if (any) {
#pragma unroll 1
                    for (int c0 = 0; c0 < 128; c0 += 32) {
                        float o[32];
                        tmem_ld32(tO + c0, o);
                        if (live) {
#pragma unroll
                            for (int c = 0; c < 32; ++c) o_to[(size_t)(c0 + c) * pitch] = o[c];
                        }
                    }
                }
            }
            tc_fence_before();  // (O has been read: the next segment's first P releases it)
            step0 += s.n1 - s.n0;
        }
        // D: every stream's work of this CTA is done, its memory free (where no wait ran out)
        failed = named_bar_or(1, 256, failed);
        if (!failed)
            few_rows<NT>(a, mk16, mv16, plan, (int)blockIdx.x - plan.runs_a, warp, base + warp * kFewWarpBytes, gbase + warp * kFewWarpBytes,
                         base + kOffFew + 8 * kFewStages * warp, failed, bad);
    }
    if (failed) bad |= HSQ_DEVERR_WAIT;
    if (bad) atomicOr(a.err, bad);
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------------------
// Join.  A CTA takes 32 dims of 32 rows of a tile of the short requests' tokens (parts of A, and of B or D), or of
// the 128 rows of a tile of a C item that a cut divides.  Lane = row; the warps deal the parts among them (for a
// cut item, of few parts, the rows too), each with several parts on their way by asynchronous copies, so that what a
// CTA waits for is one or two ways from L2 (one part at a time in registers: 16 requests over 8K 38.5 us instead of 36.9, verification of 32 x 3
// rows 48.8 instead of 48.0).  A's, B's and C's parts are read in whole lines.  Bound by latency: 5 to 10 us of a call.
// (Joined by the CTA in which the item begins, where the other part is there by then: four prompts 384 us instead of
// 357, the softmax's registers spilt.)
// ---------------------------------------------------------------------------------------

constexpr int kJoinDims = 16;  // of a warp; two warps a group
// A warp's part in flight: 16 dims of 32 rows, 2 KB (A, C: by dims, 128 bytes each; B, D: by rows, 64 bytes each, the
// 16-byte chunks exchanged so that the lanes' reads meet no bank twice), and the rows' (m, l).
constexpr int kJoinStage = 32 * kJoinDims * 4 + 32 * 8;
template <int G> constexpr int kJoinStages = G == 8 ? 5 : 3;
template <int G> constexpr int kJoinSmem = 2 * G * kJoinStages<G> * kJoinStage;

template <int N> __device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
    if constexpr (N == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(dst), "l"(src), "n"(N) : "memory");
}

// G groups of warps: 8 where all CTAs are resident together, one an SM; 4, four CTAs an SM, where they are not (us with
// G = 8 and 4: 4 requests over 1K 18.3 and 20.7, 16 over 8K 37 and 41; 61 over 5K 51 and 45, 128 over 32K 119 and 107).
template <int G>
__global__ void __launch_bounds__(64 * G, G == 8 ? 1 : 4) shared_join_kernel(const __grid_constant__ SharedArgs a, int short_ctas) {
    constexpr int S = kJoinStages<G>;
    extern __shared__ __align__(16) uint8_t join_sm[];
    // (over the stages, when they have been read)
    struct Reduce { float x[G][32][33]; float2 ml[G][32]; long long to[4][32]; float inv[4][32]; };
    static_assert(sizeof(Reduce) <= kJoinSmem<G>, "the reduction fits the stages");
    Reduce& sm = *reinterpret_cast<Reduce*>(join_sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int group = warp >> 1, quarter = blockIdx.x & 3, cta = blockIdx.x >> 2;
    const int d_cta = 32 * quarter, d_warp = 16 * (warp & 1), d0 = d_cta + d_warp;
    // row groups of 32 that the CTA has, and which this group of warps takes; of its parts it takes k0, k0 + dk, ...
    const bool brief = cta < short_ctas;
    const int row_groups = brief ? 1 : 4, mine = group % row_groups, k0 = group / row_groups, dk = G / row_groups;
    // the row's parts: n0 at o0 / ml0 (128 rows a slot), n1 at o1 / ml1, step part rows apart
    const float *o0 = nullptr, *o1 = nullptr;
    const float2 *ml0 = nullptr, *ml1 = nullptr;
    int n0 = 0, n1 = 0, apart0 = 1, step1 = 1, pitch1 = kTileRows;
    bool both = false, by_row = false;  // both: the first parts are two streams'; by_row: a row's dims lie side by side in o1
    bool live;
    size_t to = 0;
    if (brief) {  // (of the plan alone, complete before this kernel begins: looked up while the main kernel ends)
        const int h = cta % a.Hkv, grp = cta / a.Hkv, tile = grp >> 2, row = (grp & 3) * 32 + lane;
        const int at = tile * a.tpt + row / a.r;
        const bool room = row < a.tpt * a.r;
        const int b_any = __ldcg(a.of + min(at, a.tokens_cap - 1));  // (before it is known whether the row is in use)
        const PlanHead p = *a.head;
        live = room && at < p.tokens;
        if (!__any_sync(kFull, live)) {  // (the same for every warp)
            asm volatile("griddepcontrol.wait;" ::: "memory");
            return;
        }
        const int b = live ? b_any : 0;
        const int4 q = __ldcg(a.req + 2 * b);
        const int before = __ldcg(a.req + 2 * b + 1).y;
        const bool few = q.y * a.r <= kFewRows;
        const long long at1 = few ? p.work_t + __ldcg(a.d_at + b) : p.work_c + __ldcg(a.b_at + b);
        const int orow = live ? row - (q.w - tile * a.tpt) * a.r : 0;  // row among the request's
        if (p.lane_a > 0) {
            const int pair = tile >> 1, stream = tile & 1;
            both = tile == p.tiles - 1 && !stream;  // (a pair of one tile has its key tiles dealt to both streams)
            const long long keys = a_keys(a);
            const int rate = (both && p.lanes == 1 ? kCostOne : kCostPair) * kTileKeys;
            const long long w0 = h * p.head_a + (p.lanes > 1 ? 0 : pair * keys * kCostPair);
            const int c0 = run_of(p.lane_a, p.cuts_a, w0), c1 = run_of(p.lane_a, p.cuts_a, w0 + (long long)(a.prefix_tiles - 1) * rate);
            const size_t slot = (((p.lanes > 1 ? h : (size_t)h * p.pairs + pair) + c0) * p.lanes + (p.lanes > 1 ? pair : 0)) * 2 + stream;
            o0 = a.a_o + slot * 128 * kTileRows + row;
            ml0 = a.a_ml + slot * kTileRows + row;
            apart0 = 2 * p.lanes;
            n0 = (c1 - c0 + 1) * (both ? 2 : 1);
        }
        if (live && q.z > 0 && few) {
            const long long w0 = at1 + h * few_cost(q.z);
            const int v0 = few_warp_of(p, w0), v1 = few_warp_of(p, w0 + (long long)(((q.z + 15) >> 4) - 1) * 16 * kCostFew);
            const size_t slot = (size_t)b * a.Hkv + h + v0;
            by_row = true;
            pitch1 = a.few_rows;
            o1 = a.d_o + (slot * a.few_rows + orow) * 128;
            ml1 = a.d_ml + slot * a.few_rows + orow;
            n1 = v1 - v0 + 1;
        } else if (live && q.z > 0) {
            const long long w0 = at1 + h * ((long long)(q.z + kItemKeys) * kCostOwn);
            const int tiles = (q.z + kTileKeys - 1) / kTileKeys;
            const int c0 = run_of(p.work, p.runs, w0), c1 = run_of(p.work, p.runs, w0 + (long long)(tiles - 1) * kCostOwn * kTileKeys);
            const size_t slot = (size_t)own_slot(a, before, q.y, h, c0) * 2;
            pitch1 = q.y * a.r;
            o1 = a.b_o + slot * 128 + orow;
            ml1 = a.b_ml + slot + orow;
            n1 = 2 * (c1 - c0 + 1);
        }
        to = (size_t)(q.x + orow / a.r) * a.Hq + h * a.r + orow % a.r;
        asm volatile("griddepcontrol.wait;" ::: "memory");
    } else {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        const int e = cta - short_ctas, c = 1 + (e >> 1), st = e & 1, row = mine * 32 + lane;
        if (c >= a.head->runs) return;
        const CutRecord cut = *reinterpret_cast<const CutRecord*>(a.cut + 16 * c);
        if (!cut.valid) return;
        live = row < (st ? cut.toks1 : cut.toks0) * a.r;
        // slot 2 c0 + 1, then 2 c0 + 2, 2 c0 + 4, ...
        const size_t s0 = (2 * (size_t)cut.c0 + 1) * 2 + st, s1 = (2 * (size_t)cut.c0 + 2) * 2 + st;
        o0 = a.c_o + s0 * 128 * kTileRows + row;
        ml0 = a.c_ml + s0 * kTileRows + row;
        n0 = 1;
        o1 = a.c_o + s1 * 128 * kTileRows + row;
        ml1 = a.c_ml + s1 * kTileRows + row;
        step1 = 4;
        n1 = cut.c1 - cut.c0;
        to = (size_t)((st ? cut.tok1 : cut.tok0) + row / a.r) * a.Hq + cut.h * a.r + row % a.r;
    }
    if (!live) n1 = 0;
    const int n = __reduce_max_sync(kFull, n0 + n1);  // (n0 is one for the tile)
    const uint64_t o1_at = reinterpret_cast<uint64_t>(o1);
    uint8_t* mine_g = join_sm + warp * S * kJoinStage;
    const uint32_t mine_s = smem_addr(mine_g);
    auto swizzled = [](int row, int chunk) { return row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4); };
    auto fetch = [&](int k, int stage) {  // part k on its way
        const uint32_t dst = mine_s + stage * kJoinStage;
        const bool first = k < n0;
        const size_t at = !first ? (size_t)(k - n0) * step1 : both ? (size_t)(k >> 1) * apart0 + (k & 1) : (size_t)k * apart0;
        if (first || !brief) {
            const float* src = (first ? o0 : o1) - lane + (at * 128 + d0) * kTileRows;  // (of row 0 of the 32)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int dim = 4 * i + (lane >> 3), rows4 = 4 * (lane & 7);
                copy_async<16>(dst + (dim * 32 + rows4) * 4, src + dim * kTileRows + rows4);
            }
            copy_async<8>(dst + 2048 + 8 * lane, (first ? ml0 : ml1) + at * kTileRows);
            return;
        }
        const int rows_n = by_row ? n1 : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 8 * i + (lane >> 2), chunk = lane & 3;
            const float* src = reinterpret_cast<const float*>(__shfl_sync(kFull, o1_at, row)) + at * a.few_rows * 128 + d0 + 4 * chunk;
            if (k - n0 < __shfl_sync(kFull, rows_n, row)) copy_async<16>(dst + swizzled(row, chunk), src);
        }
        if (k - n0 >= n1) return;
        const size_t rows = by_row ? at * pitch1 : (at & ~(size_t)1) * a.own_rows + (at & 1) * pitch1;  // before part `at` of B or D
        if (!by_row) {
            const float* src = o1 + rows * 128 + (size_t)d0 * pitch1;
#pragma unroll
            for (int d = 0; d < kJoinDims; ++d) copy_async<4>(dst + swizzled(lane, d >> 2) + 4 * (d & 3), src + d * pitch1);
        }
        copy_async<8>(dst + 2048 + 8 * lane, ml1 + rows);
    };
    float M = -INFINITY, L = 0.f, x[kJoinDims];
#pragma unroll
    for (int d = 0; d < kJoinDims; ++d) x[d] = 0.f;
    auto add = [&](int k, int stage) {
        const uint8_t* src = mine_g + stage * kJoinStage;
        const bool first = k < n0;
        if (!live || (!first && k - n0 >= n1)) return;
        const float2 ml = reinterpret_cast<const float2*>(src + 2048)[lane];
        if (ml.y == 0.f) return;  // (a part without a key has no o)
        const float top = fmaxf(M, ml.x);
        const float was = M == -INFINITY ? 0.f : ex2_approx((M - top) * kLogitScaleLog2), w = ex2_approx((ml.x - top) * kLogitScaleLog2);
        M = top;
        L = fmaf(ml.y, w, L * was);
        if (first || !brief) {
#pragma unroll
            for (int d = 0; d < kJoinDims; ++d) x[d] = fmaf(reinterpret_cast<const float*>(src)[32 * d + lane], w, x[d] * was);
        } else {
#pragma unroll
            for (int c = 0; c < kJoinDims / 4; ++c) {
                const float4 y = *reinterpret_cast<const float4*>(src + swizzled(lane, c));
                x[4 * c] = fmaf(y.x, w, x[4 * c] * was);
                x[4 * c + 1] = fmaf(y.y, w, x[4 * c + 1] * was);
                x[4 * c + 2] = fmaf(y.z, w, x[4 * c + 2] * was);
                x[4 * c + 3] = fmaf(y.w, w, x[4 * c + 3] * was);
            }
        }
    };
    // S parts in flight a warp: their way from L2 is what the join waits for
#pragma unroll
    for (int i = 0; i < S; ++i) {
        if (k0 + i * dk < n) fetch(k0 + i * dk, i);
        asm volatile("cp.async.commit_group;\n" ::: "memory");
    }
    for (int k = k0, stage = 0; k < n; k += dk) {
        asm volatile("cp.async.wait_group %0;\n" ::"n"(S - 1) : "memory");
        __syncwarp();
        add(k, stage);
        __syncwarp();
        if (k + S * dk < n) fetch(k + S * dk, stage);
        asm volatile("cp.async.commit_group;\n" ::: "memory");
        if (++stage == S) stage = 0;
    }
    __syncthreads();
    if (d_warp == 0) sm.ml[group][lane] = make_float2(M, L);
    __syncthreads();
    float top = -INFINITY, sum = 0.f;
    for (int g = mine; g < G; g += row_groups) top = fmaxf(top, sm.ml[g][lane].x);
    for (int g = mine; g < G; g += row_groups) {
        const float2 ml = sm.ml[g][lane];
        if (ml.y != 0.f) sum = fmaf(ml.y, ex2_approx((ml.x - top) * kLogitScaleLog2), sum);
    }
    const float w = M == -INFINITY ? 0.f : ex2_approx((M - top) * kLogitScaleLog2);
#pragma unroll
    for (int d = 0; d < kJoinDims; ++d) sm.x[group][lane][d_warp + d] = x[d] * w;
    if (k0 == 0 && d_warp == 0) {
        sm.to[mine][lane] = live ? (long long)to : -1;
        sm.inv[mine][lane] = sum == 0.f ? 0.f : 1.0f / sum;
        if (live && a.lse && quarter == 0) a.lse[to] = sum == 0.f ? -INFINITY : top * kRsqrtD + logf(sum);
    }
    __syncthreads();
    const int d = 2 * (tid & 15);
    for (int e = tid >> 4; e < 32 * row_groups; e += 4 * G) {
        const int i = e >> 5, row = e & 31;
        float y0 = 0.f, y1 = 0.f;
        for (int g = i; g < G; g += row_groups) {
            y0 += sm.x[g][row][d];
            y1 += sm.x[g][row][d + 1];
        }
        const float inv = sm.inv[i][row];
        if (sm.to[i][row] >= 0)
            *reinterpret_cast<uint32_t*>(a.out + sm.to[i][row] * 128 + d_cta + d) = pack_bf16(y0 * inv, y1 * inv);
    }
}

// ---- host side --------------------------------------------------------------------------

// The workspace's pieces and their offsets.
struct Layout { size_t head, req, of, c_at, b_at, d_at, cut, a_o, a_ml, b_o, b_ml, c_o, c_ml, d_o, d_ml, bytes; int runs, own_rows, few_rows, tokens; };

Layout layout_of(const hsq_ctx* ctx, int rows, int B, int prefix_len, int max_new) {
    Layout x{};
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t here = at;
        at += (n + 255) / 256 * 256;
        return here;
    };
    const size_t Hkv = ctx->cfg.n_kv_heads, r = ctx->r, tpt = kTileRows / r;
    x.runs = ctx->num_sms;
    x.own_rows = (int)(std::min<size_t>(max_new, tpt) * r);
    x.head = take(sizeof(PlanHead));
    x.req = take((size_t)B * 32);
    x.c_at = take((size_t)(B + 1) * 8);
    x.b_at = take((size_t)(B + 1) * 8);
    x.d_at = take((size_t)(B + 1) * 8);
    x.few_rows = (size_t)max_new * r <= 8 ? 8 : 16;
    x.cut = take((size_t)x.runs * 64);
    const size_t tokens = std::min<size_t>(rows, (size_t)B * tpt), tiles = (tokens + tpt - 1) / tpt;
    x.tokens = (int)tokens;
    x.of = take(tokens * 4);
    const size_t a = prefix_len > 0 ? Hkv * ((tiles + 1) / 2) + x.runs : 0;
    const size_t b_items = std::min<size_t>((size_t)rows * r, (size_t)B * x.own_rows);  // rows of all B requests
    const size_t b = (size_t)max_new * r > kFewRows ? Hkv * b_items + (size_t)x.runs * x.own_rows : 0;  // rows of their parts
    const size_t c = (size_t)max_new > tpt ? 2 * (size_t)x.runs : 0;
    x.a_o = take(a * 2 * 128 * kTileRows * 4);
    x.a_ml = take(a * 2 * kTileRows * 8);
    x.b_o = take(b * 2 * 128 * 4);
    x.b_ml = take(b * 2 * 8);
    x.c_o = take(c * 2 * 128 * kTileRows * 4);
    x.c_ml = take(c * 2 * kTileRows * 8);
    const size_t d = (size_t)B * Hkv + (size_t)kFewWarps * x.runs;
    x.d_o = take(d * x.few_rows * 128 * 4);
    x.d_ml = take(d * x.few_rows * 8);
    x.bytes = at;
    return x;
}

}  // namespace

extern "C" {

hsq_status hsq_shared_attn_workspace_size(const hsq_ctx* ctx, int rows, int B, int prefix_len, int max_new,
                                          size_t* bytes) {
    if (!ctx || !bytes) return hsq::fail(nullptr, HSQ_ERR_INVALID, "ctx or bytes is NULL");
    if (rows < 1 || B < 1 || B > HSQ_MAX_REQUESTS || prefix_len < 0 || prefix_len > (1 << 30) || max_new < 1)
        return hsq::fail(nullptr, HSQ_ERR_INVALID,
                         "rows, B (up to HSQ_MAX_REQUESTS) and max_new must be positive, prefix_len in [0, 2^30]");
    *bytes = layout_of(ctx, rows, B, prefix_len, max_new).bytes;
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
    if (rows < 1 || width < 1 || max_new < 1 || prefix_len < 0 || prefix_len > (1 << 30))
        return hsq::fail(ctx, HSQ_ERR_INVALID, "rows, width and max_new must be positive, prefix_len in [0, 2^30]");
    if ((long long)width * pages->page_n > (1 << 30)) return hsq::fail(ctx, HSQ_ERR_INVALID, "width * page_n above 2^30");
    if (prefix_len > 0 && !prefix) return hsq::fail(ctx, HSQ_ERR_INVALID, "prefix is NULL with prefix_len > 0");
    if (((uintptr_t)q | (uintptr_t)out) & 15u)
        return hsq::fail(ctx, HSQ_ERR_INVALID, "q and out must be 16-byte aligned");
    if ((uintptr_t)workspace & 255u) return hsq::fail(ctx, HSQ_ERR_INVALID, "workspace must be 256-byte aligned");
    const Layout x = layout_of(ctx, rows, B, prefix_len, max_new);
    if (workspace_bytes < x.bytes)
        return hsq::fail(ctx, HSQ_ERR_INVALID, "workspace smaller than hsq_shared_attn_workspace_size");
    const size_t q_bytes = (size_t)rows * ctx->cfg.n_q_heads * 256, pool = (size_t)pages->n_pages * ctx->cfg.n_kv_heads * pages->page_n * 256;
    const hsq::Span ins[] = {{q, q_bytes}, {q_start, 4 * ((size_t)B + 1)}, {lens, 4 * (size_t)B}, {table, 4 * (size_t)B * width},
                             {prefix_len > 0 ? prefix : nullptr, 4 * (size_t)((prefix_len + pages->page_n - 1) / pages->page_n)},
                             {pages->k, pool}, {pages->v, pool}};
    const hsq::Span outs[] = {{out, q_bytes}, {lse_opt, (size_t)rows * ctx->cfg.n_q_heads * 4}, {workspace, x.bytes}};
    if (hsq::outputs_overlap(ins, outs))
        return hsq::fail(ctx, HSQ_ERR_INVALID, "an output or the workspace of hsq_shared_attn overlaps another argument");
    if ((st = hsq::check_device(ctx)) != HSQ_OK) return st;
    const int r = ctx->r, Hkv = ctx->cfg.n_kv_heads, tpt = kTileRows / r;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    SharedArgs a{};
    a.q = static_cast<const uint16_t*>(q);
    a.q_start = q_start; a.lens = lens; a.table = table; a.prefix = prefix;
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse_opt;
    a.rows = rows; a.B = B; a.width = width; a.prefix_len = prefix_len; a.max_new = max_new;
    a.prefix_tiles = (prefix_len + kTileKeys - 1) / kTileKeys;
    a.n_pages = pages->n_pages; a.page_n = pages->page_n;
    a.page_shift = pages->page_n == 16 ? 4 : pages->page_n == 32 ? 5 : pages->page_n == 64 ? 6 : 7;
    a.Hq = ctx->cfg.n_q_heads; a.Hkv = Hkv; a.r = r; a.tpt = tpt; a.runs = x.runs; a.own_rows = x.own_rows;
    a.head = reinterpret_cast<PlanHead*>(ws + x.head);
    a.req = reinterpret_cast<int4*>(ws + x.req);
    a.c_at = reinterpret_cast<long long*>(ws + x.c_at);
    a.b_at = reinterpret_cast<long long*>(ws + x.b_at);
    a.d_at = reinterpret_cast<long long*>(ws + x.d_at);
    a.cut = reinterpret_cast<int*>(ws + x.cut);
    a.of = reinterpret_cast<int*>(ws + x.of);
    a.tokens_cap = x.tokens;
    a.a_o = reinterpret_cast<float*>(ws + x.a_o); a.a_ml = reinterpret_cast<float2*>(ws + x.a_ml);
    a.b_o = reinterpret_cast<float*>(ws + x.b_o); a.b_ml = reinterpret_cast<float2*>(ws + x.b_ml);
    a.c_o = reinterpret_cast<float*>(ws + x.c_o); a.c_ml = reinterpret_cast<float2*>(ws + x.c_ml);
    a.d_o = reinterpret_cast<float*>(ws + x.d_o); a.d_ml = reinterpret_cast<float2*>(ws + x.d_ml);
    a.few_rows = x.few_rows;
    a.fault = (int)hsq::fault_mask() & (HSQ_FAULT_WAIT_LOAD | HSQ_FAULT_WAIT_MMA | HSQ_FAULT_WAIT_QUERY | HSQ_FAULT_WAIT_SOFTMAX | HSQ_FAULT_WAIT_FEW);
    a.polls = a.fault ? 1 << 8 : 1 << 18;  // (a poll that finds nothing takes 4 us: 1 ms, or a second, where no wait in use takes 10 ms)
    a.err = ctx->d_err;
    CUtensorMap mq, mk, mv, mk16, mv16;
    if (!encode_fn()) return hsq::fail(ctx, HSQ_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    const uint64_t n = (uint64_t)pages->n_pages * Hkv * pages->page_n;
    if (!encode_q(&mq, q, rows, a.Hq, r, tpt) || !encode_rows(&mk, pages->k, n, pages->page_n) ||
        !encode_rows(&mv, pages->v, n, pages->page_n) || !encode_rows(&mk16, pages->k, n, 16) ||
        !encode_rows(&mv16, pages->v, n, 16))
        return hsq::fail(ctx, HSQ_ERR_CUDA, "cuTensorMapEncodeTiled refused a tensor map");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int tiles = (x.tokens + tpt - 1) / tpt;
    int short_ctas = 4 * tiles * Hkv;
    const int cut_ctas = max_new > tpt ? 2 * (x.runs - 1) : 0;
    void* plan_args[] = {&a};
    void* tc_args[] = {&mq, &mk, &mv, &mk16, &mv16, &a};
    void* join_args[] = {&a, &short_ctas};
    const void* fn = x.few_rows == 8 ? (const void*)shared_tc_kernel<1> : (const void*)shared_tc_kernel<2>;
    cudaError_t e = hsq::raise_smem_limit(fn, ctx->device, kTcSmem);
    if (e != cudaSuccess) return hsq::cuda_fail(ctx, e, "cudaFuncSetAttribute(shared_attn)");
    if ((e = launch((const void*)shared_plan_kernel, 1, kPlanThreads, 0, s, false, plan_args)) != cudaSuccess)
        return hsq::cuda_fail(ctx, e, "shared_attn plan");
    if ((e = launch(fn, x.runs, kTcThreads, kTcSmem, s, true, tc_args)) != cudaSuccess)
        return hsq::cuda_fail(ctx, e, "shared_attn");
    const int join_ctas = 4 * (short_ctas + cut_ctas);
    const bool wide = join_ctas <= ctx->num_sms;
    fn = wide ? (const void*)shared_join_kernel<8> : (const void*)shared_join_kernel<4>;
    const size_t smem = wide ? kJoinSmem<8> : kJoinSmem<4>;
    if ((e = hsq::raise_smem_limit(fn, ctx->device, smem)) == cudaSuccess)
        e = launch(fn, join_ctas, wide ? 512 : 256, smem, s, true, join_args);
    if (e != cudaSuccess) return hsq::cuda_fail(ctx, e, "shared_attn join");
    return HSQ_OK;
}

}  // extern "C"
