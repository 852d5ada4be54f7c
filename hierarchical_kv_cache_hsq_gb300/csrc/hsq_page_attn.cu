// Attention over selected pages (hsq_page_attn).
//
// For row i and query head jq of KV head h: one softmax, scale 1/sqrt(128), over the tokens (up to the row's last) of the
// logical pages in sel[i][h].  Parts of a softmax over disjoint sets of keys join as
//     out = sum_p exp(m_p - M) o_p / sum_p exp(m_p - M) l_p,   M = max_p m_p,
// with m, l, o a reference exponent, the sum of exp(x - m) and the sum of exp(x - m) v of a part, all fp32.  The weights
// exp(x - m) alone are rounded to bf16, by up to 2^-8 of each, for their product with the values: the matrix instructions take both
// in one type.  (The error against 64 bits is 0.0023 of the result, in root mean square; with weights in fp32 it would be the 0.0017
// of the result's own rounding to bf16.)
#include <cooperative_groups.h>

#include <algorithm>

#include "hsq_ctx.h"
#include "hsq_paged.cuh"

namespace {

using namespace hsq_paged;
using namespace hsq_tc;
namespace cg = cooperative_groups;

struct PageAttnArgs {
    const uint16_t* q;
    const int32_t *q_start, *lens, *table, *prefix, *sel;
    uint16_t* out; float* lse;
    int rows, B, width, prefix_len, prefix_pages, max_new, n_pages, page_n, page_shift, Hq, Hkv, r, top;
    int polls;   // of a wait, before it has run out
    int fault;   // HSQ_FAULT_WAIT_*: the roles that give up at a certain wait (0 but in tests)
    int* err;
    // requests of more than `few` tokens go by tiles (few >= max_new: there are none, and nothing below is there)
    int few, tpt, words, cap, runs, units_cap, rows_cap;
    struct TileHead* head;
    int4* req;        // [B] first row, rows, own tokens held, own tokens before the first row
    int2* unit;       // [units] long requests' pairs of row tiles: request, pair
    int* short_row;   // the other requests' rows
    int4* count;      // [items] pages of both tiles, of the first alone, of the second alone; cost
    int2* ent;        // [items][3][cap] page id, logical page
    uint32_t* mask;   // [items][3][cap][2][words] the tiles' tokens that take the page
    float* part_o;    // [2 runs][2][128 dims][128 rows]
    float2* part_ml;  // [2 runs][2][128 rows] maximum of q.k, unscaled; sum
    float2* pair_ml;  // [runs][128]
    int4* cut;        // [runs][3] see CutRecord
};

struct TileHead {
    int units, shorts;
};

// The entries of a row's selection that count, by a whole warp: those below the row's number of pages c and above every entry before
// them; others that are not -1 are flagged.
template <class F>
__device__ __forceinline__ void for_selected(const PageAttnArgs& a, const int32_t* sel, int begin, int c, int& bad, F&& take) {
    const int lane = threadIdx.x & 31;
    int before = -1, next = begin;  // (the lane's of the first 32, read ahead by the caller)
    for (int i0 = 0; i0 < a.top; i0 += 32) {
        const int e = next;
        next = i0 + 32 + lane < a.top ? sel[i0 + 32 + lane] : -1;
        // the largest entry before this one: the one before it, where they ascend and no -1 stands between them
        int ahead = __shfl_up_sync(kFull, e, 1);
        if (lane == 0) ahead = before;
        const unsigned there = __ballot_sync(kFull, e >= 0);
        if ((there & (there + 1)) || __any_sync(kFull, e >= 0 && e <= ahead)) {
            int top = e;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(kFull, top, d);
                if (lane >= d) top = max(top, o);
            }
            ahead = __shfl_up_sync(kFull, top, 1);
            ahead = max(lane ? ahead : -1, before);
            before = max(before, __shfl_sync(kFull, top, 31));
        } else if (there) {
            before = __shfl_sync(kFull, e, 31 - __clz(there));
        }
        if (e >= 0) {
            if (e >= c || e <= ahead) bad |= HSQ_DEVERR_SEL;
            else take(e);
        }
    }
}

// ---------------------------------------------------------------------------------------
// Rows one by one: a cluster of CTAs for each (row, KV head), four warps a CTA.  The row's pages are listed once a CTA; the
// cluster's warps cut the line of their groups of 16 keys into equal runs.  A warp loads its groups three ahead (TMA, 128-byte
// swizzle, 8 KB each) and multiplies as
//   S^T (16 keys x 8 heads) = K (A operand, by ldmatrix) Q^T (B);
//   O^T (128 dims x 8 heads) += V^T (A, by transposing ldmatrix) P^T (B), P^T from S^T by two 8 x 8 transposes,
// so no lane exchanges logits but for a new maximum.  The warps' parts are joined in shared memory, the CTAs' through
// distributed shared memory: one launch and no workspace.
// Bound by the way of the pages: 64 rows x 8 heads x 2048 tokens take 61 us for 532 MB into the SMs (339 MB of it from HBM:
// rows share pages of the prefix), 8.7 TB/s; with a copy for each half of a row and twice the CTAs 75.  Few rows (4 x 8
// heads x 256 tokens) take 5.7 us: launch and four dependent loads.
// ---------------------------------------------------------------------------------------

constexpr int kWarps = 4, kThreadsRow = 32 * kWarps, kStages = 3;
constexpr uint32_t kStageBytes = 16 * 256 * 2, kWarpBytes = kStages * kStageBytes;
constexpr uint32_t kOffList = kWarps * kWarpBytes;                       // [top] int2: page id, tokens
constexpr uint32_t kOffWarpMl = kOffList + HSQ_MAX_BETA * 8;             // [warp][8] m, l
constexpr uint32_t kOffMl = kOffWarpMl + kWarps * 64;                    // [8] the CTA's
constexpr uint32_t kOffPart = kOffMl + 64;                               // [8][128] the CTA's o
constexpr uint32_t kOffBar = kOffPart + 8 * 512;
constexpr uint32_t kOffHead = kOffBar + kWarps * kStages * 8;            // pages listed, q row
constexpr uint32_t kRowSmem = kOffHead + 32 + 1024;                      // + alignment
static_assert(8 * 512 <= kWarpBytes, "a warp's part fits its stages");

__global__ void __launch_bounds__(kThreadsRow)
    page_attn_rows_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                          const __grid_constant__ PageAttnArgs a) {
    extern __shared__ uint8_t raw_smem[];
    const uint32_t raw = smem_addr(raw_smem), base = (raw + 1023u) & ~1023u;
    uint8_t* sm = raw_smem + (base - raw);
    int2* list = reinterpret_cast<int2*>(sm + kOffList);
    float2* warp_ml = reinterpret_cast<float2*>(sm + kOffWarpMl);
    float2* cta_ml = reinterpret_cast<float2*>(sm + kOffMl);
    float* cta_o = reinterpret_cast<float*>(sm + kOffPart);
    int* head = reinterpret_cast<int*>(sm + kOffHead);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    cg::cluster_group cluster = cg::this_cluster();
    const int S = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int unit = blockIdx.x / S, h = unit % a.Hkv;
    int row = unit / a.Hkv;
    int bad = 0;
    bool failed = false;

    if (a.few < a.max_new) {  // the rows that do not go by tiles
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (row >= a.head->shorts) return;  // (the whole cluster)
        row = a.short_row[row];
    }
    if (tid == 0) {
        for (int i = 0; i < kWarps * kStages; ++i) mbar_init(base + kOffBar + 8 * i, 1);
        mbar_init_fence();
    }
    if (warp == 0) {  // the row's pages
        const RowOf ro = warp_row(a.q_start, a.lens, a.B, a.rows, a.max_new, a.width << a.page_shift, row, bad);
        int n = 0;
        if (ro.live) {
            const int32_t* sel = a.sel + ((size_t)row * a.Hkv + h) * a.top;
            const int c = a.prefix_pages + ((ro.seen + a.page_n - 1) >> a.page_shift);
            int before = -1;  // the largest entry so far
            for (int i0 = 0; i0 < a.top; i0 += 32) {
                const int e = i0 + lane < a.top ? sel[i0 + lane] : -1;
                int most = e;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int o = __shfl_up_sync(kFull, most, d);
                    if (lane >= d) most = max(most, o);
                }
                int ahead = __shfl_up_sync(kFull, most, 1);
                ahead = max(lane ? ahead : -1, before);
                before = max(before, __shfl_sync(kFull, most, 31));
                bool ok = e >= 0;
                if (ok && (e >= c || e <= ahead)) {
                    ok = false;
                    bad |= HSQ_DEVERR_SEL;
                }
                int id = -1, tokens = 0;
                if (ok) {
                    const bool pre = e < a.prefix_pages;
                    id = pre ? a.prefix[e] : a.table[(size_t)ro.b * a.width + e - a.prefix_pages];
                    tokens = min(a.page_n, pre ? a.prefix_len - (e << a.page_shift) : ro.seen - ((e - a.prefix_pages) << a.page_shift));
                    if (id < 0 || id >= a.n_pages) {
                        ok = false;
                        bad |= HSQ_DEVERR_PAGE;
                    }
                }
                const unsigned in = __ballot_sync(kFull, ok);
                if (ok) list[n + __popc(in & ((1u << lane) - 1u))] = make_int2(id, tokens);
                n += __popc(in);
            }
        }
        if (lane == 0) {
            head[0] = n;
            head[1] = ro.live;
        }
    }
    if (blockIdx.x == 0) bad |= requests_bad(a.q_start, a.lens, a.B, a.rows, a.width << a.page_shift, kThreadsRow);
    __syncthreads();
    const int listed = head[0];
    const bool live = head[1];

    // the warp's groups [s, s1) of 16 keys
    const int sub_shift = a.page_shift - 4, groups = listed << sub_shift;
    const int w = rank * kWarps + warp, W = S * kWarps;
    const int s0 = (int)((long long)groups * w / W), s1 = (int)((long long)groups * (w + 1) / W);
    const uint32_t stages = base + warp * kWarpBytes, bars = base + kOffBar + 8 * kStages * warp;
    uint8_t* stages_g = sm + warp * kWarpBytes;
    Ring<kStages> in{0, 0}, out{0, 0};
    auto tokens_of = [&](int s) { return list[s >> sub_shift].y - 16 * (s & ((1 << sub_shift) - 1)); };  // of the group and behind
    int ask = s0;
    auto load = [&] {
        while (ask < s1 && tokens_of(ask) <= 0) ++ask;
        if (ask >= s1) return;
        const uint32_t dst = stages + in.stage * kStageBytes, bar = bars + 8 * in.stage;
        const int y = ((list[ask >> sub_shift].x * a.Hkv + h) << a.page_shift) + 16 * (ask & ((1 << sub_shift) - 1));
        if (lane == 0) mbar_expect_tx(bar, kStageBytes);
        __syncwarp();
        if (lane < 2) tma_3d(dst + 4096 * lane, lane ? &mv : &mk, 0, y, 0, bar);
        __syncwarp();
        in.advance();
        ++ask;
    };
    for (int i = 0; i < kStages; ++i) load();
    failed |= s0 < s1 && (a.fault & HSQ_FAULT_WAIT_FEW) != 0;
    uint32_t qf[8][2];
    {
        const bool in_use = live && g < a.r;
        const uint32_t* src = reinterpret_cast<const uint32_t*>(a.q + ((size_t)row * a.Hq + h * a.r + (in_use ? g : 0)) * 128 + 2 * t);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
            qf[kk][0] = in_use ? src[8 * kk] : 0u;
            qf[kk][1] = in_use ? src[8 * kk + 4] : 0u;
        }
    }
    float o[8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    // lane's row of the 8 x 8 matrices that ldmatrix takes: K: keys (lane & 15), chunks 2 kk + (lane >> 4);
    // V: keys (lane & 7) + 8 (lane >> 4), chunks 2 i + ((lane >> 3) & 1)
    const uint32_t k_row = (lane & 15) * 128, k_x = lane & 7, k_c = lane >> 4;
    const uint32_t v_row = ((lane & 7) + 8 * (lane >> 4)) * 128, v_c = (lane >> 3) & 1;
#pragma unroll 1
    for (int s = s0; s < s1 && !failed; ++s) {
        const int valid = tokens_of(s);
        if (valid <= 0) continue;
        const uint32_t kb = stages + out.stage * kStageBytes, vb = kb + 4096;
        mbar_wait_fast(bars + 8 * out.stage, out.phase, failed, a.polls);
        failed = __any_sync(kFull, failed);
        if (failed) break;
        if (valid < 16) {  // the rest of the page is stale: weight 0, but it has to be finite
            for (int i = lane; i < (16 - valid) * 16; i += 32)
                *reinterpret_cast<uint4*>(stages_g + out.stage * kStageBytes + 4096 + ((i >> 3) & 1) * 2048 + (valid + (i >> 4)) * 128 +
                                          (i & 7) * 16) = make_uint4(0, 0, 0, 0);
            fence_async_smem();
            __syncwarp();
        }
        float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
            uint32_t k[4];
            ldmatrix(k, kb + (kk >> 2) * 2048 + k_row + ((((2 * kk + k_c) & 7) ^ k_x) << 4));
            mma_16816(x, k, qf[kk][0], qf[kk][1]);
        }
        bool look = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // key g + 8 (e >> 1), head 2 t + (e & 1)
            if (g + 8 * (e >> 1) >= valid) x[e] = -INFINITY;
            look |= x[e] * kLogitScaleLog2 > m[e & 1] * kLogitScaleLog2 + 8.f;  // (the first key raises from -inf)
        }
        if (__any_sync(kFull, look)) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mx = fmaxf(m[e], fmaxf(x[e], x[e + 2]));
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, d));
                const float alpha = mx == -INFINITY ? 1.f : ex2_approx((m[e] - mx) * kLogitScaleLog2);
                m[e] = mx;
                l[e] *= alpha;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    o[i][e] *= alpha;
                    o[i][e + 2] *= alpha;
                }
            }
        }
        float pr[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float off = m[e & 1] == -INFINITY ? 0.f : m[e & 1] * kLogitScaleLog2;
            pr[e] = ex2_approx(fmaf(x[e], kLogitScaleLog2, -off));
            l[e & 1] += pr[e];
        }
        const uint32_t p0 = transpose_8x8(pack_bf16(pr[0], pr[1])), p1 = transpose_8x8(pack_bf16(pr[2], pr[3]));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t v[4];
            ldmatrix_trans(v, vb + (i >> 2) * 2048 + v_row + ((((2 * i + v_c) & 7) ^ k_x) << 4));
            mma_16816(o[i], v, p0, p1);
        }
        __syncwarp();  // (every lane has read the stage)
        out.advance();
        load();
    }
    if (failed) {  // see the copies in flight (one a stage at most) land: their memory is used again
        for (int i = 0; i < kStages; ++i) mbar_wait(bars + 8 * i, i < (int)in.stage ? in.phase : in.phase ^ 1, 1 << 12);
        bad |= HSQ_DEVERR_WAIT;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    }
    // the warp's part
    float* part = reinterpret_cast<float*>(stages_g);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[e] += __shfl_xor_sync(kFull, l[e], d);
        const int j = 2 * t + e;
        if (g == 0) warp_ml[8 * warp + j] = make_float2(m[e], l[e]);
        if (!failed) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                part[j * 128 + 16 * i + g] = o[i][e];
                part[j * 128 + 16 * i + 8 + g] = o[i][e + 2];
            }
        }
    }
    __syncthreads();
    for (int j = 0; j < a.r; ++j) {  // the CTA's: a thread a dim
        float M = -INFINITY, L = 0.f, y = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) M = fmaxf(M, warp_ml[8 * i + j].x);
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            const float2 ml = warp_ml[8 * i + j];
            if (ml.y == 0.f) continue;
            const float c = ex2_approx((ml.x - M) * kLogitScaleLog2);
            L = fmaf(ml.y, c, L);
            y = fmaf(reinterpret_cast<const float*>(sm + i * kWarpBytes)[j * 128 + tid], c, y);
        }
        cta_o[j * 128 + tid] = y;
        if (tid == 0) cta_ml[j] = make_float2(M, L);
    }
    cluster.sync();
    for (int e = rank * kThreadsRow + tid; e < a.r * 64; e += S * kThreadsRow) {
        const int j = e >> 6, d = 2 * (e & 63);
        float M = -INFINITY, L = 0.f, y0 = 0.f, y1 = 0.f;
        for (int i = 0; i < S; ++i) M = fmaxf(M, cluster.map_shared_rank(cta_ml, i)[j].x);
        for (int i = 0; i < S; ++i) {
            const float2 ml = cluster.map_shared_rank(cta_ml, i)[j];
            if (ml.y == 0.f) continue;
            const float c = ex2_approx((ml.x - M) * kLogitScaleLog2);
            const float2 y = *reinterpret_cast<const float2*>(cluster.map_shared_rank(cta_o, i) + j * 128 + d);
            L = fmaf(ml.y, c, L);
            y0 = fmaf(y.x, c, y0);
            y1 = fmaf(y.y, c, y1);
        }
        if (live) {
            const float inv = L == 0.f ? 0.f : 1.0f / L;  // (a sum that is not a number shows in the result)
            const size_t to = (size_t)row * a.Hq + h * a.r + j;
            *reinterpret_cast<uint32_t*>(a.out + to * 128 + d) = pack_bf16(y0 * inv, y1 * inv);
            if (a.lse && d == 0) a.lse[to] = L == 0.f ? -INFINITY : M * kRsqrtD + logf(L);
        }
    }
    cluster.sync();  // (no CTA ends while another reads its part)
    if (bad) atomicOr(a.err, bad);
}

// ---------------------------------------------------------------------------------------
// Requests of few rows at once (proposals): a cluster of CTAs for each (request, KV head), over the union of its rows' pages, so that
// a page that several rows take is read once.  The columns of the products are the rows (token x head); a CTA has four streams of
// keys, and H warps a stream with 16 columns each that share its stages.  The CTAs list the union in shared memory (a word of
// token bits for each page, in the memory that the stages use afterwards); the rest is as for single rows.
// 24 requests x 5 rows of 40/8 heads, 64 pages of 16 tokens each: 48 us for 146 MB (row by row 67).  Bound by latency and the
// products' pipe: a step of 16 keys takes a warp 1500 to 1900 cycles, in which an SM quarter's four warps have 1050 of products.
// ---------------------------------------------------------------------------------------

constexpr int kGroupStages = 3, kGroupList = 400;  // pages of a union at most, a CTA of the cluster
constexpr uint32_t kGroupWarpBytes = kGroupStages * kStageBytes, kGroupQPitch = 272;  // (272: a fragment's words lie in 32 banks)
constexpr uint32_t kGOffList = kWarps * kGroupWarpBytes;               // [kGroupList] int4: page id, logical page, tokens
constexpr uint32_t kGOffWeight = kGOffList;                            // (once the list has served) [warp][32] weights in the CTA's
constexpr uint32_t kGOffCta = kGOffWeight + kWarps * 32 * 4;           // [32] the CTA's m, l
constexpr uint32_t kGOffAll = kGOffCta + 32 * 8;                       // [CTA][32] the cluster's
constexpr uint32_t kGOffMl = kGOffList + kGroupList * 16;              // [warp][32] m, l
constexpr uint32_t kGOffBar = kGOffMl + kWarps * 32 * 8;
static_assert(kGOffAll + 8 * 32 * 8 <= kGOffMl, "");
constexpr uint32_t kGOffScan = kGOffBar + kWarps * kGroupStages * 16;  // [warps]
constexpr uint32_t kGOffQ = kGOffScan + 32;                            // [16 H] rows' queries
constexpr uint32_t group_smem(int H) { return kGOffQ + 16 * H * kGroupQPitch + 1024; }  // + alignment
static_assert(32 * 512 <= kGroupWarpBytes, "a stream's part fits its stages");
static_assert(kGOffQ % 16 == 0 && group_smem(2) <= 113 * 1024, "two CTAs an SM");

template <int H>
__global__ void __launch_bounds__(kThreadsRow * H, 2)
    page_attn_group_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                           const __grid_constant__ PageAttnArgs a) {
    constexpr int kThreads = kThreadsRow * H, kAllWarps = kWarps * H, NT = 2;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (the plan reads nothing of what is written here)
    extern __shared__ uint8_t raw_smem[];
    const uint32_t raw = smem_addr(raw_smem), base = (raw + 1023u) & ~1023u;
    uint8_t* sm = raw_smem + (base - raw);
    int4* list = reinterpret_cast<int4*>(sm + kGOffList);
    float2* warp_ml = reinterpret_cast<float2*>(sm + kGOffMl);
    float2* cta_ml = reinterpret_cast<float2*>(sm + kGOffCta);
    int* scan = reinterpret_cast<int*>(sm + kGOffScan);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int stream = warp / H, half = warp % H, col0 = 16 * half;  // the warp's keys, its columns' first
    cg::cluster_group cluster = cg::this_cluster();
    const int S = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int unit = blockIdx.x / S, h = unit % a.Hkv, b = unit / a.Hkv;
    int bad = 0;
    bool failed = false;

    const int first = a.q_start[b], end = a.q_start[b + 1], l_given = a.lens[b];
    int n = end - first;
    if (first < 0 || end < first || end > a.rows || n > a.max_new) {
        bad |= HSQ_DEVERR_LEN;
        n = 0;
    }
    const int held = min(max(l_given, 0), a.width << a.page_shift);
    if (held != l_given || l_given < n) bad |= HSQ_DEVERR_LEN;
    if (n > a.few) n = 0;  // (by tiles)
    const int ahead = max(l_given, 0) - n;
    auto seen_of = [&](int tok) { return min(max(ahead + tok + 1, 0), held); };
    auto pages_of = [&](int tok) { return a.prefix_pages + ((seen_of(tok) + a.page_n - 1) >> a.page_shift); };
    const int last_seen = n > 0 ? seen_of(n - 1) : 0, columns = n * a.r;

    if (tid == 0) {
        for (int i = 0; i < kWarps * kGroupStages; ++i) {
            mbar_init(base + kGOffBar + 8 * i, 1);
            mbar_init(base + kGOffBar + 8 * (kWarps * kGroupStages + i), H);
        }
        mbar_init_fence();
    }
    for (int i = tid; i < 16 * H * 16; i += kThreads) {  // 16 bytes each
        const int col = i >> 4, tok = col / a.r, head = col - tok * a.r;
        uint8_t* to = sm + kGOffQ + col * kGroupQPitch + 16 * (i & 15);
        if (col < columns) cp_async16(to, a.q + ((size_t)(first + tok) * a.Hq + h * a.r + head) * 128 + 8 * (i & 15));
        else *reinterpret_cast<uint4*>(to) = make_uint4(0, 0, 0, 0);
    }
    cp_async_commit();

    // ---- the union of the rows' pages ----
    // (the words of up to 24576 pages lie in the stages' memory; of more, which only pages of 16 or 32 tokens can be, in two
    // goes, the first only counted where a second follows)
    const int sub_shift = a.page_shift - 4;
    int listed = 0, page0 = 0, here = 0;  // pages of the union; the CTA's first and number of them
    {
        uint32_t* word = reinterpret_cast<uint32_t*>(sm);
        constexpr int kWindow = kWarps * kGroupWarpBytes / 4;
        const int most = n > 0 ? pages_of(n - 1) : 0, windows = (most + kWindow - 1) / kWindow;
        int total = 0;
        for (int go = 0; go < (windows > 1 ? 2 : 1); ++go) {
            const bool write = windows <= 1 || go == 1;
            int at0 = 0;
            for (int w0 = 0; w0 < most; w0 += kWindow) {
                const int w1 = min(most, w0 + kWindow);
                for (int i = tid; i < w1 - w0; i += kThreads) word[i] = 0;
                __syncthreads();
                const int32_t* sel = a.sel + ((size_t)(first + warp) * a.Hkv + h) * a.top;
                const size_t step = (size_t)kAllWarps * a.Hkv * a.top;
                int ahead = warp < n && lane < a.top ? sel[lane] : -1;
                for (int tok = warp; tok < n; tok += kAllWarps, sel += step) {
                    const int begin = ahead;
                    ahead = tok + kAllWarps < n && lane < a.top ? sel[step + lane] : -1;
                    for_selected(a, sel, begin, pages_of(tok), bad, [&](int e) {
                        if (e >= w0 && e < w1) atomicOr(word + e - w0, 1u << tok);
                    });
                }
                __syncthreads();
                // a thread's share of the pages (an odd number, for the banks): counted, then written
                const int share = ((w1 - w0 + kThreads - 1) / kThreads) | 1, i0 = min(tid * share, w1 - w0), i1 = min(i0 + share, w1 - w0);
                int mine = 0;
                for (int i = i0; i < i1; ++i) mine += word[i] != 0;
                int at = mine;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int x = __shfl_up_sync(kFull, at, d);
                    if (lane >= d) at += x;
                }
                if (lane == 31) scan[warp] = at;
                __syncthreads();
                at += at0 - mine;
#pragma unroll
                for (int w = 0; w < kAllWarps; ++w) {
                    if (w < warp) at += scan[w];
                    at0 += scan[w];
                }
                if (write) {
                    if (windows <= 1) total = at0;
                    // the pages of the groups [total rank / S, total (rank + 1) / S)
                    page0 = (int)((long long)total * rank / S);
                    here = (int)((long long)total * (rank + 1) / S) - page0;
                    for (int i = i0; i < i1; ++i)
                        if (word[i] != 0) {
                            if (at >= page0 && at - page0 < min(here, kGroupList)) list[at - page0] = make_int4(0, w0 + i, (int)word[i], 0);
                            ++at;
                        }
                }
                __syncthreads();
            }
            if (!write) total = at0;
        }
        listed = total;
        here = min(here, kGroupList);
        for (int i = tid; i < here; i += kThreads) {
            const int e = list[i].y;
            const int id = e < a.prefix_pages ? a.prefix[e] : a.table[(size_t)b * a.width + e - a.prefix_pages];
            const bool in = id >= 0 && id < a.n_pages;
            if (!in) bad |= HSQ_DEVERR_PAGE;
            list[i].x = in ? id : 0;
            if (!in) list[i].z = 0;
        }
        cp_async_wait_all();
        fence_async_smem();  // (the words' memory takes copies from here on)
        __syncthreads();
    }
    if (blockIdx.x == 0) bad |= requests_bad(a.q_start, a.lens, a.B, a.rows, a.width << a.page_shift, kThreads);

    // the warp's groups [s0, s1) of 16 keys, of the CTA's
    const int groups = here << sub_shift, s0 = groups * stream / kWarps, s1 = groups * (stream + 1) / kWarps;
    const uint32_t stages = base + stream * kGroupWarpBytes, bars = base + kGOffBar + 8 * kGroupStages * stream;
    const uint32_t read = bars + 8 * kWarps * kGroupStages;  // every warp of the stream has read the stage
    uint8_t* stages_g = sm + stream * kGroupWarpBytes;
    Ring<kGroupStages> in{0, 0}, out{0, 0};
    // place of the group's first key among the prefix's tokens or the request's own
    auto begin_of = [&](int s, int lp) {
        return ((lp < a.prefix_pages ? lp : lp - a.prefix_pages) << a.page_shift) + 16 * (s & ((1 << sub_shift) - 1));
    };
    auto valid_of = [&](int s) {  // tokens of the group and behind that any row sees; 0: nothing to do
        const int4 e = list[s >> sub_shift];
        return e.z == 0 ? 0 : (e.y < a.prefix_pages ? a.prefix_len : last_seen) - begin_of(s, e.y);
    };
    int ask = s0, asked = 0;
    auto load = [&] {  // (by the stream's first warp)
        if (half != 0) return;
        while (ask < s1 && valid_of(ask) <= 0) ++ask;
        if (ask >= s1) return;
        if (H > 1 && ++asked > kGroupStages) {
            mbar_wait_fast(read + 8 * in.stage, in.phase ^ 1, failed, a.polls);
            failed = __any_sync(kFull, failed);
            if (failed) return;
        }
        const uint32_t dst = stages + in.stage * kStageBytes, bar = bars + 8 * in.stage;
        const int y = ((list[ask >> sub_shift].x * a.Hkv + h) << a.page_shift) + 16 * (ask & ((1 << sub_shift) - 1));
        if (lane == 0) mbar_expect_tx(bar, kStageBytes);
        __syncwarp();
        if (lane < 2) tma_3d(dst + 4096 * lane, lane ? &mv : &mk, 0, y, 0, bar);
        __syncwarp();
        in.advance();
        ++ask;
    };
    for (int i = 0; i < kGroupStages; ++i) load();
    failed |= s0 < s1 && (a.fault & HSQ_FAULT_WAIT_FEW) != 0;
    float o[NT][8][4], m[NT][2], l[NT][2];
    int seen[NT][2];        // of the lane's columns col0 + 8 nt + 2 t + e
    uint32_t bit[NT][2];    // their tokens' bits (0: no row)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int col = col0 + 8 * nt + 2 * t + e, tok = col / a.r;
            seen[nt][e] = seen_of(tok);
            bit[nt][e] = col < columns ? 1u << tok : 0u;
            m[nt][e] = -INFINITY;
            l[nt][e] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
    }
    const uint32_t k_row = (lane & 15) * 128, k_x = lane & 7, k_c = lane >> 4;
    const uint32_t v_row = ((lane & 7) + 8 * (lane >> 4)) * 128, v_c = (lane >> 3) & 1;
    // queries: rows (lane & 7), 16 bytes lane >> 3 of the two k steps' 64
    const uint32_t q_lane = base + kGOffQ + (col0 + (lane & 7)) * kGroupQPitch + 16 * (lane >> 3);
#pragma unroll 1
    for (int s = s0; s < s1 && !failed; ++s) {
        const int valid = valid_of(s);
        if (valid <= 0) continue;
        const int4 page = list[s >> sub_shift];
        const uint32_t kb = stages + out.stage * kStageBytes, vb = kb + 4096;
        mbar_wait_fast(bars + 8 * out.stage, out.phase, failed, a.polls);
        failed = __any_sync(kFull, failed);
        if (failed) break;
        if (valid < 16) {  // the rest of the page is stale: weight 0, but it has to be finite
            for (int i = lane; i < (16 - valid) * 16; i += 32)
                *reinterpret_cast<uint4*>(stages_g + out.stage * kStageBytes + 4096 + ((i >> 3) & 1) * 2048 + (valid + (i >> 4)) * 128 +
                                          (i & 7) * 16) = make_uint4(0, 0, 0, 0);
            fence_async_smem();
            __syncwarp();
        }
        float x[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.f;
        // (tiles whose tokens do not take the page are multiplied too: a branch would keep the products of the others apart)
#pragma unroll
        for (int kk = 0; kk < 8; kk += 2) {
            uint32_t k0[4], k1[4];
            ldmatrix(k0, kb + (kk >> 2) * 2048 + k_row + ((((2 * kk + k_c) & 7) ^ k_x) << 4));
            ldmatrix(k1, kb + (kk >> 2) * 2048 + k_row + ((((2 * kk + 2 + k_c) & 7) ^ k_x) << 4));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                uint32_t q[4];
                ldmatrix(q, q_lane + nt * 8 * kGroupQPitch + 32 * kk);
                mma_16816(x[nt], k0, q[0], q[1]);
                mma_16816(x[nt], k1, q[2], q[3]);
            }
        }
        const int begin = begin_of(s, page.y);
        const bool pre = page.y < a.prefix_pages;
        bool look = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {  // key g + 8 (e >> 1), column 8 nt + 2 t + (e & 1)
                const int keys = (page.z & bit[nt][e & 1]) ? (pre ? a.prefix_len : seen[nt][e & 1]) - begin : 0;
                if (g + 8 * (e >> 1) >= keys) x[nt][e] = -INFINITY;
                look |= x[nt][e] * kLogitScaleLog2 > m[nt][e & 1] * kLogitScaleLog2 + 8.f;  // (the first key raises from -inf)
            }
        if (__any_sync(kFull, look)) {
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
        if (H > 1 && lane == 0) mbar_arrive(read + 8 * out.stage);
        out.advance();
        load();
    }
    if (failed) {  // see the copies in flight (one a stage at most) land: their memory is used again
        if (half == 0)
            for (int i = 0; i < kGroupStages; ++i) mbar_wait(bars + 8 * i, i < (int)in.stage ? in.phase : in.phase ^ 1, 1 << 12);
        bad |= HSQ_DEVERR_WAIT;
    }
    // the warp's part (its stream's stages are free once every warp of it is through)
    if (H > 1) __syncthreads();
    float* part = reinterpret_cast<float*>(stages_g);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[nt][e] += __shfl_xor_sync(kFull, l[nt][e], d);
            const int j = col0 + 8 * nt + 2 * t + e;
            if (g == 0) warp_ml[32 * stream + j] = failed ? make_float2(-INFINITY, 0.f) : make_float2(m[nt][e], l[nt][e]);
            if (!failed && j < columns) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    part[j * 128 + 16 * i + g] = o[nt][i][e];
                    part[j * 128 + 16 * i + 8 + g] = o[nt][i][e + 2];
                }
            }
        }
    __syncthreads();
    float* weight = reinterpret_cast<float*>(sm + kGOffWeight);
    {
        float M = -INFINITY;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) M = fmaxf(M, warp_ml[32 * i + lane].x);
        float L = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            const float2 ml = warp_ml[32 * i + lane];
            const float c = ml.y == 0.f ? 0.f : ex2_approx((ml.x - M) * kLogitScaleLog2);
            L = fmaf(ml.y, c, L);
            if (i == warp) weight[32 * i + lane] = c;
        }
        if (warp == 0) cta_ml[lane] = make_float2(M, L);
    }
    __syncthreads();
    float* cta_o = reinterpret_cast<float*>(sm);  // the CTA's, in the first stream's place: a thread a dim
#pragma unroll 4
    for (int j = tid >> 7; j < columns; j += H) {
        const int d = tid & 127;
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i)
            y = fmaf(reinterpret_cast<const float*>(sm + i * kGroupWarpBytes)[j * 128 + d], weight[32 * i + j], y);
        cta_o[j * 128 + d] = y;
    }
    cluster.sync();
    float2* all_ml = reinterpret_cast<float2*>(sm + kGOffAll);
    for (int i = tid; i < 32 * S; i += kThreads) all_ml[i] = cluster.map_shared_rank(cta_ml, i >> 5)[i & 31];
    __syncthreads();
#pragma unroll 1
    for (int e = rank * kThreads + tid; e < columns * 32; e += S * kThreads) {
        const int j = e >> 5, d = 4 * (e & 31);
        float4 y[8];
        float M = -INFINITY, L = 0.f, z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < S) {
                y[i] = *reinterpret_cast<const float4*>(cluster.map_shared_rank(cta_o, i) + j * 128 + d);
                M = fmaxf(M, all_ml[32 * i + j].x);
            }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < S) {
                const float2 ml = all_ml[32 * i + j];
                const float c = ml.y == 0.f ? 0.f : ex2_approx((ml.x - M) * kLogitScaleLog2);
                L = fmaf(ml.y, c, L);
                z[0] = fmaf(y[i].x, c, z[0]);
                z[1] = fmaf(y[i].y, c, z[1]);
                z[2] = fmaf(y[i].z, c, z[2]);
                z[3] = fmaf(y[i].w, c, z[3]);
            }
        const float inv = L == 0.f ? 0.f : 1.0f / L;  // (a sum that is not a number shows in the result)
        const int tok = j / a.r;
        const size_t to = (size_t)(first + tok) * a.Hq + h * a.r + j - tok * a.r;
        *reinterpret_cast<uint2*>(a.out + to * 128 + d) = make_uint2(pack_bf16(z[0] * inv, z[1] * inv), pack_bf16(z[2] * inv, z[3] * inv));
        if (a.lse && d == 0) a.lse[to] = L == 0.f ? -INFINITY : M * kRsqrtD + logf(L);
    }
    cluster.sync();  // (no CTA ends while another reads its part)
    if (bad) atomicOr(a.err, bad);
}

// ---------------------------------------------------------------------------------------
// Rows by tiles, for requests of many tokens (a prompt's chunk).  A tile is 128 rows: 128 / r neighbouring tokens times the r
// heads of a KV head.  Its tokens select different pages, but neighbours many of the same: the tile's products run over the
// UNION of their pages on the tensor cores, and the softmax hides the pages that a row did not take.
//   plan     checks the lengths; lists the pairs of tiles of the long requests, and the rows of the others;
//   list     for each item (pair, KV head): the pages that both tiles take, those of the first alone and of the second
//            alone, with the tokens that take them;
//   tiles    the items' key tiles as one line of cost, cut into equal runs, a persistent CTA each; an item that no cut
//            divides is written at once, else its parts go to the workspace;
//   join     adds the parts up.
// Two streams (a row tile each, S / P and O in tensor memory) share the key tiles that both take and have
// those that one takes in turn, so that while one stream's softmax runs the tensor cores work for the other.  A lone
// tile is given to both streams, which take its key tiles in turn and are joined through tensor memory.
// A chunk of 2048 tokens over 32K (32/8 heads, 64 of 1024 pages a row and head): 385 us, row by row 1530.  The rows of a tile
// take 450 pages, seven times a row's, so the products are 0.48 TFLOP where the selection's own are 0.07; the tiles' kernel
// does them in 356 us, 1.36 PFLOP/s.  Bound by the way of the pages into the SMs, 2.7 GB at 7.6 TB/s
// (single rows reach 8.7; with all loads from the same 256 KB the call took 371 us where it took 380), beside the MMA thread
// and the softmax in turn: a tile of 128 rows x 128 keys takes an SM 1750 cycles, 1024 of them the pipe's.  The union, and the
// time, shrink where neighbouring rows take the same pages.
// ---------------------------------------------------------------------------------------

constexpr int kTileRows = 128, kTileKeys = 128;
constexpr float kTileSum = 65536.f;  // sum of a tile's 128 weights from which the maximum is taken anew
// Requests of up to this many rows (tokens x heads) go row by row.
constexpr int kFewColumns = 32;
constexpr int kRunLeast = 6;         // cost of a run at least

constexpr int kPlanThreads = 512;

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const __grid_constant__ PageAttnArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ int s_w[2][kPlanThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int bad = 0, units = 0, shorts = 0;  // before the round
    for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int first = 0, n = 0, l = 0, held = 0;
        if (b < a.B) {
            const int s = a.q_start[b], e = a.q_start[b + 1];
            l = a.lens[b];
            if (s < 0 || e < s || e > a.rows || e - s > a.max_new) {
                bad |= HSQ_DEVERR_LEN;
            } else {
                first = s;
                n = e - s;
            }
            held = min(max(l, 0), a.width << a.page_shift);
            if (held != l || l < n) bad |= HSQ_DEVERR_LEN;
            a.req[b] = make_int4(first, n, held, max(l, 0) - n);
        }
        const int mine[2] = {n > a.few ? (n + 2 * a.tpt - 1) / (2 * a.tpt) : 0, n > a.few ? 0 : n};
        int x[2] = {min(mine[0], a.units_cap + 1), min(mine[1], a.rows_cap + 1)};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(kFull, x[k], o);
                if (lane >= o) x[k] += u;
            }
            if (lane == 31) s_w[k][warp] = x[k];
        }
        __syncthreads();
        int before[2] = {units, shorts}, total[2] = {units, shorts};
#pragma unroll
        for (int k = 0; k < 2; ++k)
            for (int w = 0; w < kPlanThreads / 32; ++w) {
                if (w == warp) before[k] = total[k];
                total[k] = min(total[k] + s_w[k][w], 1 << 29);
            }
        // (offsets that overlap can ask for more than there is room for: those behind are left out)
        const int at_u = before[0] + x[0] - mine[0], at_s = before[1] + x[1] - mine[1];
        for (int i = 0; i < mine[0]; ++i) {
            if (at_u + i >= a.units_cap) { bad |= HSQ_DEVERR_LEN; break; }
            a.unit[at_u + i] = make_int2(b, i);
        }
        for (int i = 0; i < mine[1]; ++i) {
            if (at_s + i >= a.rows_cap) { bad |= HSQ_DEVERR_LEN; break; }
            a.short_row[at_s + i] = first + i;
        }
        units = total[0];
        shorts = total[1];
        __syncthreads();
    }
    if (tid == 0) *a.head = TileHead{min(units, a.units_cap), min(shorts, a.rows_cap)};
    if (bad) atomicOr(a.err, bad);
    asm volatile("griddepcontrol.wait;" ::: "memory");  // (so that the end of the call's last kernel is the end of the groups' too)
}

// The tokens of a pair of tiles.
struct Pair {
    int b, first, toks[2];  // request; first token's row; tokens of the two tiles
    int held, ahead;        // token t of the pair sees min(max(ahead + t + 1, 0), held) own tokens
};
__device__ __forceinline__ Pair pair_of(const PageAttnArgs& a, int unit) {
    const int2 u = a.unit[unit];
    const int4 q = a.req[u.x];
    const int j0 = u.y * 2 * a.tpt, left = q.y - j0;
    Pair p;
    p.b = u.x;
    p.first = q.x + j0;
    p.toks[0] = min(left, a.tpt);
    p.toks[1] = min(max(left - a.tpt, 0), a.tpt);
    p.held = q.z;
    p.ahead = q.w + j0;
    return p;
}

constexpr int kListThreads = 1024, kListWarps = kListThreads / 32, kListBytes = 32768;

__global__ void __launch_bounds__(kListThreads) page_list_kernel(const __grid_constant__ PageAttnArgs a) {
    __shared__ uint32_t s_mask[kListBytes / 4];  // [page of the window][2][words]
    __shared__ int s_n[3][kListWarps], s_all[3];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int units = a.head->units, unit = blockIdx.x / a.Hkv, h = blockIdx.x - unit * a.Hkv;
    if (unit >= units) return;
    const int item = h * units + unit, W = a.words, W2 = 2 * W, window = kListBytes / 4 / W2;
    const Pair p = pair_of(a, unit);
    const int toks = p.toks[0] + p.toks[1];
    auto pages_of = [&](int t) {
        const int seen = min(max(p.ahead + t + 1, 0), p.held);
        return a.prefix_pages + ((seen + a.page_n - 1) >> a.page_shift);
    };
    const int most = pages_of(toks - 1);
    int bad = 0, n[3] = {0, 0, 0};
    for (int w0 = 0; w0 < most; w0 += window) {
        const int w1 = min(most, w0 + window);
        for (int i = tid; i < (w1 - w0) * W2; i += kListThreads) s_mask[i] = 0;
        __syncthreads();
        const int32_t* sel = a.sel + ((size_t)(p.first + warp) * a.Hkv + h) * a.top;
        const size_t step = (size_t)kListWarps * a.Hkv * a.top;
        int ahead = warp < toks && lane < a.top ? sel[lane] : -1;
        for (int t = warp; t < toks; t += kListWarps, sel += step) {
            const int tile = t >= p.toks[0], i = tile ? t - p.toks[0] : t, begin = ahead;
            ahead = t + kListWarps < toks && lane < a.top ? sel[step + lane] : -1;
            for_selected(a, sel, begin, pages_of(t), bad, [&](int e) {
                if (e >= w0 && e < w1) atomicOr(&s_mask[(e - w0) * W2 + tile * W + (i >> 5)], 1u << (i & 31));
            });
        }
        __syncthreads();
        for (int i0 = w0; i0 < w1; i0 += kListThreads) {
            const int e = i0 + tid;
            uint32_t m[8];
            bool in[2] = {false, false};
            int id = -1;
            if (e < w1) {
                for (int k = 0; k < W2; ++k) {
                    m[k & 7] = s_mask[(e - w0) * W2 + k];
                    in[k >= W] |= m[k & 7] != 0;
                }
                if (in[0] | in[1]) {
                    id = e < a.prefix_pages ? a.prefix[e] : a.table[(size_t)p.b * a.width + e - a.prefix_pages];
                    if (id < 0 || id >= a.n_pages) {
                        bad |= HSQ_DEVERR_PAGE;
                        in[0] = in[1] = false;
                    }
                }
            }
            const int kind = in[0] ? (in[1] ? 0 : 1) : in[1] ? 2 : 3;
            int at = 0;
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const unsigned bl = __ballot_sync(kFull, kind == k);
                if (lane == 0) s_n[k][warp] = __popc(bl);
                if (kind == k) at = __popc(bl & ((1u << lane) - 1u));
            }
            __syncthreads();
            if (warp < 3) {  // before each warp, and in all
                const int own = s_n[warp][lane];
                int x = own;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int y = __shfl_up_sync(kFull, x, d);
                    if (lane >= d) x += y;
                }
                s_n[warp][lane] = x - own;
                if (lane == 31) s_all[warp] = x;
            }
            __syncthreads();
            if (kind < 3) at += s_n[kind][warp] + (kind == 0 ? n[0] : kind == 1 ? n[1] : n[2]);
#pragma unroll
            for (int k = 0; k < 3; ++k) n[k] += s_all[k];
            if (kind < 3) {
                const size_t to = ((size_t)item * 3 + kind) * a.cap + at;
                a.ent[to] = make_int2(id, e);
                for (int k = 0; k < W2; ++k) a.mask[to * W2 + k] = m[k & 7];
            }
            __syncthreads();
        }
    }
    if (tid == 0) {
        const int per = kTileKeys >> a.page_shift;
        const int tb = (n[0] + per - 1) / per, t0 = (n[1] + per - 1) / per, t1 = (n[2] + per - 1) / per;
        a.count[item] = make_int4(n[0], n[1], n[2], max(2 * tb + t0 + t1, 1));  // (an item without a page is written too)
    }
    if (bad) atomicOr(a.err, bad);
}

// ---- tiles ------------------------------------------------------------------------------

constexpr int kTcThreads = 384, kKeyStages = 3, kValueStages = 2, kTileStages = kKeyStages + kValueStages, kQueue = 2;
constexpr uint32_t kTileBytes = 128 * 128 * 2, kHalfBytes = kTileBytes / 2;
// Keys and values lie in groups of 8 rows, the group's halves side by side (kGroupHalf apart), so that a page is one copy (with a
// copy for each half, and the copies behind the notes, a chunk of 2048 over 32K 387 us where it takes 380 otherwise).
constexpr uint32_t kGroupBytes = 8 * 256, kGroupHalf = kGroupBytes / 2;
constexpr uint32_t kOffQ = kTileStages * kTileBytes, kOffBars = kOffQ + 2 * kTileBytes;
// barriers: full[5] | empty[5] | q_full[2] | q_empty[2] | s_full[2] | p_full[2] | o_full[2] | tail | drain | m_full | m_free | seg_full[2] | seg_empty[2] | note_full[5]
constexpr int kNotes = 5;
constexpr int kTcBars = (2 * kTileStages + 16 + 2 * kQueue + kNotes + 1) / 2 * 2;
constexpr uint32_t kSegBytes = 96;
constexpr uint32_t kOffSeg = kOffBars + 8 * kTcBars;
// Notes on the key tiles, written with their keys' load: [0] what the MMA thread does (kNote*), [1] the tile's pages, bit
// 8: the softmax has to look at single keys, [4 + i] page i's logical number, then [tile][word][page] the tiles' tokens that take it.
// Five, because a softmax may be four tiles behind the loads.
constexpr int kNotePages = 4, kNoteMasks = 12, kNoteWords = kNoteMasks + 64;
enum : uint32_t { kNoteStreams = 3, kNoteFirst = 4, kNoteLast = 16, kNoteEnd = 64, kNoteGroups = 8 /* shift */ };
constexpr uint32_t kOffNote = kOffSeg + kQueue * kSegBytes + 16;        // (+ TMEM address)
static_assert(kOffNote % 16 == 0 && kNoteWords % 4 == 0, "eight words of a mask are read as two vectors");
constexpr uint32_t kTcSmem = kOffNote + kNotes * kNoteWords * 4 + 1024;  // + alignment
static_assert(kOffSeg % 16 == 0, "segments lie on 16-byte boundaries");
static_assert(kTcSmem <= 232448, "shared memory of a CTA");
constexpr int kSegReaders = 10;  // 8 softmax warps, the loaders of queries and values

// The key tiles [n0, n1) of an item that a run holds.
struct alignas(16) TileSegment {
    int live, h, item, slot;
    int n0, n1, whole, split;        // split: both streams hold the first's tokens
    int first, toks0, toks1;         // first token's row; the streams' tokens
    int held, ahead;
    int pages[3];                    // both, first alone, second alone
    int tiles[3];
    int pad[5];
};
static_assert(sizeof(TileSegment) == kSegBytes, "");

// Key tile t: the streams that take it (bits), its pages.
struct KeyTile {
    int streams, region, at, np;
};
__device__ __forceinline__ KeyTile key_tile(const TileSegment& s, int t, int per) {
    KeyTile k;
    int pages;
    const int x = t - s.tiles[0], m = 2 * min(s.tiles[1], s.tiles[2]);
    if (x < 0) {
        k.streams = 3;
        k.region = 0;
        k.at = t * per;
        pages = s.pages[0];
    } else if (s.split) {
        k.streams = 1 << (x & 1);
        k.region = 1;
        k.at = x * per;
        pages = s.pages[1];
    } else {
        const int st = x < m ? x & 1 : s.tiles[1] > s.tiles[2] ? 0 : 1;
        k.streams = 1 << st;
        k.region = 1 + st;
        k.at = (x < m ? x >> 1 : (m >> 1) + x - m) * per;
        pages = st ? s.pages[2] : s.pages[1];
    }
    k.np = min(per, pages - k.at);
    return k;
}
__device__ __forceinline__ int tiles_of(const TileSegment& s) { return s.tiles[0] + s.tiles[1] + s.tiles[2]; }
// tiles that begin before place x of the item's line (a tile of both streams costs 2, else 1)
__device__ __forceinline__ int tiles_before(const TileSegment& s, long long x) {
    const long long both = 2LL * s.tiles[0];
    return (int)min((long long)tiles_of(s), x <= 0 ? 0 : x <= both ? (x + 1) / 2 : s.tiles[0] + (x - both));
}
__device__ __forceinline__ long long begin_of(const TileSegment& s, int t) {
    return t <= s.tiles[0] ? 2LL * t : 2LL * s.tiles[0] + (t - s.tiles[0]);
}

// tiles of stream st among the first n
__device__ __forceinline__ int stream_tiles(const TileSegment& s, int st, int n) {
    const int both = min(n, s.tiles[0]), x = n - both, m = s.split ? x : min(x, 2 * min(s.tiles[1], s.tiles[2]));
    return both + (st ? m / 2 : (m + 1) / 2) + (x > m && (s.tiles[1] > s.tiles[2] ? 0 : 1) == st ? x - m : 0);
}

// What the join has to know of an item that a run is not the first to work on.
struct CutRecord {
    int live, h, first, toks0, toks1, split, c0, c1;
    int pad[4];
};
static_assert(sizeof(CutRecord) == 48, "");

__global__ void __launch_bounds__(kTcThreads, 1)
    page_tiles_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                      const __grid_constant__ CUtensorMap mv, const __grid_constant__ PageAttnArgs a) {
    extern __shared__ uint8_t raw_smem[];
    const uint32_t raw = smem_addr(raw_smem), base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = raw_smem + (base - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t full = base + kOffBars, empty = full + 8 * kTileStages, q_full = empty + 8 * kTileStages, q_empty = q_full + 16;
    const uint32_t s_full = q_empty + 16, p_full = s_full + 16, o_full = p_full + 16, tail = o_full + 16;
    const uint32_t drain = tail + 8, m_full = drain + 8, m_free = m_full + 8, seg_full = m_free + 8, seg_empty = seg_full + 8 * kQueue;
    const uint32_t note_full = seg_empty + 8 * kQueue;
    volatile uint32_t* s_tmem = reinterpret_cast<volatile uint32_t*>(gbase + kOffSeg + kQueue * kSegBytes);
    const int per = kTileKeys >> a.page_shift;  // pages of a key tile
    int bad = 0;

    if (tid == 0) {
        for (int i = 0; i < kTileStages; ++i) {
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
        mbar_init(m_full, 4);
        mbar_init(m_free, 4);
        for (int i = 0; i < kQueue; ++i) {
            mbar_init(seg_full + 8 * i, 1);
            mbar_init(seg_empty + 8 * i, kSegReaders);
        }
        for (int i = 0; i < kNotes; ++i) mbar_init(note_full + 8 * i, 1);
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
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    bool failed = false;
    TileSegment s;
    // A wait that runs out sets its warp's `failed`.  From there on the warp arms no barrier, starts no copy and writes no segment
    // (a stage or a queue place may still be in use), sees what it has in flight to its end and stops; the others' waits then run
    // out in turn.  The results are undefined, the error word says so, and the next call finds everything as it should be.
    auto wait = [&](uint32_t bar, uint32_t parity) { mbar_wait_fast(bar, parity, failed, a.polls); };

    volatile uint32_t* notes = reinterpret_cast<volatile uint32_t*>(gbase + kOffNote);
    // the next segment of the queue, read by a warp
    auto receive = [&](Ring<kQueue>& q) {
        wait(seg_full + 8 * q.stage, q.phase);
        failed = __any_sync(kFull, failed);  // (a warp stays together)
        if (failed) return false;
        const int4* src = reinterpret_cast<const int4*>(gbase + kOffSeg + q.stage * kSegBytes);
        int4* dst = reinterpret_cast<int4*>(&s);
#pragma unroll
        for (int i = 0; i < (int)(sizeof(TileSegment) / 16); ++i) dst[i] = src[i];
        __syncwarp();
        if (lane == 0) mbar_arrive(seg_empty + 8 * q.stage);
        q.advance();
        return s.live != 0;
    };

    // (128 x 168 x 3 registers at launch: 2 x 128 x 176 + 128 x 152)
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 152;\n");
        if (warp == 8) {
            // ---- the run's segments, and the key tiles' pages (lane i: page i of the tile) ----
            Ring<kKeyStages> kr{0, 1};
            Ring<kQueue> queue{0, 1};  // (a fresh barrier lets a wait for parity 1 pass: the stages start empty)
            const uint32_t page_bytes = (uint32_t)a.page_n * 256u;
            const int W2 = 2 * a.words;
            int note_at = 0;
            // where in a note the lane's two words of a tile's masks go (word i of page p from p W2 + i)
            const int mask0 = kNoteMasks + 8 * (lane % W2) + lane / W2, mask1 = kNoteMasks + 8 * ((lane + 32) % W2) + (lane + 32) / W2;
            auto note = [&](uint32_t what) {  // a tile without keys: a word to the MMA thread alone
                wait(empty + 8 * kr.stage, kr.phase);
                failed = __any_sync(kFull, failed);
                if (failed) return;
                if (lane == 0) {
                    notes[note_at * kNoteWords] = what;
                    mbar_arrive(note_full + 8 * note_at);
                    mbar_arrive(full + 8 * kr.stage);
                }
                __syncwarp();
                if (++note_at == kNotes) note_at = 0;
                kr.advance();
            };
            const int units = a.head->units, items = units * a.Hkv;
            long long total = 0;
            for (int i = lane; i < items; i += 32) total += a.count[i].w;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) total += __shfl_xor_sync(kFull, total, d);
            const int runs = (int)min((long long)a.runs, max(total / kRunLeast, 1LL)), c = blockIdx.x;
            const long long lo = c < runs ? total * c / runs : total, hi = c < runs ? total * (c + 1) / runs : total;
            CutRecord cut{};
            // the item that holds place lo
            int item = 0;
            long long at = 0;  // where it begins
            for (; item < items; item += 32) {
                const int w = item + lane < items ? a.count[item + lane].w : 0;
                int x = w;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int y = __shfl_up_sync(kFull, x, d);
                    if (lane >= d) x += y;
                }
                const int sum = __shfl_sync(kFull, x, 31);
                if (at + sum > lo) {
                    const int k = __popc(__ballot_sync(kFull, at + x <= lo));  // items of these 32 that end at or before lo
                    at += k ? __shfl_sync(kFull, x, k - 1) : 0;
                    item += k;
                    break;
                }
                at += sum;
            }
            auto send = [&] {
                wait(seg_empty + 8 * queue.stage, queue.phase);
                failed = __any_sync(kFull, failed);
                if (failed) return;
                if (lane == 0) {
                    *reinterpret_cast<TileSegment*>(gbase + kOffSeg + queue.stage * kSegBytes) = s;
                    mbar_arrive(seg_full + 8 * queue.stage);
                }
                __syncwarp();
                queue.advance();
            };
            for (; at < hi && item < items && !failed; ++item) {
                const int4 n = a.count[item];
                const int h = item / units;
                const Pair p = pair_of(a, item - h * units);
                s.live = 1;
                s.h = h;
                s.item = item;
                s.first = p.first;
                s.toks0 = p.toks[0];
                s.split = p.toks[1] == 0;
                s.toks1 = s.split ? s.toks0 : p.toks[1];
                s.held = p.held;
                s.ahead = p.ahead;
                s.pages[0] = n.x;
                s.pages[1] = n.y;
                s.pages[2] = n.z;
#pragma unroll
                for (int k = 0; k < 3; ++k) s.tiles[k] = (s.pages[k] + per - 1) / per;
                const int tiles = tiles_of(s);
                s.n0 = tiles_before(s, lo - at);
                s.n1 = tiles_before(s, hi - at);
                const bool begins = at >= lo;
                const long long begin = at;
                at += n.w;
                if (tiles == 0 ? !begins : s.n0 >= s.n1) continue;
                s.whole = s.n0 == 0 && s.n1 == tiles;
                s.slot = 2 * c + (s.n0 == 0);
                if (!s.whole && s.n0 > 0) {
                    const int c0 = (int)(((begin + 1) * runs - 1) / total);
                    cut = CutRecord{1, h, s.first, s.toks0, s.toks1, s.split, c0,
                                    (int)(((begin + begin_of(s, tiles - 1) + 1) * runs - 1) / total), {}};
                }
                send();
                if (tiles == 0) {  // (nobody may wait for a product that is due behind an item without a tile)
                    note(0);
                    continue;
                }
                int seen[2] = {0, 0};
                const int all[2] = {stream_tiles(s, 0, s.n1) - stream_tiles(s, 0, s.n0), stream_tiles(s, 1, s.n1) - stream_tiles(s, 1, s.n0)};
                const int first_sees = min(max(s.ahead + 1, 0), s.held);  // own tokens of the pair's first token
                // A tile's pages (lane i: page i) and masks are read one tile ahead.
                KeyTile k = key_tile(s, s.n0, per);
                int2 e = make_int2(0, 0);
                uint32_t m0 = 0, m1 = 0;
                auto look_up = [&](const KeyTile& u) {
                    const size_t to = ((size_t)item * 3 + u.region) * a.cap + u.at;
                    e = lane < u.np ? a.ent[to + lane] : make_int2(0, 0);
                    const uint32_t* m = a.mask + to * W2;
                    m0 = lane < u.np * W2 ? m[lane] : 0u;
                    m1 = lane + 32 < u.np * W2 ? m[lane + 32] : 0u;
                };
                look_up(k);
                for (int t = s.n0; t < s.n1 && !failed; ++t) {
                    const int np = k.np, streams = k.streams, lp = e.y;
                    const uint32_t w0 = m0, w1 = m1;
                    const int y = (e.x * a.Hkv + h) << a.page_shift;
                    int sees = a.page_n;  // tokens of the page that every row sees
                    if (lane < np) sees = lp < a.prefix_pages ? a.prefix_len - (lp << a.page_shift) : first_sees - ((lp - a.prefix_pages) << a.page_shift);
                    // (columns behind the tile's last page, where they share 32 with it, are looked at too)
                    const bool edge = __any_sync(kFull, sees < a.page_n) || ((np << a.page_shift) & 31);
                    if (t + 1 < s.n1) {
                        k = key_tile(s, t + 1, per);
                        look_up(k);
                    }
                    uint32_t what = (uint32_t)streams | (uint32_t)((np << a.page_shift) >> 4) << kNoteGroups;
#pragma unroll
                    for (int st = 0; st < 2; ++st)
                        if ((streams >> st) & 1) {
                            if (seen[st] == 0) what |= kNoteFirst << st;
                            if (++seen[st] == all[st]) what |= kNoteLast << st;
                        }
                    const uint32_t stage = base + kr.stage * kTileBytes, bar = full + 8 * kr.stage;
                    wait(empty + 8 * kr.stage, kr.phase);
                    failed = __any_sync(kFull, failed);
                    if (failed) break;
                    // (the copies first: they take longest, each some 150 cycles of the warp's and then its way)
                    if (lane == 0) mbar_expect_tx(bar, np * page_bytes);
                    __syncwarp();
                    if (lane < np) tma_4d(stage + lane * page_bytes, &mk, 0, 0, 0, y >> 3, bar);
                    volatile uint32_t* to = notes + note_at * kNoteWords;
                    if (lane < np) to[kNotePages + lane] = lp;
                    if (lane < np * W2) to[mask0] = w0;
                    if (lane + 32 < np * W2) to[mask1] = w1;
                    if (lane == 0) {
                        to[0] = what;
                        to[1] = np | (edge ? 256u : 0u);
                    }
                    warp_arrive(note_full + 8 * note_at);
                    if (++note_at == kNotes) note_at = 0;
                    kr.advance();
                    failed |= (a.fault & HSQ_FAULT_WAIT_LOAD) != 0;
                }
            }
            note(kNoteEnd);
            s.live = 0;
            send();
            if (lane == 0) *reinterpret_cast<CutRecord*>(a.cut + 3 * c) = cut;
            if (failed)  // see the copies in flight land before the CTA ends
                for (int i = 0; i < kKeyStages; ++i) mbar_wait(full + 8 * i, kr.phase ^ (i < (int)kr.stage ? 1u : 0u), 1 << 12);
        } else if (warp == 9 && elect_one()) {
            // ---- MMAs, one thread ----
            // Key tile by key tile as the notes say.  Key tile g is in key stage g mod 3 and value stage g mod 2.  A stream's product
            // with the values of its last tile is due until its next S is issued, or until it is two tiles behind, when
            // its value stage is needed again.
            constexpr uint32_t idO = idesc_bf16_f32_bmn(128, 128);
            Ring<kKeyStages> kr{0, 0};
            uint32_t q_par = 0, p_par = 0;  // a bit for each stream
            // 0: none; else 1 | its note's word from bit 8 on | behind the segment's first (2) | its last (4); and the tile's number
            uint32_t due0 = 0, due1 = 0, at0 = 0, at1 = 0;
            uint32_t users = 0;  // bit i: the tile in value stage i has two products to serve, one is still to come
            uint32_t slot = 0, note_par = 0;
            auto scores = [&](int st, uint32_t g16) {  // S = Q K^T
                const uint32_t dS = tmem + 128 * st, idS = idesc_bf16_f32(128, 16 * g16);
                const uint64_t dq = sw128_desc(base + kOffQ + st * kTileBytes), dk = sw128_desc(base + kr.stage * kTileBytes, kGroupBytes);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t q = ((k >> 2) * kHalfBytes + (k & 3) * 32) >> 4, o = ((k >> 2) * kGroupHalf + (k & 3) * 32) >> 4;
                    mma_bf16(dS, dq + q, dk + o, idS, k > 0);
                }
                mma_commit(s_full + 8 * st);
            };
            auto whole_product = [&](int st, uint32_t v) {  // O += P V of a whole tile, not the stream's first
                const uint32_t pa = tmem + 128 * st, dO = pa + 256;
                const uint64_t dv = sw128_mn_desc(base + (kKeyStages + v) * kTileBytes, kGroupHalf, kGroupBytes);
                wait(p_full + 8 * st, (p_par >> st) & 1);
                p_par ^= 1u << st;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < 8; ++k) mma_bf16_ts(dO, pa + 8 * k, dv + k * (2 * kGroupBytes >> 4), idO, 1);
            };
            // The next tile's note, where it is there already: looked for while the pipe works off a product.
            bool peeked = false;
            uint32_t next = 0;
            auto peek = [&] {
                uint32_t done;
                asm volatile(
                    "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
                    : "=r"(done)
                    : "r"(note_full + 8 * slot), "r"(note_par)
                    : "memory");
                peeked = done != 0;
                if (peeked) next = notes[slot * kNoteWords];
            };
            auto settle = [&](int st, uint32_t& due, uint32_t at) {  // O += P V of the stream's tile that is due
                const uint32_t v = at & 1, stage = kKeyStages + v, g16 = due >> 8, more = (due >> 1) & 1;
                const uint32_t pa = tmem + 128 * st, dO = pa + 256;
                const uint64_t dv = sw128_mn_desc(base + stage * kTileBytes, kGroupHalf, kGroupBytes);
                wait(full + 8 * stage, (at >> 1) & 1);
                wait(p_full + 8 * st, (p_par >> st) & 1);
                if (__builtin_expect(failed, 0)) return;
                p_par ^= 1u << st;
                tc_fence_after();
                if (g16 == 8) {
                    mma_bf16_ts(dO, pa, dv, idO, more);
#pragma unroll
                    for (int k = 1; k < 8; ++k) mma_bf16_ts(dO, pa + 8 * k, dv + k * (2 * kGroupBytes >> 4), idO, 1);
                } else {
#pragma unroll 1
                    for (uint32_t k = 0; k < g16; ++k) mma_bf16_ts(dO, pa + 8 * k, dv + k * (2 * kGroupBytes >> 4), idO, more | (k > 0));
                }
                if (!((users >> v) & 1)) mma_commit(empty + 8 * stage);
                users &= ~(1u << v);
                if (due & 4) mma_commit(o_full + 8 * st);
                due = 0;
            };
#pragma unroll 1
            for (uint32_t g = 0;; ++g) {
                if (!peeked) {
                    wait(note_full + 8 * slot, note_par);
                    next = notes[slot * kNoteWords];
                }
                peeked = false;
                const uint32_t what = next;
                if (++slot == kNotes) {
                    slot = 0;
                    note_par ^= 1;
                }
                if (__builtin_expect(failed, 0)) break;
                // What most steps are, in straight code with constant operands (the tensor pipe holds but one or two MMAs more than
                // the one it works on, so what the thread does in between shows): whole tiles, each stream's product of the tile
                // before and S of this one.
                constexpr uint32_t kWhole = 8u << kNoteGroups, kWholeDue = kWhole | 3u;
                if (due0 == kWholeDue && due1 == kWholeDue) {
                    if (what == (kWhole | 3u) && at0 == at1) {  // (then both are due of tile g - 1)
                        wait(full + 8 * (kKeyStages + ((g - 1) & 1)), ((g - 1) >> 1) & 1);
                        whole_product(0, (g - 1) & 1);
                        wait(full + 8 * kr.stage, kr.phase);
                        scores(0, 8);
                        whole_product(1, (g - 1) & 1);
                        if (__builtin_expect(failed, 0)) break;
                        mma_commit(empty + 8 * (kKeyStages + ((g - 1) & 1)));
                        peek();
                        scores(1, 8);
                        mma_commit(empty + 8 * kr.stage);
                        users = 1u << (g & 1);
                        at0 = at1 = g;
                        kr.advance();
                        continue;
                    }
                    if (what == (kWhole | 1u) && at0 + 2 == g && at1 + 1 == g && users == 0) {
                        wait(full + 8 * (kKeyStages + (g & 1)), ((g - 2) >> 1) & 1);
                        whole_product(0, g & 1);
                        wait(full + 8 * kr.stage, kr.phase);
                        if (__builtin_expect(failed, 0)) break;
                        mma_commit(empty + 8 * (kKeyStages + (g & 1)));
                        peek();
                        scores(0, 8);
                        mma_commit(empty + 8 * kr.stage);
                        at0 = g;
                        kr.advance();
                        continue;
                    }
                    if (what == (kWhole | 2u) && at1 + 2 == g && at0 + 1 == g && users == 0) {
                        wait(full + 8 * (kKeyStages + (g & 1)), ((g - 2) >> 1) & 1);
                        whole_product(1, g & 1);
                        wait(full + 8 * kr.stage, kr.phase);
                        if (__builtin_expect(failed, 0)) break;
                        mma_commit(empty + 8 * (kKeyStages + (g & 1)));
                        peek();
                        scores(1, 8);
                        mma_commit(empty + 8 * kr.stage);
                        at1 = g;
                        kr.advance();
                        continue;
                    }
                }
                wait(full + 8 * kr.stage, kr.phase);
                if (__builtin_expect(failed, 0)) break;
                const bool flush = (what & kNoteStreams) == 0;
                // (the older first: a stream whose softmax has still to join the other's part takes up no new tile before)
                if (due1 && (g - at1 >= 2 || (flush && due0 && (int)(at1 - at0) < 0))) settle(1, due1, at1);
                if (due0 && ((what & 1) || flush || g - at0 >= 2)) settle(0, due0, at0);
                if (__builtin_expect(failed, 0)) break;
                if (what & 1) {
                    if (what & kNoteFirst) {
                        wait(q_full, q_par & 1);
                        q_par ^= 1;
                    }
                    if (__builtin_expect(failed, 0)) break;
                    scores(0, what >> kNoteGroups);
                    if (what & kNoteLast) mma_commit(q_empty);
                    due0 = 1u | (what & kNoteFirst ? 0u : 2u) | (what & kNoteLast ? 4u : 0u) | (what & ~255u);
                    at0 = g;
                }
                if (due1 && ((what & 2) || flush)) settle(1, due1, at1);
                if (__builtin_expect(failed, 0)) break;
                if (what & 2) {
                    if (what & (kNoteFirst << 1)) {
                        wait(q_full + 8, (q_par >> 1) & 1);
                        q_par ^= 2;
                    }
                    if (__builtin_expect(failed, 0)) break;
                    scores(1, what >> kNoteGroups);
                    if (what & (kNoteLast << 1)) mma_commit(q_empty + 8);
                    due1 = 1u | (what & (kNoteFirst << 1) ? 0u : 2u) | (what & (kNoteLast << 1) ? 4u : 0u) | (what & ~255u);
                    at1 = g;
                }
                // (the value stage's tile of two ago has served: what was due from it has been issued)
                if ((what & kNoteStreams) == 3) users |= 1u << (g & 1);
                // (after a wait that ran out no stage is handed back: its copy may still be under way)
                if (what & kNoteEnd) break;
                mma_commit(empty + 8 * kr.stage);
                if (flush) {  // (its value stage is handed back only once it has been taken, or the stage's phases would run ahead)
                    wait(full + 8 * (kKeyStages + (g & 1)), (g >> 1) & 1);
                    if (__builtin_expect(failed, 0)) break;
                    mma_commit(empty + 8 * (kKeyStages + (g & 1)));
                }
                kr.advance();
                failed |= (a.fault & HSQ_FAULT_WAIT_MMA) != 0;
            }
            if (failed) {  // what is in flight ends before its operands' and results' memory is given up
                mma_commit(drain);
                mbar_wait(drain, 0, 1 << 12);
            }
        } else if (warp == 10) {
            // ---- queries of the segments' streams ----
            Ring<kQueue> queue{0, 0};
            uint32_t q_par = 3;  // (the buffers start empty)
            const uint32_t q_bytes = (uint32_t)a.tpt * a.r * 256u;
            while (receive(queue)) {
#pragma unroll 1
                for (int st = 0; st < 2; ++st) {
                    if (stream_tiles(s, st, s.n1) == stream_tiles(s, st, s.n0)) continue;
                    const uint32_t dst = base + kOffQ + st * kTileBytes, bar = q_full + 8 * st;
                    wait(q_empty + 8 * st, (q_par >> st) & 1);
                    if (st) failed |= (a.fault & HSQ_FAULT_WAIT_QUERY) != 0;
                    failed = __any_sync(kFull, failed);
                    if (failed) break;
                    q_par ^= 1u << st;
                    if (lane == 0) {
                        const int row = s.first + (st && !s.split ? a.tpt : 0);
                        mbar_expect_tx(bar, q_bytes);
                        tma_3d(dst, &mq, 0, s.h * a.r, row, bar);
                        tma_3d(dst + kHalfBytes, &mq, 64, s.h * a.r, row, bar);
                    }
                    __syncwarp();
                }
                if (failed) break;
            }
            if (failed)  // query tiles in flight land before the CTA ends
                for (int st = 0; st < 2; ++st) mbar_wait(q_full + 8 * st, (q_par >> st) & 1, 1 << 12);
        } else if (warp == 11) {
            // ---- the value tiles' pages.  (By the keys' warp, in turn with them, the keys waited for the values' stages, one product
            // later than their own need: a chunk of 2048 over 32K 598 us instead of 469 at the time.) ----
            Ring<kValueStages> vr{0, 1};
            Ring<kQueue> queue{0, 0};
            uint32_t tail_par = 0;
            bool tail_due = false;
            const uint32_t page_bytes = (uint32_t)a.page_n * 256u;
            while (receive(queue) && !failed) {
                auto look_up = [&](const KeyTile& u) {
                    return lane < u.np ? a.ent[((size_t)s.item * 3 + u.region) * a.cap + u.at + lane] : make_int2(0, 0);
                };
                KeyTile k = key_tile(s, s.n0, per);
                int2 e = make_int2(0, 0);
                if (s.n0 < s.n1) e = look_up(k);
                for (int t = s.n0; t < max(s.n1, s.n0 + 1); ++t) {
                    const uint32_t slot = kKeyStages + vr.stage, stage = base + slot * kTileBytes, bar = full + 8 * slot;
                    const bool none = s.n0 == s.n1;  // (an item without a tile takes a stage too, as its note does)
                    const int np = none ? 0 : k.np, y = (e.x * a.Hkv + s.h) << a.page_shift;
                    int tokens = a.page_n;  // of the page
                    if (lane < np) tokens = e.y < a.prefix_pages ? a.prefix_len - (e.y << a.page_shift) : s.held - ((e.y - a.prefix_pages) << a.page_shift);
                    // Rows of values that no token has hold whatever the page holds; their weights are 0, so they have to
                    // be finite.  Cleared here before the tile is handed over.
                    const unsigned ends = __ballot_sync(kFull, tokens < a.page_n);
                    if (t + 1 < s.n1) {
                        k = key_tile(s, t + 1, per);
                        e = look_up(k);
                    }
                    wait(empty + 8 * slot, vr.phase);
                    failed = __any_sync(kFull, failed);
                    if (failed) break;
                    const uint32_t lands = ends ? tail : bar;
                    if (lane == 0) {
                        if (none) mbar_arrive(bar);
                        else mbar_expect_tx(lands, np * page_bytes);
                    }
                    __syncwarp();
                    if (lane < np) tma_4d(stage + lane * page_bytes, &mv, 0, 0, 0, y >> 3, lands);
                    if (ends) {
                        wait(tail, tail_par);
                        failed = __any_sync(kFull, failed);
                        if (failed) {
                            tail_due = true;
                            break;
                        }
                        tail_par ^= 1;
                        for (unsigned left = ends; left; left &= left - 1) {
                            const int i = __ffs(left) - 1, have = max(__shfl_sync(kFull, tokens, i), 0);
                            const int row0 = (i << a.page_shift) + have, z = (a.page_n - have) * 16;  // 16-byte chunks of both halves
                            for (int x = lane; x < z; x += 32)
                                *reinterpret_cast<uint4*>(gbase + (stage - base) + ((row0 + (x >> 4)) >> 3) * kGroupBytes + ((x >> 3) & 1) * kGroupHalf +
                                                          ((row0 + (x >> 4)) & 7) * 128 + (x & 7) * 16) = make_uint4(0, 0, 0, 0);
                        }
                        fence_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar);
                    }
                    vr.advance();
                }
            }
            if (failed) {  // see the copies in flight land before the CTA ends
                for (int i = 0; i < kValueStages; ++i)
                    mbar_wait(full + 8 * (kKeyStages + i), vr.phase ^ (i < (int)vr.stage ? 1u : 0u), 1 << 12);
                if (tail_due) mbar_wait(tail, tail_par, 1 << 12);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 176;\n");
        // ---- softmax: thread = row of its stream's tile ----
        const int st = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t tS = tmem + lanes + 128 * st, tO = tmem + lanes + 256 + 128 * st;
        uint32_t s_par = 0, o_par = 0, m_par = 0;
        uint32_t tiles_done = 0;  // of the segments before
        Ring<kQueue> queue{0, 0};
        const int row_token = row / a.r, word = (32 * (warp & 3) / a.r) >> 5;  // (a warp's tokens share a word of the masks)
        while (receive(queue)) {
            const int toks = st ? s.toks1 : s.toks0, tile = st && !s.split ? 1 : 0, t0 = tile ? a.tpt : 0;
            const bool live = row_token < toks;
            const bool idle = 32 * (warp & 3) >= toks * a.r;  // (warp-uniform) no row of this warp in use
            const int seen = min(max(s.ahead + t0 + row_token + 1, 0), s.held);
            const int mine = stream_tiles(s, st, s.n1) - stream_tiles(s, st, s.n0);
            const int alternate = s.split ? 1 << 30 : 2 * min(s.tiles[1], s.tiles[2]);
            float m = -INFINITY, l = 0.f;
            int n = s.n0;
#pragma unroll 1
            for (int done = 0; done < mine; ++done, ++n) {
                const int x = n - s.tiles[0];  // behind the tiles of both streams they take turns as long as both have some
                if (x >= 0 && x < alternate) n += (x & 1) != st;
                const uint32_t at = tiles_done + n - s.n0, slot = at % kNotes;
                const volatile uint32_t* note = notes + slot * kNoteWords;
                wait(note_full + 8 * slot, (at / kNotes) & 1);
                const uint32_t about = note[1];
                const int np = min((int)(about & 255), per);  // (behind a wait that ran out the note may be none: not past the tensor memory)
                uint32_t gm = 0;  // the groups of 16 keys that this row takes, and those that any row of the warp takes
                {
                    uint32_t w[8];  // (behind the tile's last page: of some tile before)
                    const uint32_t from = base + kOffNote + 4 * (slot * kNoteWords + kNoteMasks + 8 * (tile * a.words + word));
                    asm volatile("ld.volatile.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(from) : "memory");
                    asm volatile("ld.volatile.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7]) : "r"(from + 16) : "memory");
                    const int per_page = a.page_n >> 4;
                    uint32_t one = (1u << per_page) - 1u;  // a page's groups
#pragma unroll
                    for (int i = 0; i < 8; ++i, one <<= per_page) gm |= (w[i] >> (row_token & 31)) & 1u ? one : 0u;
                    gm &= live ? (1u << (np * per_page)) - 1u : 0u;
                }
                const uint32_t wm = __reduce_or_sync(kFull, gm);
                wait(s_full + 8 * st, s_par);
                s_par ^= 1;
                if (!idle) {
                    tc_fence_after();
                    float t;
                    uint32_t p[2][32];
                    // A page that the row does not take is hidden by adding -inf to its logits.  That fails where one of them is no
                    // number, or +inf; it shows in the sum, and then such pages are hidden in S first.  (The way back to it costs
                    // every tile some instructions: a chunk of 2048 over 32K 385 us in place of 381.)
                    bool hide = about >> 8, hidden = hide;
                    bool look = __any_sync(kFull, gm != 0 && m == -INFINITY);
#pragma unroll 1
                    while (true) {
                        if (hide) {
                            // pages that end inside a row's sight, pages that it does not take and rows of no token: hidden in S
                            // itself, so that the code below knows whole pages of numbers only
#pragma unroll 1
                            for (int c0 = 0; c0 < (np << a.page_shift); c0 += 32) {
                                float x[32];
                                tmem_ld32(tS + c0, x);
#pragma unroll
                                for (int hf = 0; hf < 2; ++hf) {
                                    const int c = c0 + 16 * hf, i = c >> a.page_shift;
                                    const int p = note[kNotePages + (i & 7)];
                                    const int lim = p < a.prefix_pages ? a.prefix_len - (p << a.page_shift) : seen - ((p - a.prefix_pages) << a.page_shift);
                                    const int keys = (gm >> (c >> 4)) & 1u ? lim - (c & (a.page_n - 1)) : 0;
#pragma unroll
                                    for (int e = 0; e < 16; ++e)
                                        if (e >= keys) x[16 * hf + e] = -INFINITY;
                                }
                                tmem_st32(tS + c0, x);
                            }
                        }
                        if (look) {
                            // The running maximum need not be one: any m that keeps the sums in range gives the same result, p and
                            // l being floating point.  So it is looked for in a row's first tile and where the tile's sum shows
                            // that the logits have outgrown m by far.
                            float mn = m;
#pragma unroll 1
                            for (int c0 = 0; c0 < (np << a.page_shift); c0 += 32) {
                                if (!((wm >> (c0 >> 4)) & 3u)) continue;
                                const bool h0 = (gm >> (c0 >> 4)) & 1u, h1 = (gm >> (c0 >> 4)) & 2u;
                                float x[32], m0 = -INFINITY, m1 = -INFINITY;
                                tmem_ld32(tS + c0, x);
#pragma unroll
                                for (int c = 0; c < 16; ++c) {
                                    m0 = fmaxf(m0, x[c]);
                                    m1 = fmaxf(m1, x[16 + c]);
                                }
                                if (h0) mn = fmaxf(mn, m0);
                                if (h1) mn = fmaxf(mn, m1);
                            }
                            const float alpha = m == -INFINITY ? 0.f : ex2_approx((m - mn) * kLogitScaleLog2);
                            m = mn;
                            l *= alpha;
                            if (done > 0) {  // O holds the tiles before (S of this tile follows their P V)
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
                        const uint64_t scale2 = pack2(kLogitScaleLog2, kLogitScaleLog2);
                        uint64_t l2[2] = {0, 0};
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t* pq = p[q >> 1] + 16 * (q & 1);
                            if ((wm >> (2 * q)) & 3u) {
                                float x[32];
                                tmem_ld32(tS + 32 * q, x);
                                const float f0 = (gm >> (2 * q)) & 1u ? off : -INFINITY, f1 = (gm >> (2 * q)) & 2u ? off : -INFINITY;
#pragma unroll
                                for (int c = 0; c < 32; c += 2) {
                                    const float f = c < 16 ? f0 : f1;
                                    float e0, e1;
                                    unpack2(fma2(pack2(x[c], x[c + 1]), scale2, pack2(f, f)), e0, e1);
                                    e0 = ex2_approx(e0);
                                    e1 = ex2_approx(e1);
                                    l2[(c >> 1) & 1] = add2(l2[(c >> 1) & 1], pack2(e0, e1));
                                    pq[c >> 1] = pack_bf16(e0, e1);
                                }
                            } else {
#pragma unroll
                                for (int c = 0; c < 16; ++c) pq[c] = 0u;
                            }
                        }
                        float lo, hi;
                        unpack2(add2(l2[0], l2[1]), lo, hi);
                        t = lo + hi;
                        if (!__any_sync(kFull, live && !(t < kTileSum))) break;  // (rows of no token hold anything)
                        hide = !hidden && __any_sync(kFull, live && t != t);
                        if (!hide && (look || !__any_sync(kFull, live && t >= kTileSum))) break;
                        hidden |= hide;
                        look = !hide;
                    }
                    tmem_st32_nowait(tS, p[0]);
                    tmem_st32_nowait(tS + 32, p[1]);
                    l += t;
                    tmem_st_wait();
                    tc_fence_before();
                }
                warp_arrive(p_full + 8 * st);
            }
            tiles_done += max(s.n1 - s.n0, 1);  // (an item without a tile has a note too)
            if (mine > 0) {
                wait(o_full + 8 * st, o_par);
                o_par ^= 1;
            }
            failed |= (a.fault & HSQ_FAULT_WAIT_SOFTMAX) != 0;
            failed = __any_sync(kFull, failed);
            if (failed) break;
            tc_fence_after();
            bool other = false;  // a lone tile: the second stream's share joins the first's
            float w0 = 1.f, w1 = 0.f;
            if (s.split) {
                float2* ml = a.pair_ml + (size_t)blockIdx.x * kTileRows + row;
                if (st) {
                    __stcg(ml, make_float2(m, l));
                    __threadfence_block();
                    tc_fence_before();
                    warp_arrive(m_full);
                    wait(m_free, m_par);  // (O is read, and the sums)
                    m_par ^= 1;
                    failed = __any_sync(kFull, failed);
                    if (failed) break;
                    tc_fence_after();
                    continue;
                }
                wait(m_full, m_par);
                m_par ^= 1;
                failed = __any_sync(kFull, failed);
                if (failed) break;
                tc_fence_after();
                other = stream_tiles(s, 1, s.n1) > stream_tiles(s, 1, s.n0);
                const float2 x = __ldcg(ml);
                const float M = fmaxf(m, x.x);
                w0 = m == -INFINITY && l == 0.f ? 0.f : ex2_approx((m - M) * kLogitScaleLog2);
                w1 = x.x == -INFINITY && x.y == 0.f ? 0.f : ex2_approx((x.x - M) * kLogitScaleLog2);
                l = l * w0 + x.y * w1;
                m = M;
            }
            const bool cut = !s.whole;
            const float inv = cut ? 1.f : l == 0.f ? 0.f : 1.0f / l;  // (a sum that is not a number shows in the result)
            const size_t to = (size_t)(s.first + t0 + row_token) * a.Hq + s.h * a.r + (row - row_token * a.r);
            const size_t part = ((size_t)s.slot * 2 + st) * kTileRows;
            if (live) {
                if (cut) a.part_ml[part + row] = make_float2(m, l);
                else if (a.lse) a.lse[to] = l == 0.f ? -INFINITY : m * kRsqrtD + logf(l);
            }
            if (!idle) {
#pragma unroll 1
                for (int c0 = 0; c0 < 128; c0 += 32) {
                    float o[32], y[32];
                    if (mine > 0) tmem_ld32(tO + c0, o);
                    if (other) {
                        tmem_ld32(tO + 128 + c0, y);
#pragma unroll
                        for (int c = 0; c < 32; ++c) o[c] = fmaf(y[c], w1, mine > 0 ? o[c] * w0 : 0.f);
                    } else if (s.split) {
#pragma unroll
                        for (int c = 0; c < 32; ++c) o[c] *= w0;
                    }
                    if (!live) continue;
                    if (cut) {  // dims apart, rows side by side, so that a warp writes whole lines
                        if (mine > 0 || other) {
#pragma unroll
                            for (int c = 0; c < 32; ++c) a.part_o[part * 128 + (size_t)(c0 + c) * kTileRows + row] = o[c];
                        }
                    } else {
                        uint4* dst = reinterpret_cast<uint4*>(a.out + to * 128 + c0);
#pragma unroll
                        for (int c = 0; c < 32; c += 8)
                            dst[c >> 3] = l == 0.f ? make_uint4(0, 0, 0, 0)
                                                   : make_uint4(pack_bf16(o[c] * inv, o[c + 1] * inv), pack_bf16(o[c + 2] * inv, o[c + 3] * inv),
                                                                pack_bf16(o[c + 4] * inv, o[c + 5] * inv), pack_bf16(o[c + 6] * inv, o[c + 7] * inv));
                    }
                }
            }
            tc_fence_before();  // (O has been read: the next segment's first P releases it)
            if (s.split) warp_arrive(m_free);
        }
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

// Join.  The runs of a cut item behind its first deal its dims among them, in eighths; a CTA takes a run's share of one tile's 32 rows
// (lane = row).  A warp has 16 dims; where the share has fewer eighths than the CTA warps, they deal the parts among them too (one
// warp after the other, eight items in 19 parts each took 32 us).
__global__ void __launch_bounds__(256) page_join_kernel(const __grid_constant__ PageAttnArgs a) {
    __shared__ float s_o[8][32][17];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, run = blockIdx.x >> 3, st = blockIdx.x & 1;
    const int quarter = (blockIdx.x >> 1) & 3, row = 32 * quarter + lane;
    const CutRecord c = *reinterpret_cast<const CutRecord*>(a.cut + 3 * run);
    if (!c.live || (st && c.split)) return;
    const int rows = (st ? c.toks1 : c.toks0) * a.r;
    if (32 * quarter >= rows) return;
    const int shares = min(c.c1 - c.c0, 8), share = run - c.c0 - 1;
    if (share >= shares) return;
    const int w0 = 8 * share / shares, eighths = 8 * (share + 1) / shares - w0, groups = 8 / eighths;
    const int mine = warp % eighths, group = warp / eighths;  // eighth of the share, group of parts (the last warps may have none)
    const bool live = row < rows;
    const int first = c.first + (st ? a.tpt : 0);
    float M = -INFINITY, L = 0.f, o[16];
#pragma unroll
    for (int d = 0; d < 16; ++d) o[d] = 0.f;
    if (live && group < groups) {
        auto slot_of = [&](int k) { return ((size_t)(k == c.c0 ? 2 * k + 1 : 2 * k) * 2 + st) * kTileRows + row; };
        for (int k0 = c.c0; k0 <= c.c1; k0 += 8) {
            float2 v[8];
            float top = M;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = k0 + i <= c.c1 ? a.part_ml[slot_of(k0 + i)] : make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, v[i].x);
            if (L != 0.f) L *= ex2_approx((M - top) * kLogitScaleLog2);
            M = top;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (v[i].y != 0.f) L = fmaf(v[i].y, ex2_approx((v[i].x - M) * kLogitScaleLog2), L);
        }
        for (int k = c.c0 + group; k <= c.c1; k += 2 * groups) {
            float x[2][16];
            float2 ml[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const size_t at = slot_of(min(k + i * groups, c.c1));
                const float* src = a.part_o + (at - row) * 128 + (size_t)16 * (w0 + mine) * kTileRows + row;
                ml[i] = k + i * groups <= c.c1 ? a.part_ml[at] : make_float2(-INFINITY, 0.f);
#pragma unroll
                for (int d = 0; d < 16; ++d) x[i][d] = src[(size_t)d * kTileRows];
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float w = ex2_approx((ml[i].x - M) * kLogitScaleLog2);
                if (ml[i].y != 0.f) {  // (else nothing was written)
#pragma unroll
                    for (int d = 0; d < 16; ++d) o[d] = fmaf(x[i][d], w, o[d]);
                }
            }
        }
    }
    const float inv = L == 0.f ? 0.f : 1.0f / L;
#pragma unroll
    for (int d = 0; d < 16; ++d) s_o[warp][lane][d] = o[d] * inv;
    if (live && warp == 0 && w0 == 0 && a.lse)
        a.lse[(size_t)(first + row / a.r) * a.Hq + c.h * a.r + row % a.r] = L == 0.f ? -INFINITY : M * kRsqrtD + logf(L);
    __syncthreads();
    const int pairs = 8 * eighths;  // of dims
    for (int e = tid; e < 32 * pairs; e += 256) {
        const int i = e / pairs, y = 32 * quarter + i, d = 2 * (e - i * pairs), u = d >> 4;
        if (y >= rows) break;
        float y0 = 0.f, y1 = 0.f;
        for (int q = 0; q < groups; ++q) {
            y0 += s_o[q * eighths + u][i][d & 15];
            y1 += s_o[q * eighths + u][i][(d & 15) + 1];
        }
        const size_t to = (size_t)(first + y / a.r) * a.Hq + c.h * a.r + y % a.r;
        *reinterpret_cast<uint32_t*>(a.out + to * 128 + 16 * w0 + d) = pack_bf16(y0, y1);
    }
}

// CTAs of a cluster for units of some `keys` keys each where `slots` CTAs run at once: what a CTA costs, its share of the keys and
// what it costs beside them (in keys), times the CTAs a slot has (one at least).
int cluster_of(long long units, long long slots, long long keys, long long beside) {
    int best = 1;
    long long least = -1;
    for (int S = 1; S <= 8; ++S) {
        const long long cost = std::max(units * S, slots) * (beside + 16 * S + (keys + S - 1) / S);
        if (least < 0 || cost < least) {
            least = cost;
            best = S;
        }
    }
    return best;
}

// The workspace's pieces and their offsets.
struct Layout {
    size_t head, req, unit, short_row, count, ent, mask, part_o, part_ml, pair_ml, cut, bytes;
    int few, tpt, words, cap, runs, units, rows;
};

Layout layout_of(const hsq_ctx* ctx, int page_n, int rows, int B, int width, int prefix_len, int top, int max_new) {
    Layout x{};
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t here = at;
        at += (n + 255) / 256 * 256;
        return here;
    };
    const int r = ctx->r, Hkv = ctx->cfg.n_kv_heads;
    x.tpt = kTileRows / r;
    x.words = (x.tpt + 31) / 32;
    x.few = kFewColumns / r;
    x.runs = ctx->num_sms;
    x.head = take(256);
    if (max_new > x.few) {
        const int D = 2 * x.tpt;
        x.units = rows / D + 1 + std::min(B, rows / (x.few + 1));
        x.rows = (int)std::min<long long>(rows, (long long)B * x.few);
        x.cap = (int)std::min<long long>((prefix_len + page_n - 1) / page_n + (long long)width, (long long)x.tpt * top);
        const size_t items = (size_t)x.units * Hkv, lists = items * 3 * x.cap;
        x.req = take((size_t)B * 16);
        x.unit = take((size_t)x.units * 8);
        x.short_row = take((size_t)x.rows * 4);
        x.count = take(items * 16);
        x.ent = take(lists * 8);
        x.mask = take(lists * 8 * x.words);
        x.part_o = take((size_t)x.runs * 4 * kTileRows * 128 * 4);
        x.part_ml = take((size_t)x.runs * 4 * kTileRows * 8);
        x.pair_ml = take((size_t)x.runs * kTileRows * 8);
        x.cut = take((size_t)x.runs * 48);
    }
    x.bytes = at;
    return x;
}

}  // namespace

extern "C" {

hsq_status hsq_page_attn_workspace_size(const hsq_ctx* ctx, int page_n, int rows, int B, int width, int prefix_len,
                                        int top, int max_new, size_t* bytes) {
    if (!ctx || !bytes) return hsq::fail(nullptr, HSQ_ERR_INVALID, "ctx or bytes is NULL");
    const char* wrong = hsq::selection_shape_wrong(page_n, rows, B, width, prefix_len, top, max_new);
    if (wrong) return hsq::fail(nullptr, HSQ_ERR_INVALID, wrong);
    *bytes = layout_of(ctx, page_n, rows, B, width, prefix_len, top, max_new).bytes;
    return HSQ_OK;
}

hsq_status hsq_page_attn(hsq_ctx* ctx, const hsq_pages* pages, int rows, int B, int width, int prefix_len, int top,
                         int max_new, const void* q, const int32_t* q_start, const int32_t* lens, const int32_t* table,
                         const int32_t* prefix, const int32_t* sel, void* out, float* lse_opt, void* workspace,
                         size_t workspace_bytes, hsq_stream_t stream) {
    hsq_status st = hsq::check_pages(ctx, pages, true);
    if (st != HSQ_OK) return st;
    if (!q || !q_start || !lens || !table || !sel || !out || !workspace)
        return hsq::fail(ctx, HSQ_ERR_INVALID, "an argument of hsq_page_attn is NULL");
    const char* wrong = hsq::selection_shape_wrong(pages->page_n, rows, B, width, prefix_len, top, max_new);
    if (wrong) return hsq::fail(ctx, HSQ_ERR_INVALID, wrong);
    if (B > ctx->cfg.max_batch) return hsq::fail(ctx, HSQ_ERR_INVALID, "B above max_batch");
    if (prefix_len > 0 && !prefix) return hsq::fail(ctx, HSQ_ERR_INVALID, "prefix is NULL with prefix_len > 0");
    if (((uintptr_t)q | (uintptr_t)out) & 15u) return hsq::fail(ctx, HSQ_ERR_INVALID, "q and out must be 16-byte aligned");
    if ((uintptr_t)workspace & 255u) return hsq::fail(ctx, HSQ_ERR_INVALID, "workspace must be 256-byte aligned");
    const Layout x = layout_of(ctx, pages->page_n, rows, B, width, prefix_len, top, max_new);
    if (workspace_bytes < x.bytes)
        return hsq::fail(ctx, HSQ_ERR_INVALID, "workspace smaller than hsq_page_attn_workspace_size");
    const int Hq = ctx->cfg.n_q_heads, Hkv = ctx->cfg.n_kv_heads, P = pages->page_n, np = (prefix_len + P - 1) / P;
    if ((long long)rows * Hkv >= (1LL << 27)) return hsq::fail(ctx, HSQ_ERR_INVALID, "too many rows");
    const size_t q_bytes = (size_t)rows * Hq * 256, pool = (size_t)pages->n_pages * Hkv * P * 256;
    const hsq::Span ins[] = {{q, q_bytes}, {q_start, 4 * ((size_t)B + 1)}, {lens, 4 * (size_t)B}, {table, 4 * (size_t)B * width},
                             {prefix_len > 0 ? prefix : nullptr, 4 * (size_t)np}, {sel, (size_t)rows * Hkv * top * 4},
                             {pages->k, pool}, {pages->v, pool}};
    const hsq::Span outs[] = {{out, q_bytes}, {lse_opt, (size_t)rows * Hq * 4}, {workspace, x.bytes}};
    if (hsq::outputs_overlap(ins, outs))
        return hsq::fail(ctx, HSQ_ERR_INVALID, "an output or the workspace of hsq_page_attn overlaps another argument");
    if ((st = hsq::check_device(ctx)) != HSQ_OK) return st;
    PageAttnArgs a{};
    a.q = static_cast<const uint16_t*>(q);
    a.q_start = q_start; a.lens = lens; a.table = table; a.prefix = prefix; a.sel = sel;
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse_opt;
    a.rows = rows; a.B = B; a.width = width; a.prefix_len = prefix_len; a.prefix_pages = np; a.max_new = max_new;
    a.n_pages = pages->n_pages; a.page_n = P; a.page_shift = P == 16 ? 4 : P == 32 ? 5 : P == 64 ? 6 : 7;
    a.Hq = Hq; a.Hkv = Hkv; a.r = ctx->r; a.top = top;
    a.fault = (int)hsq::fault_mask() & (HSQ_FAULT_WAIT_LOAD | HSQ_FAULT_WAIT_MMA | HSQ_FAULT_WAIT_QUERY | HSQ_FAULT_WAIT_SOFTMAX | HSQ_FAULT_WAIT_FEW);
    a.polls = a.fault ? 1 << 8 : 1 << 18;  // (a poll that finds nothing takes 4 us: 1 ms, or a second)
    a.err = ctx->d_err;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.few = x.few; a.tpt = x.tpt; a.words = x.words; a.cap = x.cap; a.runs = x.runs; a.units_cap = x.units; a.rows_cap = x.rows;
    a.head = reinterpret_cast<TileHead*>(ws + x.head);
    a.req = reinterpret_cast<int4*>(ws + x.req);
    a.unit = reinterpret_cast<int2*>(ws + x.unit);
    a.short_row = reinterpret_cast<int*>(ws + x.short_row);
    a.count = reinterpret_cast<int4*>(ws + x.count);
    a.ent = reinterpret_cast<int2*>(ws + x.ent);
    a.mask = reinterpret_cast<uint32_t*>(ws + x.mask);
    a.part_o = reinterpret_cast<float*>(ws + x.part_o);
    a.part_ml = reinterpret_cast<float2*>(ws + x.part_ml);
    a.pair_ml = reinterpret_cast<float2*>(ws + x.pair_ml);
    a.cut = reinterpret_cast<int4*>(ws + x.cut);
    CUtensorMap mq, mk, mv, mk16, mv16;
    if (!encode_fn()) return hsq::fail(ctx, HSQ_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    const uint64_t n = (uint64_t)pages->n_pages * Hkv * P;
    if (!encode_halves(&mk16, pages->k, n, 16) || !encode_halves(&mv16, pages->v, n, 16))
        return hsq::fail(ctx, HSQ_ERR_CUDA, "cuTensorMapEncodeTiled refused a tensor map");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    const bool tiles = max_new > x.few;
    // requests of a few rows together, where the union of their pages has room
    const int most = std::min(max_new, x.few);
    const long long unit_pages = std::min<long long>(np + width, (long long)most * top);
    const bool group = most > 1 && unit_pages <= 8 * (kGroupList - 1);
    if (group) {
        const long long units = (long long)B * Hkv;
        int S = cluster_of(units, 2LL * ctx->num_sms, std::max<long long>(top, unit_pages / 2) * P, 512);
        while (unit_pages > S * (kGroupList - 1LL)) ++S;
        const int H = most * a.r <= 16 ? 1 : 2;
        const void* fn = H == 1 ? (const void*)page_attn_group_kernel<1> : (const void*)page_attn_group_kernel<2>;
        void* args[] = {&mk16, &mv16, &a};
        if ((e = hsq::raise_smem_limit(fn, ctx->device, group_smem(H))) == cudaSuccess)
            e = launch_cluster(fn, (unsigned)(units * S), kThreadsRow * H, S, group_smem(H), s, false, args);
        if (e != cudaSuccess) return hsq::cuda_fail(ctx, e, "page_attn groups");
    }
    if (tiles) {
        if (!encode_q(&mq, q, rows, Hq, a.r, x.tpt) || !encode_groups(&mk, pages->k, n, P) || !encode_groups(&mv, pages->v, n, P))
            return hsq::fail(ctx, HSQ_ERR_CUDA, "cuTensorMapEncodeTiled refused a tensor map");
        void* args[] = {&a};
        void* tc_args[] = {&mq, &mk, &mv, &a};
        if ((e = hsq::raise_smem_limit((const void*)page_tiles_kernel, ctx->device, kTcSmem)) != cudaSuccess)
            return hsq::cuda_fail(ctx, e, "cudaFuncSetAttribute(page_tiles)");
        // (each begins while the one before ends, and waits for it before it reads; the plan needs nothing of the groups' kernel, which
        // everything before the call precedes)
        if ((e = launch((const void*)page_plan_kernel, 1, kPlanThreads, 0, s, group, args)) != cudaSuccess ||
            (e = launch((const void*)page_list_kernel, x.units * Hkv, kListThreads, 0, s, true, args)) != cudaSuccess ||
            (e = launch((const void*)page_tiles_kernel, x.runs, kTcThreads, kTcSmem, s, true, tc_args)) != cudaSuccess ||
            (e = launch((const void*)page_join_kernel, x.runs * 8, 256, 0, s, true, args)) != cudaSuccess)
            return hsq::cuda_fail(ctx, e, "page_attn tiles");
    }
    if (group) return HSQ_OK;
    const long long units = (tiles ? (long long)x.rows : rows) * Hkv;
    const int S = cluster_of(units, 2LL * ctx->num_sms, (long long)top * P, 256);
    const void* fn = (const void*)page_attn_rows_kernel;
    e = hsq::raise_smem_limit(fn, ctx->device, kRowSmem);
    if (e != cudaSuccess) return hsq::cuda_fail(ctx, e, "cudaFuncSetAttribute(page_attn)");
    void* args[] = {&mk16, &mv16, &a};
    if ((e = launch_cluster(fn, (unsigned)(units * S), kThreadsRow, S, kRowSmem, s, tiles, args)) != cudaSuccess)
        return hsq::cuda_fail(ctx, e, "page_attn");
    return HSQ_OK;
}

}  // extern "C"
