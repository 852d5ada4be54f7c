// Attention over selected pages (hsq_page_attn).
//
// For row i and query head jq of KV head h: one softmax, scale 1/sqrt(128), over the tokens (up to the row's last) of the
// logical pages in sel[i][h].  Parts of a softmax over disjoint sets of keys join as
//     out = sum_p exp(m_p - M) o_p / sum_p exp(m_p - M) l_p,   M = max_p m_p,
// with m, l, o a reference exponent, the sum of exp(x - m) and the sum of exp(x - m) v of a part.
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
    int fault;   // HSQ_FAULT_WAIT_FEW: as if one had (0 but in tests)
    int* err;
};

// ---------------------------------------------------------------------------------------
// Rows one by one: a cluster of CTAs for each (row, KV head), four warps a CTA.  The row's pages are listed once a CTA; the
// cluster's warps cut the line of their groups of 16 keys into equal runs.  A warp loads its groups three ahead (TMA, 128-byte
// swizzle, 8 KB each) and multiplies as
//   S^T (16 keys x 8 heads) = K (A operand, by ldmatrix) Q^T (B);
//   O^T (128 dims x 8 heads) += V^T (A, by transposing ldmatrix) P^T (B), P^T from S^T by two 8 x 8 transposes,
// so no lane exchanges logits but for a new maximum.  The warps' parts are joined in shared memory, the CTAs' through
// distributed shared memory.
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
    const int unit = blockIdx.x / S, h = unit % a.Hkv, row = unit / a.Hkv;
    int bad = 0;
    bool failed = false;

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
    if (blockIdx.x == 0) bad |= offsets_bad(a.q_start, a.B, a.rows, kThreadsRow);
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
        if (lane == 0) {
            const uint32_t dst = stages + in.stage * kStageBytes, bar = bars + 8 * in.stage;
            const int y = ((list[ask >> sub_shift].x * a.Hkv + h) << a.page_shift) + 16 * (ask & ((1 << sub_shift) - 1));
            mbar_expect_tx(bar, kStageBytes);
            tma_2d(dst, &mk, 0, y, bar);
            tma_2d(dst + 2048, &mk, 64, y, bar);
            tma_2d(dst + 4096, &mv, 0, y, bar);
            tma_2d(dst + 6144, &mv, 64, y, bar);
        }
        __syncwarp();
        in.advance();
        ++ask;
    };
    for (int i = 0; i < kStages; ++i) load();
    failed |= (a.fault & HSQ_FAULT_WAIT_FEW) != 0;
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

cudaError_t launch_cluster(const void* fn, unsigned grid, int threads, int cluster, size_t smem, cudaStream_t st, void** args) {
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3(grid);
    lc.blockDim = dim3(threads);
    lc.dynamicSmemBytes = smem;
    lc.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    lc.attrs = at;
    lc.numAttrs = 1;
    return cudaLaunchKernelExC(&lc, fn, args);
}

}  // namespace

extern "C" {

hsq_status hsq_page_attn_workspace_size(const hsq_ctx* ctx, int page_n, int rows, int B, int width, int prefix_len,
                                        int top, int max_new, size_t* bytes) {
    if (!ctx || !bytes) return hsq::fail(nullptr, HSQ_ERR_INVALID, "ctx or bytes is NULL");
    const char* wrong = hsq::selection_shape_wrong(page_n, rows, B, width, prefix_len, top, max_new);
    if (wrong) return hsq::fail(nullptr, HSQ_ERR_INVALID, wrong);
    *bytes = 256;
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
    size_t need = 0;
    hsq_page_attn_workspace_size(ctx, pages->page_n, rows, B, width, prefix_len, top, max_new, &need);
    if (workspace_bytes < need)
        return hsq::fail(ctx, HSQ_ERR_INVALID, "workspace smaller than hsq_page_attn_workspace_size");
    const int Hq = ctx->cfg.n_q_heads, Hkv = ctx->cfg.n_kv_heads, P = pages->page_n, np = (prefix_len + P - 1) / P;
    if ((long long)rows * Hkv >= (1LL << 27)) return hsq::fail(ctx, HSQ_ERR_INVALID, "too many rows");
    const size_t q_bytes = (size_t)rows * Hq * 256, pool = (size_t)pages->n_pages * Hkv * P * 256;
    const hsq::Span ins[] = {{q, q_bytes}, {q_start, 4 * ((size_t)B + 1)}, {lens, 4 * (size_t)B}, {table, 4 * (size_t)B * width},
                             {prefix_len > 0 ? prefix : nullptr, 4 * (size_t)np}, {sel, (size_t)rows * Hkv * top * 4},
                             {pages->k, pool}, {pages->v, pool}};
    const hsq::Span outs[] = {{out, q_bytes}, {lse_opt, (size_t)rows * Hq * 4}, {workspace, need}};
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
    a.fault = (int)hsq::fault_mask() & HSQ_FAULT_WAIT_FEW;
    a.polls = a.fault ? 1 << 8 : 1 << 18;  // (a poll that finds nothing takes 4 us: 1 ms, or a second)
    a.err = ctx->d_err;
    CUtensorMap mk, mv;
    if (!encode_fn()) return hsq::fail(ctx, HSQ_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    const uint64_t n = (uint64_t)pages->n_pages * Hkv * P;
    if (!encode_rows(&mk, pages->k, n, 16) || !encode_rows(&mv, pages->v, n, 16))
        return hsq::fail(ctx, HSQ_ERR_CUDA, "cuTensorMapEncodeTiled refused a tensor map");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const long long units = (long long)rows * Hkv;
    int S = 1;
    while (S < 8 && units * S < 4LL * ctx->num_sms && (long long)top * P >= 128LL * S) S *= 2;
    const void* fn = (const void*)page_attn_rows_kernel;
    cudaError_t e = hsq::raise_smem_limit(fn, ctx->device, kRowSmem);
    if (e != cudaSuccess) return hsq::cuda_fail(ctx, e, "cudaFuncSetAttribute(page_attn)");
    void* args[] = {&mk, &mv, &a};
    if ((e = launch_cluster(fn, (unsigned)(units * S), kThreadsRow, S, kRowSmem, s, args)) != cudaSuccess)
        return hsq::cuda_fail(ctx, e, "page_attn");
    return HSQ_OK;
}

}  // extern "C"
