"""Long contexts on the GPU against the 64-bit oracle: the paged write with a
model's own rotation, the pages' summaries, the selection of pages, the
attention over them, and a run of the four together."""

import numpy as np
import pytest

from hsq_harness import ensure_built
from oracle import paged as P
from test_gpu_paged import attn_inputs, host, i32, i64, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def word(ctx):
    import hierarchical_kv_cache_hsq_gb300 as H
    w = H.hsq_sync_status(ctx)
    return {n for n in ("PAGE", "LEN", "POS", "SEL") if w & getattr(H, "HSQ_DEVERR_" + n)}


# -- rotation --------------------------------------------------------------------------------

@pytest.mark.parametrize("rows", [1, 7, 600])
@pytest.mark.parametrize("dims,interleaved", [(128, False), (128, True), (64, False), (64, True), (8, False), (8, True),
                                              (96, False), (104, True)])
@pytest.mark.parametrize("dtype,fused,Hq,Hkv", [("bfloat16", True, 40, 8), ("float32", False, 5, 1),
                                                ("bfloat16", False, 4, 4), ("float32", True, 16, 8)])
def test_write_with_a_rotation(rows, dims, interleaved, dtype, fused, Hq, Hkv):
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    rng = np.random.default_rng(rows + dims)
    page, max_pos = 32, 70000
    ctx = make(Hq, Hkv, 1, 1000)  # the rotation has a limit of its own
    scaling = {128: "yarn", 64: "linear", 8: "none", 96: "base", 104: "yarn"}[dims]
    kw = dict(dims=dims, theta=5e5, scaling=scaling, factor=4.0, original=17500.0)
    rope = H.make_rope(ctx, interleaved=interleaved, max_pos=max_pos, **kw)
    omega, amp = P.rope_frequencies(**kw)
    x = torch.from_numpy(rng.standard_normal((rows, Hq + 2 * Hkv, 128)).astype(np.float32)).cuda().to(getattr(torch, dtype))
    q, k, v = x[:, :Hq], x[:, Hq: Hq + Hkv], x[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    n_pages = -(-rows // page) + 2
    pool = H.PagePool(*[torch.full((n_pages, Hkv, page, 128), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)])
    before = host(pool.k), host(pool.v)
    slots = rng.permutation(n_pages * page)[:rows].astype(np.int64)
    pos = rng.integers(0, max_pos, rows).astype(np.int32)
    pos[0] = max_pos - 1
    if rows > 4:
        pos[1], slots[2], pos[3], slots[4] = -1, -1, 0, -9
    q_out = torch.full((rows, Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    H.hsq_page_write(ctx, pool, q, k, v, i32(pos), i64(slots), q_out, rope=rope)
    assert word(ctx) == set()
    wq, wk, wv = P.page_write_rope(*before, host(q), host(k), host(v), pos, slots, omega, amp, interleaved, max_pos)
    # as for the context's rotation: one rounding to bf16, and under 8 roundings of 2^-24 of |a| + |b| <= 12, amp times
    for got, want in ((host(pool.k), wk), (host(pool.v), wv)):
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + amp * 12 * 2.0 ** -21).all()
    live = pos >= 0
    g = host(q_out)
    assert (np.abs(g - wq) <= 2.0 ** -8 * np.abs(wq) + amp * 12 * 2.0 ** -21)[live].all()
    assert (g[~live] == 7.0).all()
    # dims that are not turned are copied: one rounding of the input, none for bf16
    np.testing.assert_array_equal(g[live][..., dims:], host(q.to(torch.bfloat16))[live][..., dims:])


def test_the_contexts_rotation_as_a_table_gives_the_same_results():
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    ctx = make(8, 4, 1, 4096)
    q, k = torch.randn(300, 8, 128, device="cuda"), torch.randn(300, 4, 128, device="cuda")
    pos, slots = i32(np.arange(300) * 13), i64(np.arange(300))
    got = []
    for rope in (None, H.make_rope(ctx)):
        pool, out = H.allocate_pages(ctx, 20, 16), torch.empty(300, 8, 128, dtype=torch.bfloat16, device="cuda")
        H.hsq_page_write(ctx, pool, q, k, k, pos, slots, out, rope=rope)
        got.append((host(out), host(pool.k)))
    assert word(ctx) == set()
    np.testing.assert_array_equal(got[0][0], got[1][0])
    np.testing.assert_array_equal(got[0][1], got[1][1])


def test_a_rotation_of_given_frequencies_and_its_limit():
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    ctx = make(4, 2, 1, 64)
    omega = [0.5, 0.25, 0.0, -1.0]
    rope = H.make_rope(ctx, omega=omega, amplitude=1.5, max_pos=300, interleaved=True)
    assert rope.dims == 8 and rope.max_pos == 300
    k = torch.randn(2, 2, 128, device="cuda")
    pool = H.allocate_pages(ctx, 1, 16)
    H.hsq_page_write(ctx, pool, None, k, k, i32([299, 300]), i64([0, 1]), None, rope=rope)
    assert word(ctx) == {"POS"}
    for i in range(2):
        want = P.rotate(host(k)[i].astype(np.float64), 299, np.array(omega), 1.5, True)
        assert (np.abs(host(pool.k)[0, :, i] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -17).all()


# -- summaries ---------------------------------------------------------------------------------

def check_summaries(codes, scale, want_codes, want_scale):
    np.testing.assert_array_equal(codes, want_codes)
    # the sum's rounding to fp32 and the division's: 2^-24 each, and its last bits
    fine = np.isfinite(want_scale)
    assert (np.isposinf(scale) == ~fine).all()
    assert (np.abs(scale - want_scale)[fine] <= want_scale[fine] * 2.0 ** -22).all()


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Hkv,spans", [(1, [(0, 1)]), (2, [(3, 40), (15, 1), (0, 16), (127, 130)]), (8, [(5, 700)]),
                                       (3, [(i % 16, 1) for i in range(70)]), (8, [(0, 6000)])])
def test_summaries(page, Hkv, spans):
    """spans: (first token inside its page, tokens) of each request."""
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    rng = np.random.default_rng(page + Hkv)
    ctx = make(Hkv, Hkv, 1)
    spans = [(a % page, n) for a, n in spans]
    used = [-(-(a + n) // page) for a, n in spans]
    n_pages = sum(used) + 3
    ids, at, slots = rng.permutation(n_pages), 0, []
    for (a, n), u in zip(spans, used):
        t = a + np.arange(n)
        slots.append(ids[at + t // page] * page + t % page)
        at += u
    slots = np.concatenate(slots + [np.full(3, -1)])
    k = (rng.standard_normal((n_pages, Hkv, page, 128)) + rng.standard_normal((n_pages, Hkv, 1, 128))).astype(np.float32)
    pool = H.PagePool(*[torch.from_numpy(k).cuda().bfloat16()] * 2)
    codes = rng.integers(-127, 128, (n_pages, Hkv, 128)).astype(np.int8)
    scale = rng.random((n_pages, Hkv)).astype(np.float32)
    sums = H.PageSummaries(torch.from_numpy(codes).cuda(), torch.from_numpy(scale).cuda())
    H.hsq_page_summaries(ctx, pool, sums, i64(slots))
    assert word(ctx) == set()
    wc, ws, _ = P.page_summaries(host(pool.k), slots, codes, scale)
    check_summaries(sums.codes.cpu().numpy(), host(sums.scale), wc, ws)


def test_summaries_of_numbers_that_are_hard():
    """Ties at half a code, sums that cancel, huge, tiny and missing numbers, and stale tokens behind a page's end."""
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    rng = np.random.default_rng(7)
    k = np.full((12, 2, 16, 128), np.nan, np.float32)
    k[0, :, 0] = rng.choice([127.0, 63.5, -63.5, 1.0, 0.5, -0.5, 2.5], (2, 128))  # one token: ties
    k[0, :, 0, 0] = 127.0
    k[1, :, :2] = rng.standard_normal((2, 1, 128))
    k[1, 1, 1] *= -1  # the head's sum is 0
    k[2, :, :16] = rng.standard_normal((2, 16, 128)) * 10.0 ** rng.integers(-20, 20, (2, 16, 128))
    k[3, :, :3] = 1e-30 * rng.standard_normal((2, 3, 128))
    k[4, :, :3] = 1e37 * rng.standard_normal((2, 3, 128))
    k[5, :, :5] = rng.standard_normal((2, 5, 128))
    k[5, 0, 2, 9], k[5, 1, 3, 100] = np.inf, np.nan
    k[6, :, :4] = 3e38
    k[7, :, :16] = 1.0 + 2.0 ** -7 * rng.integers(0, 2, (2, 16, 128))
    k[8, :, :9] = 0.0
    k[9, :, :16] = np.where(np.arange(16)[:, None] % 2, 1e20, -1e20) + rng.standard_normal((2, 16, 128))
    ends = [0, 1, 15, 2, 2, 4, 3, 15, 8, 15]
    slots = np.array([16 * i + e for i, e in enumerate(ends)] + [16 * 12, 1 << 40])
    ctx = make(2, 2, 1)
    pool = H.PagePool(*[torch.from_numpy(k).cuda().bfloat16()] * 2)
    sums = H.allocate_summaries(ctx, pool)
    H.hsq_page_summaries(ctx, pool, sums, i64(slots))
    assert word(ctx) == {"PAGE"}
    wc, ws, _ = P.page_summaries(host(pool.k), slots, np.zeros((12, 2, 128), np.int8), np.zeros((12, 2), np.float32))
    check_summaries(sums.codes.cpu().numpy(), host(sums.scale), wc, ws)
    assert np.isposinf(ws[[5, 6]]).all() and (ws[[3, 8]] == 0).all()


# -- selection ------------------------------------------------------------------------------------

def selection_inputs(Hq, Hkv, page, prefix, own, new, top, pad=0, seed=0, levels=0):
    """attn_inputs with summaries of whole numbers (levels > 0: of so few that scores tie)."""
    x = attn_inputs(Hq, Hkv, page, prefix, own, new, pad, seed)
    rng = np.random.default_rng(seed + 1)
    n_pages = x["k"].shape[0]
    most = levels or 127
    x["codes"] = rng.integers(-most, most + 1, (n_pages, Hkv, 128)).astype(np.int8)
    x["scale"] = np.ones((n_pages, Hkv), np.float32) if levels else rng.random((n_pages, Hkv)).astype(np.float32)
    if levels:
        x["codes"][:, :, 2:] = 0
    x["top"] = top
    return x


def run_select(x, first=1, recent=2, ctx=None, max_new=None):
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    ctx = ctx or make(x["Hq"], x["Hkv"], len(x["lens"]))
    pool = H.PagePool(x["k"], x["v"])
    sums = H.PageSummaries(torch.from_numpy(x["codes"]).cuda(), torch.from_numpy(x["scale"]).cuda())
    rows, mx = x["q"].shape[0], max_new or x["max_new"]
    sel = torch.full((rows, x["Hkv"], x["top"]), -2, dtype=torch.int32, device="cuda")
    n = H.hsq_page_select_workspace_size(ctx, pool, rows, len(x["lens"]), x["table"].shape[1], x["prefix_len"], x["top"], mx)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    H.hsq_page_select(ctx, pool, sums, x["q"], i32(x["q_start"]), i32(x["lens"]), i32(x["table"]), sel, ws,
                      prefix=i32(x["prefix"]) if x["prefix_len"] else None, prefix_len=x["prefix_len"], first=first,
                      recent=recent, max_new=mx)
    return host(sel), word(ctx)


def want_select(x, first=1, recent=2):
    return P.page_select(x["codes"], x["scale"], host(x["q"]), x["q_start"], x["lens"], x["table"], x["prefix"],
                         x["prefix_len"], x["k"].shape[2], x["top"], first, recent)


@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (4, 2), (8, 2), (5, 1), (16, 2)])
@pytest.mark.parametrize("page,prefix,own,new,top", [
    (16, 0, [1, 15, 16, 17, 200, 600, 3000], 1, 8), (16, 1000, [0, 5, 33, 400], 1, 16), (32, 77, [900, 40, 333], 3, 7),
    (128, 5000, [4000, 1], 1, 37), (16, 100, [700], 150, 12), (64, 0, [5000, 90], 40, 20), (16, 0, [20000], 1, 512),
    (16, 300, [2500, 2600, 1], 20, 4), (16, 64, [3000], 129, 100)])
def test_selection(Hq, Hkv, page, prefix, own, new, top):
    for levels in (0, 1):
        x = selection_inputs(Hq, Hkv, page, prefix, own, [min(new, n) for n in own], top, pad=2, seed=Hq + page + top,
                             levels=levels)
        sel, err = run_select(x)
        assert not err
        np.testing.assert_array_equal(sel, want_select(x)[0])


@pytest.mark.parametrize("first,recent,top", [(0, 1, 1), (0, 1, 4), (3, 1, 4), (2, 5, 9), (0, 4, 4), (4, 4, 8)])
@pytest.mark.parametrize("new", [1, 40])
def test_pages_that_are_always_taken(first, recent, top, new):
    x = selection_inputs(8, 2, 16, 40, [50, 300, 45], [new, new, new], top, seed=top)
    sel, err = run_select(x, first, recent)
    assert not err
    np.testing.assert_array_equal(sel, want_select(x, first, recent)[0])


@pytest.mark.parametrize("new", [1, 60])
def test_scores_that_are_no_numbers_and_queries_without_a_direction(new):
    x = selection_inputs(8, 2, 16, 160, [400, 500, 600], [new] * 3, 9, seed=21)
    x["scale"][::3] = np.inf
    x["codes"][::3] = 0
    x["scale"][1::5] = 3e38  # scores beyond fp32's range on both sides
    q = x["q"].clone()
    q[0, :4], q[1, 4] = 0.0, float("nan")
    q[2, 0, 0], q[2, 1, 0] = float("inf"), -float("inf")
    x["q"] = q
    sel, err = run_select(x)
    assert not err
    np.testing.assert_array_equal(sel, want_select(x)[0])


@pytest.mark.parametrize("new", [1, 60])
def test_selection_leaves_out_pages_outside_the_pool(new):
    x = selection_inputs(8, 2, 16, 160, [400, 70], [new] * 2, 9, seed=22)
    x["table"][0, 3:9], x["table"][0, 11:20] = -1, x["k"].shape[0]
    x["prefix"][2:9] = 1 << 30
    sel, err = run_select(x)
    assert err == {"PAGE"}
    np.testing.assert_array_equal(sel, want_select(x)[0])
    # of request 1, at most pages 1, 9 .. 12 have a score and six are asked for
    assert (sel[new] == -1).any()


@pytest.mark.parametrize("new", [1, 40])
def test_selection_with_lengths_that_contradict(new):
    x = selection_inputs(8, 2, 16, 40, [100, 300, 200], [new, new + 1, new], 5, seed=23)
    sel, err = run_select(x, max_new=new)  # request 1 has more rows than max_new: not written
    assert err == {"LEN"}
    want = want_select(x)[0]
    want[new: 2 * new + 1] = -2
    np.testing.assert_array_equal(sel, want)
    x["table"] = x["table"].clip(0)
    x["lens"][2], x["lens"][0] = 10 ** 6, new - 1
    sel, err = run_select(x)
    assert err == {"LEN"}
    np.testing.assert_array_equal(sel, want_select(x)[0])
    x["q_start"] = np.array([0, new + 2, new, 3 * new], np.int32)
    assert run_select(x)[1] == {"LEN"}


# -- attention ------------------------------------------------------------------------------------

def some_selection(x, page, top, seed, order=True):
    """Random ascending pages of each row, fewer in some rows, none in some."""
    rng = np.random.default_rng(seed)
    rows, Hkv = x["q"].shape[0], x["Hkv"]
    sel = np.full((rows, Hkv, top), -1, np.int32)
    for i in range(rows):
        at = P.row_pages(i, x["q_start"], x["lens"], x["table"], page, x["prefix_len"])
        if at is None:
            continue
        for h in range(Hkv):
            n = min(at[2], top if rng.random() < 0.6 else int(rng.integers(0, top + 1)))
            take = np.sort(rng.permutation(at[2])[:n])
            if n and rng.random() < 0.7:
                take[-1] = at[2] - 1
            sel[i, h, :n] = take
    return sel


def run_page_attn(x, sel, ctx=None, lse=True, max_new=None):
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    ctx = ctx or make(x["Hq"], x["Hkv"], len(x["lens"]))
    pool = H.PagePool(x["k"], x["v"])
    out = torch.full_like(x["q"], 7.0)
    ls = torch.full(x["q"].shape[:2], 7.0, device="cuda") if lse else None
    mx = max_new or x["max_new"]
    n = H.hsq_page_attn_workspace_size(ctx, pool, x["q"].shape[0], len(x["lens"]), x["table"].shape[1], x["prefix_len"],
                                       sel.shape[2], mx)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN as float: nothing of it is read
    H.hsq_page_attn(ctx, pool, x["q"], i32(x["q_start"]), i32(x["lens"]), i32(x["table"]), i32(sel), out, ws,
                    prefix=i32(x["prefix"]) if x["prefix_len"] else None, prefix_len=x["prefix_len"], max_new=mx, lse=ls)
    return host(out), None if ls is None else host(ls), word(ctx)


def check_page_attn(x, sel, out, lse, live=None):
    """Bounds as for the attention over all tokens (test_gpu_paged.check_attn)."""
    want, wl, spread, mass, _ = P.page_attn(host(x["k"]), host(x["v"]), host(x["q"]), x["q_start"], x["lens"], x["table"],
                                            x["prefix"], x["prefix_len"], sel)
    rows = int(x["q_start"][-1])
    live = np.arange(len(want)) < rows if live is None else live
    d = mass * 2.0 ** -17
    tol = 2.0 ** -8 * np.abs(want) + spread * (2.0 ** -8 + 2 * d[..., None] + 2.0 ** -18) * 1.01
    bad = ~(np.abs(out - want) <= tol)
    assert not bad[live].any(), (np.argwhere(bad & live[:, None, None])[:5], np.abs(out - want)[live].max())
    assert (out[~live] == 7.0).all()
    if lse is not None:
        fine = np.isfinite(wl) & live[:, None]
        assert (np.isneginf(lse) == np.isneginf(wl))[live].all()
        n_keys = sel.shape[2] * x["k"].shape[2]
        tol = d[fine] + n_keys * 2.0 ** -24 + 2.0 ** -20 * (1 + np.abs(wl[fine]))
        assert (np.abs(lse - np.where(fine, wl, 0))[fine] <= tol).all()
        assert (lse[~live] == 7.0).all()


@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (4, 2), (8, 2), (5, 1), (16, 2), (40, 8)])
@pytest.mark.parametrize("page,prefix,own,new,top", [
    (16, 0, [1, 15, 16, 17, 200, 600], 1, 8), (128, 300, [0, 5, 133, 400], 1, 3), (32, 77, [900, 40, 333], 3, 7),
    (64, 500, [700, 90], 1, 1), (16, 100, [700], 150, 12), (64, 0, [1000, 90], 40, 6), (16, 0, [9000], 1, 512),
    (16, 300, [500, 260, 1], 20, 5), (32, 64, [1000], 260, 10), (128, 0, [640], 77, 4), (16, 5, [40, 30], 33, 40)])
def test_attention(Hq, Hkv, page, prefix, own, new, top):
    x = attn_inputs(Hq, Hkv, page, prefix, own, [min(new, n) for n in own], pad=2, seed=Hq + page + top)
    sel = some_selection(x, page, top, seed=top)
    out, lse, err = run_page_attn(x, sel)
    assert not err
    check_page_attn(x, sel, out, lse)


@pytest.mark.parametrize("new", [[1, 1, 1], [3, 200, 1], [64, 64, 64], [1, 33, 5]])
def test_attention_of_requests_of_many_kinds(new):
    x = attn_inputs(8, 2, 16, 150, [400, 300, 250], new, pad=1, seed=31)
    sel = some_selection(x, 16, 14, seed=32)
    out, lse, err = run_page_attn(x, sel)
    assert not err
    check_page_attn(x, sel, out, lse)
    out2, _, _ = run_page_attn(x, sel, lse=False)
    np.testing.assert_array_equal(out, out2)


@pytest.mark.parametrize("new", [1, 70])
def test_all_pages_selected_is_the_attention_over_all_tokens(new):
    import torch
    from test_gpu_paged import check_attn
    x = attn_inputs(8, 2, 32, 100, [300, 177], [new, new], seed=33)
    pages = 4 + 10
    sel = np.full((2 * new, 2, pages), -1, np.int32)
    for i in range(2 * new):
        c = P.row_pages(i, x["q_start"], x["lens"], x["table"], 32, 100)[2]
        sel[i, :, :c] = np.arange(c)
    out, lse, err = run_page_attn(x, sel)
    assert not err
    check_attn(x, out, lse)
    assert torch.is_tensor(x["q"])


@pytest.mark.parametrize("new", [1, 50])
def test_entries_that_are_wrong_are_left_out_and_none_counts_twice(new):
    x = attn_inputs(8, 2, 16, 100, [200, 260], [new, new], seed=34)
    rng = np.random.default_rng(35)
    sel = rng.integers(-3, 30, (2 * new, 2, 45)).astype(np.int32)
    sel[0, 0] = 1 << 30
    sel[-1, 1, :3] = [5, 5, 5]
    out, lse, err = run_page_attn(x, sel)
    assert err == {"SEL"}
    check_page_attn(x, sel, out, lse)
    assert (out[0, :4] == 0).all() and np.isneginf(lse[0, :4]).all()


@pytest.mark.parametrize("new", [1, 50])
def test_selected_pages_outside_the_pool(new):
    x = attn_inputs(8, 2, 16, 100, [160, 90], [new, new], seed=36)
    sel = some_selection(x, 16, 9, seed=37)
    x["table"][0, 1:4], x["table"][1, 2], x["prefix"][3] = -1, x["k"].shape[0], -7
    out, lse, err = run_page_attn(x, sel)
    assert err == {"PAGE"}
    check_page_attn(x, sel, out, lse)


@pytest.mark.parametrize("new", [1, 40])
def test_attention_with_lengths_that_contradict(new):
    x = attn_inputs(8, 2, 16, 40, [100, 300, 200], [new, new + 1, new], seed=38)
    sel = some_selection(x, 16, 6, seed=39)
    live = np.ones(3 * new + 1, bool)
    live[new: 2 * new + 1] = False
    out, lse, err = run_page_attn(x, sel, max_new=new)
    assert err == {"LEN"}
    check_page_attn(x, sel, out, lse, live)
    x["table"] = x["table"].clip(0)
    x["lens"][2], x["lens"][0] = 10 ** 6, new - 1  # past its table; below its rows: the first sees the prefix only
    x["k"], x["v"] = x["k"].nan_to_num(0.25), x["v"].nan_to_num(0.25)
    sel = some_selection(x, 16, 6, seed=40)
    out, lse, err = run_page_attn(x, sel)
    assert err == {"LEN"}
    check_page_attn(x, sel, out, lse)
    x["q_start"] = np.array([0, new + 2, new, 3 * new], np.int32)
    assert "LEN" in run_page_attn(x, sel)[2]


@pytest.mark.parametrize("stale", [float("inf"), -3.0e38])
@pytest.mark.parametrize("new", [1, 40])
def test_what_lies_past_a_row_does_not_matter(stale, new):
    x = attn_inputs(8, 2, 64, 75, [45, 70, 200], [new] * 3, seed=41, stale=stale)
    sel = some_selection(x, 64, 4, seed=42)
    out, lse, err = run_page_attn(x, sel)
    assert not err
    check_page_attn(x, sel, out, lse)


@pytest.mark.parametrize("new", [1, 40])
def test_a_query_that_is_no_number_shows_in_its_row_alone(new):
    x = attn_inputs(8, 2, 16, 75, [345, 70], [new] * 2, seed=43)
    sel = some_selection(x, 16, 5, seed=44)
    sel[0, :, 0] = 0
    sel[0, :, 1:] = -1
    q = x["q"].clone()
    q[0, 2] = float("nan")
    x["q"] = q
    out, lse, err = run_page_attn(x, sel)
    assert not err and np.isnan(out[0, 2]).all() and np.isnan(lse[0, 2])
    x["q"] = q.nan_to_num(0.0)
    live = np.ones((2 * new, 8), bool)
    live[0, 2] = False
    want = P.page_attn(host(x["k"]), host(x["v"]), host(x["q"]), x["q_start"], x["lens"], x["table"], x["prefix"], 75, sel)[0]
    assert (np.abs(out - want)[live] < 0.05).all()


def test_large_logits():
    for new in (1, 48):
        x = attn_inputs(8, 2, 16, 60, [200, 180], [new] * 2, seed=45, scale=40.0)
        sel = some_selection(x, 16, 8, seed=46)
        out, lse, err = run_page_attn(x, sel)
        assert not err
        check_page_attn(x, sel, out, lse)


# -- together -------------------------------------------------------------------------------------

@pytest.mark.parametrize("chunk", [1, 90])
def test_a_step_of_the_four_calls_captured_and_replayed(chunk):
    """Tables, rotated write, summaries, selection and attention of growing requests, in one graph."""
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    rng = np.random.default_rng(50 + chunk)
    Hq, Hkv, page, top, B, width, n_pages, rows = 8, 2, 16, 6, 3, 60, 200, 3 * chunk + 2
    ctx = make(Hq, Hkv, B, 8192)
    kw = dict(dims=64, theta=1e6, scaling="yarn", factor=4.0, original=256.0)
    rope = H.make_rope(ctx, interleaved=True, **kw)
    omega, amp = P.rope_frequencies(**kw)
    pool = H.allocate_pages(ctx, n_pages, page)
    sums = H.allocate_summaries(ctx, pool)
    pre = 50
    free = rng.permutation(n_pages).astype(np.int32)
    d = dict(cached=i32([0, 0, 0]), fresh=i32([0, 0, 0]), free=i32(free[4:]), used=i32([0]), table=i32(np.full((B, width), -1)),
             slots=i64(np.zeros(rows)), pos=i32(np.zeros(rows)), q_start=i32(np.zeros(B + 1)), lens=i32(np.zeros(B)),
             used_out=i32([0]))
    prefix = i32(free[:4])
    x = torch.zeros(rows, Hq + 2 * Hkv, 128, dtype=torch.bfloat16, device="cuda")
    q_rot = torch.zeros(rows, Hq, 128, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.zeros_like(q_rot), torch.zeros(rows, Hq, device="cuda")
    sel = torch.full((rows, Hkv, top), -2, dtype=torch.int32, device="cuda")
    ws = [torch.empty(f(ctx, pool, rows, B, width, pre, top, chunk), dtype=torch.uint8, device="cuda")
          for f in (H.hsq_page_select_workspace_size, H.hsq_page_attn_workspace_size)]

    def step():
        H.hsq_page_tables(ctx, pool, d["cached"], d["fresh"], d["free"], d["used"], d["table"], d["slots"], d["pos"],
                          d["q_start"], d["lens"], d["used_out"], base=pre)
        H.hsq_page_write(ctx, pool, x[:, :Hq], x[:, Hq: Hq + Hkv], x[:, Hq + Hkv:], d["pos"], d["slots"], q_rot, rope=rope)
        H.hsq_page_summaries(ctx, pool, sums, d["slots"])
        H.hsq_page_select(ctx, pool, sums, q_rot, d["q_start"], d["lens"], d["table"], sel, ws[0], prefix=prefix,
                          prefix_len=pre, max_new=chunk)
        H.hsq_page_attn(ctx, pool, q_rot, d["q_start"], d["lens"], d["table"], sel, out, ws[1], prefix=prefix,
                        prefix_len=pre, max_new=chunk, lse=lse)

    # the prefix: its own pages' slots
    pk = torch.randn(pre, Hkv, 128, dtype=torch.bfloat16, device="cuda")
    ps = free[np.arange(pre) // page].astype(np.int64) * page + np.arange(pre) % page
    H.hsq_page_write(ctx, pool, None, pk, pk, i32(np.arange(pre)), i64(ps), None, rope=rope)
    H.hsq_page_summaries(ctx, pool, sums, i64(ps))
    g = torch.cuda.CUDAGraph()
    step()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step()
    cached = np.zeros(B, np.int64)
    for it in range(6):
        fresh = np.minimum(rng.integers(0, chunk + 1, B), 150) if chunk > 1 else np.array([1, it % 2, 1])
        d["cached"].copy_(i32(cached))
        d["fresh"].copy_(i32(fresh))
        x.copy_(torch.randn(x.shape, device="cuda"))
        n = int(fresh.sum())
        before = host(pool.k), host(pool.v)
        out.fill_(7.0)
        lse.fill_(7.0)
        sel.fill_(-2)
        g.replay()
        d["used"].copy_(d["used_out"])
        assert word(ctx) == set()
        slots, pos = host(d["slots"]), host(d["pos"])
        xs = host(x)
        wq, wk, _ = P.page_write_rope(*before, xs[:, :Hq], xs[:, Hq: Hq + Hkv], xs[:, Hq + Hkv:], pos, slots, omega, amp,
                                      True, 8192)
        assert (np.abs(host(pool.k) - wk) <= 2.0 ** -8 * np.abs(wk) + 2.0 ** -16).all()
        wc, wsc, _ = P.page_summaries(host(pool.k), slots, sums.codes.cpu().numpy(), host(sums.scale))
        check_summaries(sums.codes.cpu().numpy(), host(sums.scale), wc, wsc)
        y = dict(q=q_rot, k=pool.k, v=pool.v, q_start=host(d["q_start"]), lens=host(d["lens"]), table=host(d["table"]),
                 prefix=free[:4], prefix_len=pre, Hq=Hq, Hkv=Hkv, codes=sums.codes.cpu().numpy(), scale=host(sums.scale), top=top)
        assert (y["lens"] == cached + fresh).all()
        want = want_select(y)[0]
        np.testing.assert_array_equal(host(sel), want)
        if n:
            check_page_attn(y, host(sel), host(out), host(lse))
        cached += fresh


# -- refusals -------------------------------------------------------------------------------------

def test_refusals():
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    x = selection_inputs(8, 2, 16, 40, [60, 70], [1, 1], 5, seed=60)
    ctx = make(8, 2, 2)
    pool = H.PagePool(x["k"], x["v"])
    sums = H.PageSummaries(torch.from_numpy(x["codes"]).cuda(), torch.from_numpy(x["scale"]).cuda())
    base = dict(q=x["q"], q_start=i32(x["q_start"]), lens=i32(x["lens"]), table=i32(x["table"]),
                sel=torch.zeros(2, 2, 5, dtype=torch.int32, device="cuda"), workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"),
                prefix=i32(x["prefix"]), prefix_len=40, max_new=1)
    out = torch.zeros_like(x["q"])

    def select(**kw):
        a = dict(base, first=1, recent=2, sums=sums)
        a.update(kw)
        H.hsq_page_select(ctx, a.pop("pool", pool), a.pop("sums"), **a)

    def attn(**kw):
        a = dict(base, out=out, lse=None)
        a.update(kw)
        H.hsq_page_attn(ctx, a.pop("pool", pool), **a)

    select()
    attn()
    other = torch.zeros(2, 2, 513, dtype=torch.int32, device="cuda")
    wide = torch.zeros(2, 40000, dtype=torch.int32, device="cuda")
    for f in (select, attn):
        for kw in (dict(prefix_len=-1), dict(prefix_len=1 << 40), dict(max_new=0), dict(sel=other), dict(table=wide),
                   dict(workspace=base["workspace"][:8]), dict(workspace=base["workspace"][1:]), dict(prefix=None),
                   dict(prefix=base["prefix"][:1]), dict(q=x["q"].float()), dict(sel=base["sel"][:1]), dict(sel=base["sel"].long()),
                   dict(q_start=base["q_start"][:2]), dict(lens=base["lens"].cpu()), dict(table=base["table"][0]),
                   dict(q=x["q"][:, :4]), dict(workspace=base["workspace"].cpu())):
            with pytest.raises((ValueError, H.HSQError)):
                f(**kw)
    for kw in (dict(first=-1), dict(recent=0), dict(first=4), dict(first=1 << 33), dict(recent=6),
               dict(sel=base["table"].view(-1)[:20].view(2, 2, 5) if base["table"].numel() >= 20 else base["q_start"]),
               dict(sums=H.PageSummaries(sums.codes[:-1].contiguous(), sums.scale[:-1].contiguous()))):
        with pytest.raises((ValueError, H.HSQError)):
            select(**kw)
    for kw in (dict(out=x["q"]), dict(out=out[:1]), dict(lse=torch.zeros(2, 4, device="cuda")), dict(out=out.float()),
               dict(lse=torch.zeros(2, 8, device="cuda", dtype=torch.float64))):
        with pytest.raises((ValueError, H.HSQError)):
            attn(**kw)
    rope = H.make_rope(ctx, dims=32)
    k = torch.zeros(2, 2, 128, device="cuda")
    with pytest.raises(H.HSQError):  # the table is an input that the pool may not overlap
        bad = torch.zeros(pool.k.numel(), dtype=torch.bfloat16, device="cuda").view(pool.k.shape)
        shared = bad.view(-1).view(torch.float32)[: 272 * 32].view(272, 32)
        H.hsq_page_write(ctx, H.PagePool(bad, torch.zeros_like(bad)), None, k, k, i32([0, 1]), i64([0, 1]), None,
                         rope=H.Rope(shared, False, 4096))
    for bad in (lambda: H.Rope(rope.table, False, 10000), lambda: H.Rope(rope.table.double(), False, 4096),
                lambda: H.Rope(rope.table.cpu(), False, 4096), lambda: H.PageSummaries(sums.codes.float(), sums.scale),
                lambda: H.PageSummaries(sums.codes, sums.scale[:1]), lambda: H.hsq_page_summaries(ctx, pool, sums, i32([0])),
                lambda: H.hsq_page_summaries(ctx, pool, sums, i64([])),
                lambda: H.hsq_page_summaries(ctx, pool, H.PageSummaries(sums.codes, sums.scale), sums.codes.view(-1)[:64].view(torch.int64))):
        with pytest.raises((ValueError, H.HSQError)):
            bad()
    torch.cuda.synchronize()
    assert word(ctx) == set()
