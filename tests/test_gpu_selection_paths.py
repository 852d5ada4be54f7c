"""The ways that the selection of pages and the attention over them divide their
work, at the sizes where one way ends and another begins: more pages than a
chunk, a window or a thread's registers hold, unions that fit and that do not,
requests of all kinds in one call, streams, waits that run out, overlaps."""

import time

import numpy as np
import pytest

from hsq_harness import ensure_built
from oracle import paged as P
from test_gpu_paged import attn_inputs, host, i32, i64, make
from test_gpu_selection import (check_page_attn, check_summaries, run_page_attn, run_select, selection_inputs, some_selection,
                                want_select, word)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def long_inputs(Hq, Hkv, page, own, new, seed=0):
    """attn_inputs for long contexts: numbers for every token, made at once (no stale ones behind a length)."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    own, new = np.asarray(own), np.asarray(new)
    ns = -(-own // page)
    n_pages = int(ns.sum()) + 2
    ids = np.random.default_rng(seed).permutation(n_pages)
    table, at = np.full((len(own), int(ns.max()) + 1), -1, np.int32), 0
    for b in range(len(own)):
        table[b, : ns[b]] = ids[at: at + ns[b]]
        at += ns[b]
    k, v = (torch.randn((n_pages, Hkv, page, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    q = (1.5 * torch.randn((int(new.sum()), Hq, 128), generator=g, device="cuda")).bfloat16()
    return dict(q=q, k=k, v=v, table=table, prefix=np.zeros(0, np.int32), prefix_len=0,
                q_start=np.concatenate([[0], np.cumsum(new)]).astype(np.int32), lens=own.astype(np.int32),
                max_new=int(new.max()), Hq=Hq, Hkv=Hkv)


def with_summaries(x, top, levels=0, seed=0):
    rng = np.random.default_rng(seed)
    n_pages, Hkv = x["k"].shape[:2]
    most = levels or 127
    x["codes"] = rng.integers(-most, most + 1, (n_pages, Hkv, 128)).astype(np.int8)
    x["scale"] = np.ones((n_pages, Hkv), np.float32) if levels else rng.random((n_pages, Hkv)).astype(np.float32)
    if levels:
        x["codes"][:, :, 2:] = 0
    x["top"] = top
    return x


# pages: 2048, 4096, 8192 are where a row's selection takes more keys a thread; 1024 is a tile's chunk
@pytest.mark.parametrize("pages,new,top,levels", [
    (2047, 1, 64, 0), (2053, 2, 64, 1), (4099, 1, 300, 0), (8195, 1, 64, 0), (8200, 1, 512, 1), (20000, 1, 100, 0),
    (1027, 20, 64, 0), (1030, 17, 64, 1), (2060, 9, 512, 0), (3100, 33, 512, 1), (5000, 10, 4, 0), (1026, 9, 3, 0)])
def test_selection_of_many_pages(pages, new, top, levels):
    x = with_summaries(long_inputs(2, 1, 16, [16 * pages - 5, 300], [new, 1], seed=pages), top, levels, seed=top)
    sel, err = run_select(x)
    assert not err
    np.testing.assert_array_equal(sel, want_select(x)[0])


@pytest.mark.parametrize("new", [1, 12])
@pytest.mark.parametrize("kind", ["ascending", "descending", "one", "two", "huge", "negative"])
def test_selection_of_scores_that_lie_badly(new, kind):
    """Scores in order, all alike, of two values, over all magnitudes, all below zero: every way the search can go."""
    pages = 2100
    x = with_summaries(long_inputs(4, 2, 16, [16 * pages - 3], [new], seed=7), 64, seed=8)
    q = x["q"].clone()
    q[:] = 0
    q[:, :, 0] = 1.0  # the score is the first code times the scale
    x["q"] = q
    rng = np.random.default_rng(9)
    place = np.zeros(x["codes"].shape[0], int)
    place[x["table"][0, :pages]] = np.arange(pages)
    x["codes"][:], x["codes"][:, :, 0] = 0, 1
    scale = {"ascending": 1.0 + place, "descending": 1e4 - place, "one": np.full(len(place), 3.0),
             "two": rng.integers(1, 3, len(place)), "huge": 10.0 ** rng.uniform(-37, 36, len(place)),
             "negative": 1.0 + rng.random(len(place))}[kind]
    x["scale"][:] = np.asarray(scale, np.float32)[:, None]
    if kind == "negative":
        x["codes"][:, :, 0] = -5
    if kind == "huge":
        x["codes"][:, :, 0] = rng.choice([-3, 1, 2], len(place))[:, None]
    sel, err = run_select(x)
    assert not err
    np.testing.assert_array_equal(sel, want_select(x)[0])


@pytest.mark.parametrize("new", [1, 12])
@pytest.mark.parametrize("most", [1e-3, 1e-40, np.inf])
@pytest.mark.parametrize("top", [20, 64])
def test_selection_where_most_scores_lie_far_below_the_best(new, most, top):
    """A few small (or infinite) scores above zero, the others below it by factors of up to 1e6 of the largest."""
    pages = 2100
    x = with_summaries(long_inputs(4, 2, 16, [16 * pages - 3], [new], seed=17), top, seed=18)
    q = x["q"].clone()
    q[:] = 0
    q[:, :, 0] = 1.0
    x["q"] = q
    rng = np.random.default_rng(19)
    n = x["codes"].shape[0]
    good = rng.random(n) < 0.005  # (some ten pages: fewer than are taken)
    far = np.where(rng.random(n) < 0.2, rng.uniform(-1, 6, n), rng.uniform(5, 6, n))
    x["codes"][:], x["codes"][:, :, 0] = 0, np.where(good, 1, -1)[:, None]
    # the first head's rest below zero, the second's some at zero too
    x["codes"][:, 1, 0][~good & (rng.random(n) < 0.5)] = 0
    low = (most if 0 < most < np.inf else 1e-3) / 127 * 10.0 ** far
    x["scale"][:] = np.where(good, most / 127 * (1 - rng.random(n) / 8), low).astype(np.float32)[:, None]
    sel, err = run_select(x)
    assert not err
    np.testing.assert_array_equal(sel, want_select(x)[0])


# tiles' lists go by windows of 1024 (one head a KV head), 2048 and 4096 pages; a group's by 24576
@pytest.mark.parametrize("Hq,Hkv,page,own,new,top", [
    (1, 1, 16, [18000, 40], [140, 1], 20), (2, 1, 16, [36000], [70], 30), (4, 1, 16, [70000], [40], 9),
    (2, 1, 16, [24576 * 16 + 900], [5], 40), (1, 1, 16, [24576 * 16 + 900, 30], [2, 3], 12)])
def test_attention_over_lists_of_many_pages(Hq, Hkv, page, own, new, top):
    x = long_inputs(Hq, Hkv, page, own, new, seed=top)
    sel = some_selection(x, page, top, seed=top)
    out, lse, err = run_page_attn(x, sel)
    assert not err
    check_page_attn(x, sel, out, lse)


def test_unions_too_large_for_a_group_go_row_by_row():
    x = long_inputs(1, 1, 16, [16 * 3700, 900, 500], [3, 40, 1], seed=3)
    sel = some_selection(x, 16, 512, seed=4)
    out, lse, err = run_page_attn(x, sel)
    assert not err
    check_page_attn(x, sel, out, lse)


@pytest.mark.parametrize("Hq,Hkv", [(8, 8), (8, 4), (16, 4), (10, 2), (16, 2)])
def test_every_number_of_rows(Hq, Hkv):
    """1 .. 2 tiles and a bit: groups of one and two warps a stream, single tiles, pairs."""
    per = 128 // (Hq // Hkv)
    for new in (2, 3, 4, 5, 8, 16, 17, 32, 33, per - 1, per, per + 1, 2 * per, 2 * per + 1):
        x = attn_inputs(Hq, Hkv, 16, 37, [new + 75, new, new + 200], [new, min(new, 3), 1], pad=1, seed=new)
        sel = some_selection(x, 16, 7, seed=new)
        out, lse, err = run_page_attn(x, sel)
        assert not err
        check_page_attn(x, sel, out, lse)


@pytest.mark.parametrize("top,page", [(1, 16), (2, 128), (5, 32)])
def test_prompts_of_several_tiles_cut_between_the_runs(top, page):
    x = attn_inputs(8, 2, page, 100, [700, 900], [650, 333], pad=3, seed=top)
    sel = some_selection(x, page, top, seed=top + 1)
    out, lse, err = run_page_attn(x, sel)
    assert not err
    check_page_attn(x, sel, out, lse)


@pytest.mark.parametrize("new", [1, 4, 60])
def test_rows_that_take_no_page_at_all(new):
    x = attn_inputs(8, 2, 16, 50, [100, 200], [new, new], seed=5)
    sel = np.full((2 * new, 2, 6), -1, np.int32)
    out, lse, err = run_page_attn(x, sel)
    assert not err and (out == 0).all() and np.isneginf(lse).all()
    sel[new:, 1] = [0, 1, 2, -1, -1, -1]
    out, lse, err = run_page_attn(x, sel)
    assert not err
    check_page_attn(x, sel, out, lse)


@pytest.mark.parametrize("new", [1, 3, 80])
def test_a_longer_bound_on_rows_changes_nothing(new):
    x = attn_inputs(8, 2, 16, 50, [100, 200, 90], [new, new, 1], seed=6)
    sel = some_selection(x, 16, 6, seed=7)
    for bound in (new, 9, 100, 4000):
        if bound < new:
            continue
        out, lse, err = run_page_attn(x, sel, max_new=bound)
        assert not err
        check_page_attn(x, sel, out, lse)
    y = selection_inputs(8, 2, 16, 50, [100, 200, 90], [new, new, 1], 5, seed=6)
    for bound in (new, 9, 4000):
        if bound >= new:
            sel, err = run_select(y, max_new=bound)
            assert not err
            np.testing.assert_array_equal(sel, want_select(y)[0])


@pytest.mark.parametrize("new", [1, 4, 60])
def test_pages_past_four_gigabytes(new):
    """The same pages behind some 2^31 elements of others give the same results."""
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    x = selection_inputs(8, 8, 64, 100, [700, 300], [new, 1], 5, seed=70)
    few, off = x["k"].shape[0], (1 << 32) // (8 * 64 * 256) + 7
    y = dict(x, prefix=x["prefix"] + off, table=np.where(x["table"] >= 0, x["table"] + off, -1).astype(np.int32),
             codes=np.zeros((off + few, 8, 128), np.int8), scale=np.zeros((off + few, 8), np.float32))
    y["codes"][off:], y["scale"][off:] = x["codes"], x["scale"]
    for n in "kv":
        y[n] = torch.empty((off + few, 8, 64, 128), dtype=torch.bfloat16, device="cuda")
        y[n][off:] = x[n]
    sel, err = run_select(y)
    assert not err
    np.testing.assert_array_equal(sel, want_select(x)[0])
    out, lse, err = run_page_attn(y, sel)
    assert not err
    check_page_attn(x, sel, out, lse)
    ctx, pool = make(8, 8, 1), H.PagePool(y["k"], y["v"])
    sums = H.allocate_summaries(ctx, pool)
    pages = np.unique(np.concatenate([x["prefix"][:1], x["table"][0, :4]]))
    slots = pages.astype(np.int64) * 64 + 63
    H.hsq_page_summaries(ctx, pool, sums, i64(slots + 64 * off))
    assert word(ctx) == set()
    want = P.page_summaries(host(x["k"]), slots, np.zeros((few, 8, 128), np.int8), np.zeros((few, 8), np.float32))
    check_summaries(sums.codes[off:].cpu().numpy(), host(sums.scale[off:]), want[0], want[1])


@pytest.mark.parametrize("most", [1, 4, 40])
def test_more_requests_than_a_block_has_threads(most):
    """1300 requests, the kernels that look through all of them in several rounds."""
    rng = np.random.default_rng(most)
    own = rng.integers(1, 120, 1300)
    new = np.minimum(own, rng.integers(1, most + 1, 1300) if most < 9 else np.where(rng.random(1300) < 0.03, most, 1))
    x = selection_inputs(2, 1, 16, 20, [int(n) for n in own], [int(n) for n in new], 4, pad=2, seed=most)
    sel, err = run_select(x)
    assert not err
    np.testing.assert_array_equal(sel, want_select(x)[0])
    out, lse, err = run_page_attn(x, sel)
    assert not err
    check_page_attn(x, sel, out, lse)


def test_calls_on_two_streams_at_once():
    """Each with its own context, workspace and outputs; the same pool."""
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    x = attn_inputs(8, 2, 16, 60, [400, 300], [90, 1], seed=8)
    sel = some_selection(x, 16, 9, seed=9)
    pool = H.PagePool(x["k"], x["v"])
    dev = [i32(x[n]) for n in ("q_start", "lens", "table")] + [i32(sel)]
    prefix = i32(x["prefix"])
    runs = []
    for _ in range(2):
        ctx = make(8, 2, 2)
        n = H.hsq_page_attn_workspace_size(ctx, pool, 91, 2, x["table"].shape[1], 60, 9, 90)
        runs.append((ctx, torch.cuda.Stream(), torch.full_like(x["q"], 7.0), torch.zeros(x["q"].shape[:2], device="cuda"),
                     torch.full((n,), 255, dtype=torch.uint8, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(5):
        for ctx, s, out, lse, ws in runs:
            H.hsq_page_attn(ctx, pool, x["q"], *dev, out, ws, prefix=prefix, prefix_len=60, max_new=90, lse=lse, stream=s)
    torch.cuda.synchronize()
    for ctx, _, out, lse, _ in runs:
        assert word(ctx) == set()
        check_page_attn(x, sel, host(out), host(lse))


def test_outputs_that_overlap_are_refused():
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    x = selection_inputs(8, 2, 16, 40, [60, 70], [1, 1], 5, seed=60)
    ctx, pool = make(8, 2, 2), H.PagePool(x["k"], x["v"])
    sums = H.PageSummaries(torch.from_numpy(x["codes"]).cuda(), torch.from_numpy(x["scale"]).cuda())
    ints = torch.zeros(1 << 16, dtype=torch.int32, device="cuda")
    sel, ws = ints[:20].view(2, 2, 5), ints[256:].view(torch.uint8)
    rest = dict(prefix=i32(x["prefix"]), prefix_len=40)
    args = (x["q"], i32(x["q_start"]), i32(x["lens"]))
    table = i32(x["table"])
    H.hsq_page_select(ctx, pool, sums, *args, table, sel, ws, **rest)
    bad_table = ints[: table.numel()].view(table.shape)
    for kw in (dict(table=bad_table, sel=sel, ws=ws), dict(table=table, sel=ints[300:320].view(2, 2, 5), ws=ws)):
        with pytest.raises(H.HSQError):
            H.hsq_page_select(ctx, pool, sums, *args, kw["table"], kw["sel"], kw["ws"], **rest)
    out = torch.zeros_like(x["q"])
    H.hsq_page_attn(ctx, pool, *args, table, sel, out, ws, **rest)
    with pytest.raises(H.HSQError):
        H.hsq_page_attn(ctx, pool, *args, table, sel, x["k"].view(-1)[: out.numel()].view(out.shape), ws, **rest)
    with pytest.raises(H.HSQError):
        H.hsq_page_attn(ctx, pool, *args, table, sel, out, ws, lse=out.view(torch.float32).view(-1)[:16].view(2, 8), **rest)
    with pytest.raises(H.HSQError):
        H.hsq_page_summaries(ctx, H.PagePool(x["k"], x["v"]),
                             H.PageSummaries(sums.codes, sums.codes.view(-1)[: sums.scale.numel() * 4].view(torch.float32).view(sums.scale.shape)),
                             i64([0]))
    torch.cuda.synchronize()
    assert word(ctx) == set()


# -- waits that run out -------------------------------------------------------------------------------

def attn_word(x, sel, ctx):
    """run_page_attn with the whole device error word"""
    import hierarchical_kv_cache_hsq_gb300 as H
    words, read = [], H.hsq_sync_status
    H.hsq_sync_status = lambda c, stream=None: words.append(read(c, stream)) or words[-1]
    try:
        out, lse, _ = run_page_attn(x, sel, ctx)
    finally:
        H.hsq_sync_status = read
    return out, lse, words[-1]


@pytest.mark.expects_wait
@pytest.mark.parametrize("role", ["LOAD", "MMA", "QUERY", "SOFTMAX", "FEW", "ALL"])
@pytest.mark.parametrize("own,new", [([300, 20, 60, 900], [200, 1, 9, 70]), ([400, 300], [1, 1]), ([400, 300], [4, 3]),
                                     ([500], [40])])
def test_a_wait_that_runs_out_ends_the_call_and_no_more(role, own, new):
    import hierarchical_kv_cache_hsq_gb300 as H
    x = attn_inputs(8, 2, 16, 300, own, new, seed=len(own))
    sel = some_selection(x, 16, 12, seed=11)
    ctx = make(8, 2, len(own))
    tiles, few = max(new) > 8, min(new) <= 8
    acts = {"LOAD": tiles, "MMA": tiles, "QUERY": tiles, "SOFTMAX": tiles, "FEW": few, "ALL": True}[role]
    roles = ["LOAD", "MMA", "QUERY", "SOFTMAX", "FEW"] if role == "ALL" else [role]
    try:
        for _ in range(2):
            H.hsq_debug_set_fault(sum(getattr(H, "HSQ_FAULT_WAIT_" + r) for r in roles))
            t0 = time.monotonic()
            _, _, w = attn_word(x, sel, ctx)
            assert time.monotonic() - t0 < 20
            assert w == (H.HSQ_DEVERR_WAIT if acts else 0)
            H.hsq_debug_set_fault(0)
            out, lse, w = attn_word(x, sel, ctx)
            assert w == 0
            check_page_attn(x, sel, out, lse)
    finally:
        H.hsq_debug_set_fault(0)
    assert P is not None
