"""Attention over paged tokens where its work is divided differently: more row
tiles than lanes, requests cut over many SMs, every head ratio, batches of
long and short requests in any order, graphs and streams, and numbers that are
not finite.  Against the 64-bit oracle, with the bounds of test_gpu_paged."""

import numpy as np
import pytest

from hsq_harness import ensure_built
from test_gpu_paged import attn_inputs, check_attn, host, i32, make, run_attn, word

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def run_and_check(x, **kw):
    out, lse, err = run_attn(x, **kw)
    assert not err
    check_attn(x, out, lse)


def test_offsets_that_do_not_ascend_leave_no_row_to_two_requests():
    # rows [0, 4) belong to request 0 alone; requests 2 and 4 would begin below an earlier offset
    x = attn_inputs(8, 2, 16, 40, [20, 30, 25, 18, 40], [4, 0, 4, 0, 4], seed=21)
    x["q_start"] = np.array([0, 4, 0, 4, 0, 4], np.int32)
    x["q"] = x["q"][:4].contiguous()
    out, lse, err = run_attn(x, max_new=32)
    assert err == {"LEN"}
    check_attn(dict(x, q_start=np.array([0, 4, 4, 4, 4, 4], np.int32)), out, lse)
    # an offset past the rows spoils the requests beside it, not the later ones
    x = attn_inputs(8, 2, 16, 40, [20, 30, 25, 18], [1, 1, 1, 1], seed=22)
    x["q_start"][1] = 99
    out, lse, err = run_attn(x)
    assert err == {"LEN"}
    check_attn(dict(x, q_start=np.arange(5, dtype=np.int32)), out, lse, np.array([False, False, True, True]))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (4, 1), (10, 2), (8, 1)])
@pytest.mark.parametrize("new", [2, 9, 27])
def test_head_ratios(Hq, Hkv, new):
    own = [new, 20, 131]
    x = attn_inputs(Hq, Hkv, 32, 150, own, [new] * 3, pad=1, seed=Hq + new)
    out, lse, err = run_attn(x)
    assert err == ({"LEN"} if new > 20 else set())  # (more rows than tokens)
    check_attn(x, out, lse)


@pytest.mark.parametrize("Hq,Hkv,n", [(4, 4, 16), (4, 4, 17), (4, 4, 128), (4, 4, 129), (8, 2, 4), (8, 2, 5), (8, 2, 32), (8, 2, 33),
                                      (8, 2, 64), (8, 2, 65), (8, 1, 16), (8, 1, 17), (5, 1, 25), (5, 1, 26), (5, 1, 51)])
def test_rows_at_the_limits_of_a_tile(Hq, Hkv, n):
    run_and_check(attn_inputs(Hq, Hkv, 16, 77, [n, n + 50], [n, n], seed=n))


@pytest.mark.parametrize("B", [129, 160, 270])
def test_more_row_tiles_than_lanes(B):
    rng = np.random.default_rng(B)
    run_and_check(attn_inputs(8, 2, 16, 517, rng.integers(1, 20, B), [1] * B, seed=B))


def test_the_largest_batch():
    rng = np.random.default_rng(4)
    run_and_check(attn_inputs(4, 2, 16, 40, rng.integers(1, 5, 4096), [1] * 4096, seed=23))


@pytest.mark.parametrize("own,new", [([5000, 3001], [20, 9]), ([2049], [32]), ([4100, 17, 900], [5, 17, 30])])
@pytest.mark.parametrize("prefix", [0, 1000])
def test_requests_of_some_rows_cut_over_many_runs(own, new, prefix):
    run_and_check(attn_inputs(8, 2, 16, prefix, own, new, seed=own[0]))


@pytest.mark.parametrize("own,new,prefix,page", [
    ([300], [300], 5003, 16), ([3000], [70], 1, 64), ([1500, 200], [150, 130], 129, 16), ([129], [129], 4000, 128), ([700], [700], 0, 32)])
def test_long_requests_cut_over_many_runs(own, new, prefix, page):
    run_and_check(attn_inputs(8, 2, page, prefix, own, new, pad=1, seed=prefix))


@pytest.mark.parametrize("new", [[1, 100, 1, 1, 64, 3, 200, 1], [90, 1, 0, 1, 5, 0, 33, 1], [1, 1, 1, 1, 1, 1, 1, 300]])
@pytest.mark.parametrize("Hq,Hkv,prefix", [(8, 2, 300), (16, 2, 1111), (4, 4, 31)])
def test_long_and_short_requests_in_any_order(new, Hq, Hkv, prefix):
    rng = np.random.default_rng(len(new) + prefix)
    own = np.asarray(new) + rng.integers(0, 400, len(new))
    run_and_check(attn_inputs(Hq, Hkv, 16, prefix, own, new, pad=2, seed=prefix))


def test_a_first_row_behind_others():
    x = attn_inputs(8, 2, 16, 100, [20, 30], [1, 2], pad=6, seed=24)
    x["q_start"] = x["q_start"] + 4  # rows 0 .. 3 belong to no request
    out, lse, err = run_attn(x)
    assert not err
    check_attn(x, out, lse, np.array([False] * 4 + [True] * 3 + [False] * 2))


def test_no_new_rows_at_all():
    x = attn_inputs(8, 2, 16, 100, [20, 30], [0, 0], seed=25)
    out, lse, err = run_attn(x)
    assert not err and (out == 7.0).all() and (lse == 7.0).all()


@pytest.mark.parametrize("new", [1, 6, 40])
def test_a_number_that_is_none_shows_in_its_rows_only(new):
    x = attn_inputs(8, 2, 16, 100, [40, 60, 50], [new, new, new], seed=26)
    x["k"][int(x["table"][1, 0]), 1, 3, 5] = float("nan")  # a key of request 1's, of KV head 1
    x["q"][0, 0, 7] = float("nan")                          # a query of request 0's
    out, lse, err = run_attn(x)
    nan = np.zeros(lse.shape, bool)
    nan[new: 2 * new, 4:] = True
    nan[0, 0] = True
    assert not err and (np.isnan(lse) == nan).all() and (np.isnan(out).any(-1) == nan).all() and (np.isnan(out).all(-1) == nan).all()
    x["k"].nan_to_num_(0.0)
    x["q"].nan_to_num_(0.0)
    want, wl, _ = run_attn(x)
    check_attn(x, np.where(nan[..., None], want, out), np.where(nan, wl, lse))
    x["v"][int(x["prefix"][2]), 0, 1, 9] = float("inf")  # a value of the prefix: of every row, in this dim
    out, _, _ = run_attn(x)
    assert np.isinf(out[:, :4, 9]).all() and np.isfinite(out[:, 4:]).all()


def test_a_graph_goes_on_with_other_lengths():
    """One captured call over a padded batch, replayed as decode, proposals, a prompt's chunk and nothing."""
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    steps = [([20, 300, 1], [1, 1, 1]), ([30, 200, 9], [4, 1, 5]), ([250, 5, 40], [230, 5, 1]), ([9, 9, 9], [0, 0, 0]),
             ([400, 130, 260], [70, 130, 40])]
    rows = 256
    xs = [attn_inputs(8, 2, 16, 333, own, new, pad=rows - int(np.sum(new)), seed=30 + i) for i, (own, new) in enumerate(steps)]
    pages, width = max(x["k"].shape[0] for x in xs), max(x["table"].shape[1] for x in xs)
    ctx = make(8, 2, 3)
    pool = H.allocate_pages(ctx, pages, 16)
    q = torch.zeros((rows, 8, 128), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros((rows, 8), device="cuda")
    table, prefix, q_start, lens = i32(np.zeros((3, width))), i32(np.zeros(21)), i32(np.zeros(4)), i32(np.zeros(3))
    ws = torch.full((H.hsq_shared_attn_workspace_size(ctx, rows, 3, 333, 256),), 255, dtype=torch.uint8, device="cuda")
    call = lambda: H.hsq_shared_attn(ctx, pool, q, q_start, lens, table, out, ws, prefix=prefix, prefix_len=333,  # noqa: E731
                                     max_new=256, lse=lse)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for x in xs + xs[::-1]:
        n = x["k"].shape[0]
        pool.k[:n].copy_(x["k"])
        pool.v[:n].copy_(x["v"])
        t = np.full((3, width), -1, np.int32)
        t[:, : x["table"].shape[1]] = x["table"]
        table.copy_(i32(t))
        prefix.copy_(i32(x["prefix"]))
        q_start.copy_(i32(x["q_start"]))
        lens.copy_(i32(x["lens"]))
        q.copy_(x["q"])
        out.fill_(7.0)
        lse.fill_(7.0)
        g.replay()
        assert not word(ctx)
        check_attn(x, host(out), host(lse))


def test_two_calls_at_once():
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    xs = [attn_inputs(8, 2, 16, 900, [200, 100, 40], new, seed=40 + i) for i, new in enumerate(([1, 1, 1], [150, 1, 9]))]
    ctx = make(8, 2, 3)
    streams, todo = [torch.cuda.Stream() for _ in xs], []
    for x in xs:
        n = H.hsq_shared_attn_workspace_size(ctx, x["q"].shape[0], 3, 900, x["max_new"])
        todo.append((H.PagePool(x["k"], x["v"]), x["q"], i32(x["q_start"]), i32(x["lens"]), i32(x["table"]), torch.full_like(x["q"], 7.0),
                     torch.empty(n, dtype=torch.uint8, device="cuda"), i32(x["prefix"])))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, x, (pool, q, q_start, lens, table, out, ws, prefix) in zip(streams, xs, todo):
            H.hsq_shared_attn(ctx, pool, q, q_start, lens, table, out, ws, prefix=prefix, prefix_len=900, max_new=x["max_new"],
                              stream=s)
    torch.cuda.synchronize()
    assert not word(ctx)
    for x, t in zip(xs, todo):
        check_attn(x, host(t[5]), None)


def test_a_call_gives_the_same_bits_again():
    for own, new in (([300, 20, 700], [1, 1, 1]), ([300, 20, 700], [200, 3, 20])):
        x = attn_inputs(8, 2, 16, 2000, own, new, seed=27)
        first = run_attn(x)
        again = run_attn(x)
        assert (first[0] == again[0]).all() and (first[1] == again[1]).all()


def test_more_refusals(monkeypatch):
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    ctx = make(8, 2, 2, 512)
    pool = H.allocate_pages(ctx, 4, 16)
    z = lambda n, dt=torch.int32: torch.zeros(n, dtype=dt, device="cuda")  # noqa: E731
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    ws = torch.empty(H.hsq_shared_attn_workspace_size(ctx, 3, 2, 0, 2), dtype=torch.uint8, device="cuda")
    a = dict(q=b(3, 8, 128), q_start=z(3), lens=z(2), table=z((2, 2)), out=b(3, 8, 128), workspace=ws, max_new=2)
    w = dict(q=b(3, 8, 128), k=b(3, 2, 128), v=b(3, 2, 128), pos=z(3), slots=z(3, torch.int64), q_out=b(3, 8, 128))
    t = dict(cached=z(2), fresh=z(2), free_ids=z(4), used=z(1), table=z((2, 2)), slots=z(3, torch.int64), pos=z(3),
             q_start=z(3), lens=z(2), used_out=z(1))
    for size in ((3, 4097, 0, 1), (3, 2, (1 << 30) + 1, 1), (3, 2, -1, 1), (3, 2, 0, 0)):
        with pytest.raises(H.HSQError):
            H.hsq_shared_attn_workspace_size(ctx, *size)
    with pytest.raises(H.HSQError):  # queries rotated in place
        H.hsq_page_write(ctx, pool, **dict(w, q_out=w["q"]))
    with pytest.raises(H.HSQError):
        H.hsq_page_tables(ctx, pool, **t, base=1 << 30)
    big = torch.zeros(ws.numel(), dtype=torch.bfloat16, device="cuda")
    for change in (dict(out=a["q"]), dict(workspace=big, out=big[: 3 * 8 * 128].view(3, 8, 128))):
        with pytest.raises(H.HSQError):
            H.hsq_shared_attn(ctx, pool, **dict(a, **change))
    index = pool.index
    monkeypatch.setattr(torch.cuda, "current_device", lambda: index + 1)
    for call in (lambda: H.hsq_shared_attn(ctx, pool, **a), lambda: H.hsq_page_write(ctx, pool, **w),
                 lambda: H.hsq_page_tables(ctx, pool, **t)):
        with pytest.raises(ValueError):
            call()
    monkeypatch.undo()
    assert word(ctx) == set()


def test_the_first_call_of_a_process_may_be_captured():
    """Nothing that a call does once (limits, entry points, modules) breaks a capture."""
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    code = """
import numpy as np, torch
from test_gpu_paged import attn_inputs, check_attn, host, i32, make
import hierarchical_kv_cache_hsq_gb300 as H
x = attn_inputs(8, 2, 16, 300, [40, 9, 130], [1, 2, 100], seed=50)
ctx = make(8, 2, 3)
pool = H.PagePool(x["k"], x["v"])
out, lse = torch.zeros_like(x["q"]), torch.zeros(x["q"].shape[:2], device="cuda")
n = H.hsq_shared_attn_workspace_size(ctx, x["q"].shape[0], 3, 300, 100)
args = (i32(x["q_start"]), i32(x["lens"]), i32(x["table"]), out, torch.empty(n, dtype=torch.uint8, device="cuda"))
prefix = i32(x["prefix"])
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    H.hsq_shared_attn(ctx, pool, x["q"], *args, prefix=prefix, prefix_len=300, max_new=100, lse=lse)
g.replay()
torch.cuda.synchronize()
assert H.hsq_sync_status(ctx) == 0
check_attn(x, host(out), host(lse))
print("captured")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=os.path.dirname(here), capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, PYTHONPATH=os.pathsep.join([here, os.path.dirname(here)])))
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
