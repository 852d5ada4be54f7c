"""Paged serving on the GPU against the 64-bit oracle: block tables and slot
maps, the rotated paged write, the attention of a batch that shares a prefix,
and a run of the three together."""

import numpy as np
import pytest

from hsq_harness import ensure_built
from oracle import paged as P

pytestmark = pytest.mark.gpu

THETA = 1.0e6


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def make(Hq=8, Hkv=4, B=4, max_pos=4096):
    import hierarchical_kv_cache_hsq_gb300 as H
    return H.Context(H.make_config(Hq, Hkv, 16, 1, B, 16, 0, max_pos, theta=THETA))


def i32(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def i64(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, np.int64)).cuda()


def host(x):
    return x.float().cpu().numpy() if x.is_floating_point() else x.cpu().numpy()


def word(ctx):
    import hierarchical_kv_cache_hsq_gb300 as H
    w = H.hsq_sync_status(ctx)
    return {n for n, bit in (("PAGE", H.HSQ_DEVERR_PAGE), ("LEN", H.HSQ_DEVERR_LEN), ("POS", H.HSQ_DEVERR_POS)) if w & bit}


# -- tables ------------------------------------------------------------------------------

def run_tables(cached, fresh, free, used, table, rows, page, n_pages, base=0, stream=None):
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    B = len(cached)
    ctx = make(B=B)
    pool = H.allocate_pages(ctx, n_pages, page)
    d = dict(table=i32(table), slots=i64(np.full(rows, 77)), pos=i32(np.full(rows, 77)), q_start=i32(np.full(B + 1, 77)),
             lens=i32(np.full(B, 77)), used=i32([77]))
    args = (i32(cached), i32(fresh), i32(free), i32([used]))
    for _ in range(2):  # inputs are not written: the same again
        H.hsq_page_tables(ctx, pool, *args, d["table"], d["slots"], d["pos"], d["q_start"], d["lens"], d["used"], base=base)
    torch.cuda.synchronize()
    return {k: host(v) for k, v in d.items()}, word(ctx)


@pytest.mark.parametrize("B,page,hi,new,pad", [
    (1, 16, 0, 1, 0), (1, 128, 5, 300, 3), (2, 16, 16, 16, 0), (7, 32, 100, 3, 5), (33, 64, 200, 70, 0),
    (512, 16, 50, 2, 1), (513, 16, 40, 3, 0), (1500, 16, 30, 4, 9), (5, 16, 64, 0, 4), (4096, 16, 20, 1, 0)])
def test_tables(B, page, hi, new, pad):
    rng = np.random.default_rng(B * 1000 + page + new)
    cached, fresh = rng.integers(0, hi + 1, B), rng.integers(0, new + 1, B)
    if B > 2:
        cached[1], fresh[2] = page, page  # lengths that end a page
    n_pages = int((-(-(cached + fresh) // page)).sum()) + 3
    ids = rng.permutation(n_pages)
    table = np.full((B, int((-(-(cached + fresh) // page)).max()) + 1), -1)
    at = 0
    for b in range(B):
        n = -(-int(cached[b]) // page)
        table[b, :n] = ids[at: at + n]
        at += n
    rows = int(fresh.sum()) + pad
    rows = max(rows, 1)
    want = P.page_tables(cached, fresh, ids, at, table, rows, page, n_pages, base=1000)
    got, err = run_tables(cached, fresh, ids, at, table, rows, page, n_pages, base=1000)
    assert err == want["err"] == set()
    for k in got:
        np.testing.assert_array_equal(got[k].reshape(-1), np.asarray(want[k]).reshape(-1), err_msg=k)


@pytest.mark.parametrize("cached,fresh,free,used,width,rows,n_pages", [
    ([0, 20], [40, 20], [1, 2], 0, 4, 60, 5),         # the list runs out inside a request
    ([0, 0], [20, 3], [1, 99, -4], 0, 2, 23, 4),      # ids outside the pool
    ([30, 0], [10, 20], [0, 1, 2, 3], 0, 2, 30, 5),   # past the table's width
    ([1, 2], [9, 9], [0, 1], 0, 2, 12, 5),            # more rows than given
    ([-5, 3], [2, -1], [0, 1, 2], 0, 2, 4, 5),        # negative lengths
    ([0], [1], [0, 1], 7, 2, 1, 5),                   # *used past the list
    ([0], [1], [0, 1], -2, 2, 1, 5),
    ([2 ** 31 - 1, 5], [1, 2 ** 31 - 1], [0, 1, 2, 3], 0, 3, 40, 5),
])
def test_tables_refuse_what_does_not_fit(cached, fresh, free, used, width, rows, n_pages):
    table = np.full((len(cached), width), 3, np.int32)
    want = P.page_tables(cached, fresh, free, used, table, rows, 16, n_pages)
    got, err = run_tables(cached, fresh, free, used, table, rows, 16, n_pages)
    assert err == want["err"] and err
    for k in got:
        np.testing.assert_array_equal(got[k].reshape(-1), np.asarray(want[k]).reshape(-1), err_msg=k)


# -- write -----------------------------------------------------------------------------------

@pytest.mark.parametrize("Hq,Hkv,page,dtype,fused,rows", [
    (4, 2, 16, "bf16", True, 1), (8, 8, 32, "f32", False, 5), (16, 8, 64, "bf16", False, 33),
    (40, 8, 128, "f32", True, 70), (64, 8, 16, "bf16", True, 19), (5, 1, 16, "bf16", True, 130)])
def test_write(Hq, Hkv, page, dtype, fused, rows):
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    rng = np.random.default_rng(rows)
    max_pos = 1 << 20
    ctx = make(Hq, Hkv, 1, max_pos)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = torch.from_numpy(rng.standard_normal((rows, Hq + 2 * Hkv, 128)).astype(np.float32)).cuda().to(dt)
    q, k, v = x[:, :Hq], x[:, Hq: Hq + Hkv], x[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    n_pages = -(-rows // page) + 2
    base = rng.standard_normal((2, n_pages, Hkv, page, 128)).astype(np.float32)
    pool = H.PagePool(*[torch.from_numpy(b).cuda().bfloat16() for b in base])
    before = host(pool.k), host(pool.v)
    slots = rng.permutation(n_pages * page)[:rows].astype(np.int64)
    pos = rng.integers(0, max_pos, rows).astype(np.int32)
    pos[0] = max_pos - 1
    if rows > 4:
        pos[1], slots[2], pos[3], slots[4] = -1, -1, 0, -9
    q_out = torch.full((rows, Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    H.hsq_page_write(ctx, pool, q, k, v, i32(pos), i64(slots), q_out)
    assert word(ctx) == set()
    wq, wk, wv = P.page_write(*before, host(q), host(k), host(v), pos, slots, THETA, max_pos)
    # one rounding to bf16 (half a step, 2^-8 of the value), and cos and sin from float32 tables by
    # angle addition and the rotation: under 8 roundings of 2^-24 of |lo| + |hi| <= 12
    for got, want, was in ((host(pool.k), wk, before[0]), (host(pool.v), wv, before[1])):
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 12 * 2.0 ** -21).all()
        untouched = np.ones(was.shape, bool)
        for i in range(rows):
            if pos[i] >= 0 and slots[i] >= 0:
                untouched[slots[i] // page, :, slots[i] % page] = False
        np.testing.assert_array_equal(got[untouched], was[untouched])
    live = pos >= 0
    g = host(q_out)
    assert (np.abs(g - wq) <= 2.0 ** -8 * np.abs(wq) + 12 * 2.0 ** -21)[live].all()
    assert (g[~live] == 7.0).all()  # rows without a position are left as they were


def test_write_flags_bad_slots_and_positions_and_takes_no_queries():
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    ctx = make(4, 2, 1, 64)
    pool = H.allocate_pages(ctx, 2, 16)
    k = torch.randn(3, 2, 128, device="cuda")
    H.hsq_page_write(ctx, pool, None, k, k, i32([1, 2, 3]), i64([32, 1 << 40, 31]), None)
    assert word(ctx) == {"PAGE"}
    assert (host(pool.v)[1, :, 15] == host(k.bfloat16())[2]).all() and np.abs(host(pool.v)).sum(-1).astype(bool).sum() == 2
    H.hsq_page_write(ctx, pool, None, k, k, i32([64, 63, 5]), i64([0, 1, 2]), None)
    assert word(ctx) == {"POS"}
    _, wk, _ = P.page_write(np.zeros((2, 2, 16, 128)), np.zeros((2, 2, 16, 128)), np.zeros((3, 4, 128)), host(k), host(k),
                            [63, 63, 5], [0, 1, 2], THETA, 64)
    assert np.abs(host(pool.k)[0, :, :3] - wk[0, :, :3]).max() < 2 ** -7 * 5


# -- attention ------------------------------------------------------------------------------------

def attn_inputs(Hq, Hkv, page, prefix, own, new, pad=0, seed=0, stale=float("nan"), scale=1.5):
    """Requests with own[b] tokens in all, new[b] of them the rows of this step."""
    import torch
    rng = np.random.default_rng(seed)
    own, new = np.asarray(own), np.asarray(new)
    np_, ns = -(-prefix // page), -(-own // page)
    n_pages = int(np_ + ns.sum()) + 2
    ids = rng.permutation(n_pages)
    k = rng.standard_normal((n_pages, Hkv, page, 128)).astype(np.float32)
    v = rng.standard_normal((n_pages, Hkv, page, 128)).astype(np.float32)
    table = np.full((len(own), max(1, int(ns.max()) + 1)), -1, np.int32)
    at = np_
    used = np.zeros((n_pages, page), bool)
    for b in range(len(own)):
        table[b, : ns[b]] = ids[at: at + ns[b]]
        at += ns[b]
        for t in range(own[b]):
            used[table[b, t // page], t % page] = True
    for t in range(prefix):
        used[ids[t // page], t % page] = True
    k.transpose(0, 2, 1, 3)[~used] = stale  # what lies past a length
    v.transpose(0, 2, 1, 3)[~used] = stale
    rows = max(1, int(new.sum()) + pad)
    q = scale * rng.standard_normal((rows, Hq, 128))
    bf = lambda x: torch.from_numpy(np.asarray(x, np.float32)).cuda().bfloat16()  # noqa: E731
    return dict(q=bf(q), k=bf(k), v=bf(v), table=table, prefix=ids[:np_].astype(np.int32), prefix_len=prefix,
                q_start=np.concatenate([[0], np.cumsum(new)]).astype(np.int32), lens=own.astype(np.int32),
                max_new=max(1, int(new.max())), Hq=Hq, Hkv=Hkv)


def run_attn(x, ctx=None, lse=True, max_new=None, workspace=None):
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    ctx = ctx or make(x["Hq"], x["Hkv"], len(x["lens"]))
    pool = H.PagePool(x["k"], x["v"])
    out = torch.full_like(x["q"], 7.0)
    ls = torch.full(x["q"].shape[:2], 7.0, device="cuda") if lse else None
    mx = max_new or x["max_new"]
    if workspace is None:
        n = H.hsq_shared_attn_workspace_size(ctx, x["q"].shape[0], len(x["lens"]), x["prefix_len"], mx)
        workspace = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN as float: nothing of it is read
    H.hsq_shared_attn(ctx, pool, x["q"], i32(x["q_start"]), i32(x["lens"]), i32(x["table"]), out, workspace,
                      prefix=i32(x["prefix"]) if x["prefix_len"] else None, prefix_len=x["prefix_len"], max_new=mx, lse=ls)
    return host(out), None if ls is None else host(ls), word(ctx)


def check_attn(x, out, lse, live=None):
    """Bounds: logits are fp32 sums of 128 exact products (128 roundings of 2^-24 of their absolute sum;
    d bounds a logit's error), a weight's relative error is then at most 2 d plus its rounding to bf16 (2^-8) and
    the exponential's (2^-20), and the result is rounded to bf16 once more."""
    want, wl, spread, mass = P.shared_attn(host(x["k"]), host(x["v"]), host(x["q"]), x["q_start"], x["lens"], x["table"],
                                           x["prefix"], x["prefix_len"])
    rows = int(x["q_start"][-1])
    live = np.arange(len(want)) < rows if live is None else live
    d = mass * 2.0 ** -17
    tol = 2.0 ** -8 * np.abs(want) + spread * (2.0 ** -8 + 2 * d[..., None] + 2.0 ** -18) * 1.01
    bad = np.abs(out - want) > tol
    assert not bad[live].any(), (np.argwhere(bad & live[:, None, None])[:5], np.abs(out - want)[live].max())
    assert (out[~live] == 7.0).all()
    if lse is not None:
        fine = np.isfinite(wl) & live[:, None]
        assert (np.isneginf(lse) == np.isneginf(wl))[live].all()
        n_keys = x["prefix_len"] + max(1, int(np.max(x["lens"])))
        tol = d[fine] + n_keys * 2.0 ** -24 + 2.0 ** -20 * (1 + np.abs(wl[fine]))
        assert (np.abs(lse - np.where(fine, wl, 0))[fine] <= tol).all()
        assert (lse[~live] == 7.0).all()


HEADS = [(4, 4), (4, 2), (8, 2), (5, 1), (16, 2), (40, 8)]


@pytest.mark.parametrize("Hq,Hkv", HEADS)
@pytest.mark.parametrize("page", [16, 128])
def test_decode_rows(Hq, Hkv, page):
    own = [1, 2, 15, 16, 17, 64, 127, 128, 129, 300]
    x = attn_inputs(Hq, Hkv, page, 200, own, [1] * len(own), pad=3, seed=Hq + page)
    out, lse, err = run_attn(x)
    assert not err
    check_attn(x, out, lse)


@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 127, 128, 129, 255, 256, 257, 1000, 2100])
def test_prefix_lengths(prefix):
    x = attn_inputs(8, 2, 16, prefix, [3, 40, 200], [1, 1, 1], seed=prefix)
    out, lse, err = run_attn(x)
    assert not err
    check_attn(x, out, lse)


@pytest.mark.parametrize("own,new", [
    ([3, 4, 5], [3, 3, 3]), ([10, 1, 30], [2, 1, 3]), ([5, 0, 7], [1, 0, 2]), ([17, 33], [17, 33]), ([130], [130]),
    ([300, 5, 1], [257, 1, 1]), ([64, 200, 9, 1], [32, 100, 9, 1]), ([500], [3]), ([0, 0, 4], [0, 0, 4]), ([31], [31])])
@pytest.mark.parametrize("Hq,Hkv,page,prefix", [(8, 2, 16, 70), (5, 1, 32, 0), (2, 2, 64, 300), (16, 2, 128, 128)])
def test_several_rows_of_a_request(own, new, Hq, Hkv, page, prefix):
    x = attn_inputs(Hq, Hkv, page, prefix, own, new, pad=2, seed=len(own) + prefix)
    out, lse, err = run_attn(x)
    assert not err
    check_attn(x, out, lse)


def test_many_requests_share_tiles():
    rng = np.random.default_rng(5)
    own = rng.integers(1, 60, 150)
    x = attn_inputs(8, 2, 16, 333, own, np.minimum(own, rng.integers(0, 3, 150)), pad=1, seed=6)
    out, lse, err = run_attn(x)
    assert not err
    check_attn(x, out, lse)


@pytest.mark.parametrize("new", [1, 40])
def test_rows_that_see_nothing(new):
    x = attn_inputs(8, 2, 16, 0, [new, new + 20], [new, new], seed=3)
    x["lens"] = np.array([new - 1 if new > 1 else 0, new + 20], np.int32)  # below its row count: the first row sees nothing
    out, lse, err = run_attn(x)
    assert err == {"LEN"}
    assert (out[0] == 0).all() and np.isneginf(lse[0]).all()
    check_attn(x, out, lse)


@pytest.mark.parametrize("stale", [float("inf"), -float("inf"), 1e30, -3.0e38])
def test_what_lies_past_a_length_does_not_matter(stale):
    for new in ([1, 1, 1], [1, 20, 3]):
        x = attn_inputs(8, 2, 64, 75, [5, 70, 200], new, seed=9, stale=stale)
        out, lse, err = run_attn(x)
        assert not err
        check_attn(x, out, lse)


@pytest.mark.parametrize("new", [1, 50])
def test_pages_outside_the_pool_are_not_attended_to(new):
    x = attn_inputs(8, 2, 16, 100, [60, 90], [new, new], seed=11)
    x["table"][0, 1] = -1
    x["table"][1, 2] = x["k"].shape[0]
    x["prefix"][3] = -7
    out, lse, err = run_attn(x)
    assert err == {"PAGE"}
    check_attn(x, out, lse)


def test_every_page_missing():
    x = attn_inputs(8, 2, 16, 40, [20], [1], seed=12)
    x["table"][:] = -1
    x["prefix"][:] = 1 << 30
    out, lse, err = run_attn(x)
    assert err == {"PAGE"} and (out == 0).all() and np.isneginf(lse).all()


def test_lengths_that_contradict():
    x = attn_inputs(8, 2, 16, 40, [20, 30, 25], [1, 2, 1], seed=13)
    live = np.array([True, False, False, True])
    out, lse, err = run_attn(x, max_new=1)  # request 1 has more rows than max_new: not written
    assert err == {"LEN"}
    check_attn(x, out, lse, live)
    x = attn_inputs(8, 2, 16, 40, [20, 30, 25], [1, 2, 1], seed=13, stale=0.5)
    x["table"] = x["table"].clip(0)
    x["lens"][2] = 10 ** 6  # past its table: clamped to it
    out, lse, err = run_attn(x)
    assert err == {"LEN"}
    check_attn(dict(x, lens=np.array([20, 30, x["table"].shape[1] * 16])), out, lse)
    x["q_start"] = np.array([0, 3, 2, 4], np.int32)  # not ascending
    _, _, err = run_attn(x)
    assert err == {"LEN"}


def test_large_logits():
    x = attn_inputs(8, 2, 16, 500, [30, 200], [1, 20], seed=14, scale=30.0)
    out, lse, err = run_attn(x)
    assert not err
    check_attn(x, out, lse)


def test_without_lse_and_on_another_stream():
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    x = attn_inputs(8, 2, 32, 300, [30, 200, 9], [1, 20, 2], seed=15)
    ctx = make(8, 2, 3)
    a, _, _ = run_attn(x, ctx)
    b, none, _ = run_attn(x, ctx, lse=False)
    assert none is None and (a == b).all()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    pool, out = H.PagePool(x["k"], x["v"]), torch.full_like(x["q"], 7.0)
    ws = torch.empty(H.hsq_shared_attn_workspace_size(ctx, 23, 3, 300, 20), dtype=torch.uint8, device="cuda")
    args = [i32(x[k]) for k in ("q_start", "lens", "table", "prefix")]
    torch.cuda.synchronize()
    H.hsq_shared_attn(ctx, pool, x["q"], *args[:3], out, ws, prefix=args[3], prefix_len=300, max_new=20, stream=s)
    s.synchronize()
    assert (host(out) == a).all()  # the same bits: no order of arrival enters the result


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes: the last pages are read and written where they lie."""
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    Hkv, page = 8, 128
    n = (1 << 31) // (Hkv * page) - 1  # 2^31 - 1024 rows of 256 bytes: 512 GB would be the limit; take 24 GB of it
    n = min(n, 45000)
    ctx = make(16, Hkv, 2, 4096)
    pool = H.PagePool(*[torch.zeros((n, Hkv, page, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)])
    k = torch.randn(140, Hkv, 128, device="cuda").bfloat16()
    v = torch.randn(140, Hkv, 128, device="cuda").bfloat16()
    ids = np.array([n - 1, n - 3], np.int32)
    at = np.arange(140)
    slots = ids[at // page].astype(np.int64) * page + at % page
    q = torch.randn(140, 16, 128, device="cuda").bfloat16()
    q_out = torch.empty_like(q)
    H.hsq_page_write(ctx, pool, q, k, v, i32(at), i64(slots), q_out)
    assert (host(pool.v[n - 1])[:, 127] == host(v[127])).all() and (host(pool.v[n - 3])[:, 11] == host(v[139])).all()
    small_k, small_v = pool.k[[n - 1, n - 3]].contiguous(), pool.v[[n - 1, n - 3]].contiguous()
    x = dict(q=q_out[138:].contiguous(), k=pool.k, v=pool.v, table=np.array([[n - 1, n - 3]] * 2, np.int32),
             prefix=ids[:1], prefix_len=128, q_start=np.array([0, 1, 2], np.int32), lens=np.array([139, 140], np.int32),
             max_new=1, Hq=16, Hkv=Hkv)
    out, lse, err = run_attn(x, ctx)
    assert not err
    y = dict(x, k=small_k, v=small_v, table=np.array([[0, 1]] * 2, np.int32), prefix=np.array([0], np.int32))
    check_attn(y, out, lse)


# -- a run of the three -----------------------------------------------------------------------------

def test_a_serving_run_matches_dense_attention():
    """A shared prompt is written as a request of its own; then the batch's prompts, then decode steps
    from a captured graph, every step's attention against the dense oracle over all tokens so far."""
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    rng = np.random.default_rng(21)
    Hq, Hkv, page, B, shared = 8, 2, 16, 3, 37
    ctx = make(Hq, Hkv, B, 512)
    pool = H.allocate_pages(ctx, 40, page)
    free = i32(rng.permutation(40))
    used = i32([0])
    n = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda().bfloat16()  # noqa: E731
    pk, pv = np.zeros((40, Hkv, page, 128)), np.zeros((40, Hkv, page, 128))

    class Step:
        def __init__(self, B, width, rows, base, mx):
            self.B, self.rows, self.base, self.mx = B, rows, base, mx
            self.cached, self.fresh, self.lens = i32([0] * B), i32([0] * B), i32([0] * B)
            self.table, self.q_start, self.used = i32(np.full((B, width), -1)), i32([0] * (B + 1)), i32([0])
            self.slots, self.pos = i64([0] * rows), i32([0] * rows)
            self.q, self.k, self.v = n(rows, Hq, 128), n(rows, Hkv, 128), n(rows, Hkv, 128)
            self.q_rot, self.out = torch.zeros_like(self.q), torch.zeros_like(self.q)
            self.ws = torch.empty(H.hsq_shared_attn_workspace_size(ctx, rows, B, base, mx), dtype=torch.uint8, device="cuda")

        def run(self, prefix):
            H.hsq_page_tables(ctx, pool, self.cached, self.fresh, free, used, self.table, self.slots, self.pos,
                              self.q_start, self.lens, self.used, base=self.base)
            H.hsq_page_write(ctx, pool, self.q, self.k, self.v, self.pos, self.slots, self.q_rot)
            H.hsq_shared_attn(ctx, pool, self.q_rot, self.q_start, self.lens, self.table, self.out, self.ws,
                              prefix=prefix, prefix_len=self.base, max_new=self.mx)

        def check(self, prefix):
            nonlocal pk, pv
            pos, slots = host(self.pos), host(self.slots)
            q, pk, pv = P.page_write(pk, pv, host(self.q), host(self.k), host(self.v), pos, slots, THETA, 512)
            live = pos >= 0
            assert np.abs(host(pool.k) - pk).max() < 2 ** -7 * 6
            x = dict(q=self.q_rot, k=pool.k, v=pool.v, table=host(self.table), prefix=prefix, prefix_len=self.base,
                     q_start=host(self.q_start), lens=host(self.lens), Hq=Hq, Hkv=Hkv)
            out = host(self.out)
            out[~live] = 7.0
            check_attn(x, out, None)
            assert np.abs(host(self.q_rot)[live] - q[live]).max() < 2 ** -7 * 6

    first = Step(1, 3, shared, 0, shared)  # the shared prompt
    first.fresh.fill_(shared)
    first.run(None)
    first.check(np.zeros(0, np.int32))
    used.copy_(first.used)
    prefix = first.table[0].contiguous()
    step = Step(B, 4, 45, shared, 30)  # the requests' own prompts; one has none yet
    step.fresh.copy_(i32([30, 0, 12]))
    step.run(prefix)
    step.check(host(prefix))
    used.copy_(step.used)
    dec = Step(B, 4, B + 1, shared, 1)
    dec.cached.copy_(step.lens)
    dec.table.copy_(step.table)
    dec.fresh.fill_(1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        keep = pool.k.clone(), pool.v.clone(), dec.table.clone()
        dec.run(prefix)  # sets the kernels up outside the capture
    torch.cuda.current_stream().wait_stream(s)
    pool.k.copy_(keep[0]), pool.v.copy_(keep[1]), dec.table.copy_(keep[2])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dec.run(prefix)
    for t in range(5):
        for name, heads in (("q", Hq), ("k", Hkv), ("v", Hkv)):
            getattr(dec, name).copy_(n(B + 1, heads, 128))
        g.replay()
        torch.cuda.synchronize()
        dec.check(host(prefix))
        dec.cached.copy_(dec.lens)
        used.copy_(dec.used)
    assert host(dec.lens).tolist() == [35, 5, 17] and word(ctx) == set()


# -- refusals ----------------------------------------------------------------------------------------

def test_refusals():
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    ctx = make(8, 2, 2, 512)
    pool = H.allocate_pages(ctx, 4, 16)
    z = lambda n, dt=torch.int32: torch.zeros(n, dtype=dt, device="cuda")  # noqa: E731
    t = dict(cached=z(2), fresh=z(2), free_ids=z(4), used=z(1), table=z((2, 2)), slots=z(3, torch.int64), pos=z(3),
             q_start=z(3), lens=z(2), used_out=z(1))
    H.hsq_page_tables(ctx, pool, **t)
    for name, x in (("cached", z(2, torch.int64)), ("fresh", z(3)), ("table", z((3, 2))), ("slots", z(3)), ("pos", z(4)),
                    ("q_start", z(2)), ("used_out", z(2)), ("lens", torch.zeros(2, dtype=torch.int32)),
                    ("table", z((2, 4))[:, ::2])):
        with pytest.raises(ValueError):
            H.hsq_page_tables(ctx, pool, **dict(t, **{name: x}))
    for change in (dict(lens=t["cached"]), dict(used_out=t["used"]), dict(base=-1), dict(slots=z(0, torch.int64), pos=z(0))):
        with pytest.raises(H.HSQError) as e:
            H.hsq_page_tables(ctx, pool, **dict(t, **change))
        assert e.value.status == 1
    with pytest.raises(H.HSQError):  # more requests than the context has
        H.hsq_page_tables(ctx, pool, z(3), z(3), z(4), z(1), z((3, 2)), z(3, torch.int64), z(3), z(4), z(3), z(1))
    for shape in ((4, 2, 24, 128), (4, 2, 8, 128)):
        odd = H.PagePool(*[torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)])
        with pytest.raises(H.HSQError):
            H.hsq_page_tables(ctx, odd, **t)
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    q, k, pos, slots = b(3, 8, 128), b(3, 2, 128), z(3), z(3, torch.int64)
    w = dict(q=q, k=k, v=k, pos=pos, slots=slots, q_out=b(3, 8, 128))
    H.hsq_page_write(ctx, pool, **w)
    for change in (dict(k=k.half(), v=k.half()), dict(v=k.float()), dict(q=b(3, 4, 128)), dict(q=None), dict(q_out=None),
                   dict(slots=z(2, torch.int64)), dict(k=b(3, 2, 256)[..., ::2]), dict(k=b(3, 4, 128)[:, ::2]),
                   dict(q_out=b(3, 8, 256)[..., :128])):
        with pytest.raises(ValueError):
            H.hsq_page_write(ctx, pool, **dict(w, **change))
    odd = torch.zeros(3 * 260 + 4, dtype=torch.bfloat16, device="cuda")
    for change in (dict(k=odd[4: 4 + 780].view(3, 260)[:, :256].view(3, 2, 128)),):  # rows off 16 bytes
        with pytest.raises(H.HSQError):
            H.hsq_page_write(ctx, pool, **dict(w, **change))
    with pytest.raises(H.HSQError):  # every row the same: a stride of 0
        H.hsq_page_write(ctx, pool, **dict(w, k=b(1, 2, 128).expand(3, 2, 128)))
    with pytest.raises(ValueError):
        H.hsq_page_write(ctx, H.allocate_pages(make(4, 4), 4, 16), **w)
    ws = torch.empty(H.hsq_shared_attn_workspace_size(ctx, 3, 2, 20, 2), dtype=torch.uint8, device="cuda")
    a = dict(q=q, q_start=z(3), lens=z(2), table=z((2, 2)), out=b(3, 8, 128), workspace=ws, prefix=z(2), prefix_len=20,
             max_new=2)
    H.hsq_shared_attn(ctx, pool, **a)
    for change in (dict(q=q.float()), dict(out=b(2, 8, 128)), dict(lens=z(3)), dict(prefix=None), dict(prefix=z(1)),
                   dict(lse=z((3, 8))), dict(lse=z((3, 4), torch.float32)), dict(table=z((1, 2))),
                   dict(q=b(3, 8, 256)[..., :128])):
        with pytest.raises(ValueError):
            H.hsq_shared_attn(ctx, pool, **dict(a, **change))
    for change in (dict(max_new=0), dict(prefix_len=-1), dict(workspace=ws[:128]), dict(workspace=ws[1:])):
        with pytest.raises(H.HSQError):
            H.hsq_shared_attn(ctx, pool, **dict(a, **change))
    with pytest.raises(H.HSQError):
        H.hsq_shared_attn_workspace_size(ctx, 0, 1, 0, 1)
    assert word(ctx) == set()
