"""Paged serving where lengths, sizes and arguments go past what a step has
room for: what is refused, and what the calls do with the rest."""

import numpy as np
import pytest

from hsq_harness import ensure_built
from oracle import paged as P
from test_gpu_paged import THETA, attn_inputs, check_attn, host, i32, i64, make, run_attn, run_tables, word

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def test_tables_refuse_sizes_past_their_sums():
    """Refused by the library before anything is launched: the buffers behind the sizes are small."""
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    ctx = make(B=2)
    pool = H.allocate_pages(ctx, 4, 16)
    t = [i32([0, 0]), i32([1, 1]), i32([0, 1]), i32([0]), i32(np.zeros((2, 1))), i64([0, 0]), i32([0, 0]), i32([0] * 3), i32([0, 0]),
         i32([0])]

    def call(rows, n_free):
        return ctx.lib.hsq_page_tables(ctx.handle, pool.ref, 2, 1, rows, n_free, 0, *[x.data_ptr() for x in t],
                                       torch.cuda.current_stream().cuda_stream)
    for rows, n_free in ((1 << 30, 2), (2 ** 31 - 1, 2), (2, 1 << 30), (2, 2 ** 31 - 1), (0, 2), (2, 0)):
        assert call(rows, n_free) == 1, (rows, n_free)
    assert call(2, 2) == 0 and word(ctx) == set() and t[5].tolist() == [0, 16]


@pytest.mark.parametrize("cached,fresh,rows", [([3], [50], 40), ([0, 7], [0, 41], 40), ([16, 1, 2], [50, 0, 0], 1), ([5, 6], [40, 1], 40)])
def test_a_request_of_more_rows_than_there_are_is_flagged(cached, fresh, rows):
    table = np.full((len(cached), 6), 2, np.int32)
    want = P.page_tables(cached, fresh, np.arange(8), 3, table, rows, 16, 8)
    got, err = run_tables(cached, fresh, np.arange(8), 3, table, rows, 16, 8)
    assert err == want["err"] == {"LEN"}
    for k in got:
        np.testing.assert_array_equal(got[k].reshape(-1), np.asarray(want[k]).reshape(-1), err_msg=k)


@pytest.mark.parametrize("cached,fresh,rows", [
    ([5, 40, 0, 3], [1, 30, 4, 1], 20), ([0, 0], [16, 16], 16), ([0, 0, 0], [16, 33, 5], 40), ([17], [100], 15), ([3, 16, 2], [2, 40, 0], 18),
    (list(range(700)), [2] * 700, 1001), (list(range(700)), [2] * 700, 1), (list(range(700)), [2] * 700, 1024)])
def test_tokens_without_a_row_count_as_not_brought(cached, fresh, rows):
    table = np.full((len(cached), 60), 2, np.int32)
    n = 8 + sum(-(-(c + f) // 16) for c, f in zip(cached, fresh))
    want = P.page_tables(cached, fresh, np.arange(n), 3, table, rows, 16, n)
    listed = np.diff(want["q_start"])
    assert listed.sum() == rows and (want["lens"] == np.asarray(cached) + listed).all()
    got, err = run_tables(cached, fresh, np.arange(n), 3, table, rows, 16, n)
    assert err == want["err"] == {"LEN"}
    for k in got:
        np.testing.assert_array_equal(got[k].reshape(-1), np.asarray(want[k]).reshape(-1), err_msg=k)


def test_a_step_without_room_for_all_rows_attends_to_what_is_stored():
    """Tables, write and attention with fewer rows than new tokens: each listed row sees the shared prefix and its
    own tokens up to its own position; the next step brings the rest."""
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    rng = np.random.default_rng(3)
    Hq, Hkv, page, B, shared, rows = 8, 2, 16, 3, 20, 30
    ctx = make(Hq, Hkv, B, 512)
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda().bfloat16()  # noqa: E731
    pool = H.PagePool(bf(24, Hkv, page, 128), bf(24, Hkv, page, 128))  # pages hold other tokens before they are written
    free, used = i32(rng.permutation(24)), i32([2])
    prefix = free[:2].contiguous()
    total = np.array([9, 40, 5])
    k, v = [bf(n, Hkv, 128) for n in total], [bf(n, Hkv, 128) for n in total]
    table, cached = i32(np.full((B, 4), -1)), np.zeros(B, np.int64)
    for step, listed in enumerate(([9, 21, 0], [0, 19, 5])):
        fresh = total - cached
        slots, pos, q_start, lens, used_out = i64([0] * rows), i32([0] * rows), i32([0] * (B + 1)), i32([0] * B), i32([0])
        H.hsq_page_tables(ctx, pool, i32(cached), i32(fresh), free, used, table, slots, pos, q_start, lens, used_out, base=shared)
        assert word(ctx) == ({"LEN"} if step == 0 else set())
        assert np.diff(host(q_start)).tolist() == listed
        # a program's rows: token cached[b] + j of request b, as q_start and pos say
        at = [(b, int(cached[b]) + j) for b in range(B) for j in range(listed[b])]
        ks, vs = torch.zeros(rows, Hkv, 128, device="cuda").bfloat16(), torch.zeros(rows, Hkv, 128, device="cuda").bfloat16()
        for i, (b, t) in enumerate(at):
            ks[i], vs[i] = k[b][t], v[b][t]
        q, rot = bf(rows, Hq, 128), torch.zeros(rows, Hq, 128, device="cuda").bfloat16()
        H.hsq_page_write(ctx, pool, q, ks, vs, pos, slots, rot)
        out, lse = torch.full_like(q, 7.0), torch.full((rows, Hq), 7.0, device="cuda")
        ws = torch.empty(H.hsq_shared_attn_workspace_size(ctx, rows, B, shared, rows), dtype=torch.uint8, device="cuda")
        H.hsq_shared_attn(ctx, pool, rot, q_start, lens, table, out, ws, prefix=prefix, prefix_len=shared, max_new=rows, lse=lse)
        assert word(ctx) == set()
        # dense attention over each row's true tokens, from what a write of every token one by one gives
        zero = np.zeros((24, Hkv, page, 128))
        seen = cached + listed
        for b in range(B):
            ids = host(table)[b]
            where = np.array([ids[t // page] * page + t % page for t in range(seen[b])], np.int64)
            _, wk, wv = P.page_write(zero, zero, np.zeros((seen[b], Hq, 128)), host(k[b])[: seen[b]], host(v[b])[: seen[b]],
                                     shared + np.arange(seen[b]), where, THETA, 512)
            for t, s in enumerate(where):
                assert np.abs(host(pool.k)[s // page, :, s % page] - wk[s // page, :, s % page]).max() < 2 ** -7 * 6
                assert (host(pool.v)[s // page, :, s % page] == wv[s // page, :, s % page]).all()
        x = dict(q=rot, k=pool.k, v=pool.v, table=host(table), prefix=host(prefix), prefix_len=shared,
                 q_start=np.concatenate([[0], np.cumsum(listed)]), lens=seen, Hq=Hq, Hkv=Hkv)
        check_attn(x, host(out), host(lse))
        cached = host(lens).astype(np.int64)
        assert (cached == seen).all()
        used = used_out
    assert (cached == total).all()


def test_outputs_that_overlap_are_refused():
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    z = lambda n, dt=torch.int32: torch.zeros(n, dtype=dt, device="cuda")  # noqa: E731
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731

    def refused(call, base, *changes):
        call(**base)
        for change in changes:
            with pytest.raises(H.HSQError) as e:
                call(**dict(base, **change))
            assert e.value.status == 1 and "overlap" in str(e.value)
    ctx = make(8, 2, 1, 512)
    pool = H.allocate_pages(ctx, 4, 16)
    t = dict(cached=z(1), fresh=z(1), free_ids=z(4), used=z(1), table=z((1, 2)), slots=z(1, torch.int64), pos=z(1),
             q_start=z(2), lens=z(1), used_out=z(1))
    both = z(8)
    refused(lambda **k: H.hsq_page_tables(ctx, pool, **k), t,
            dict(pos=t["lens"]), dict(used_out=t["lens"]), dict(pos=t["used_out"]), dict(lens=t["q_start"][1:]),
            dict(free_ids=both[:4], q_start=both[3:5]), dict(table=both[:2].view(1, 2), used_out=both[1:2]), dict(used_out=t["fresh"]),
            dict(slots=both[:2].view(torch.int64), lens=both[1:2]))
    H.hsq_page_tables(ctx, pool, **dict(t, used=both[:1], used_out=both[1:2], lens=both[2:3], q_start=both[3:5]))  # side by side
    w = dict(q=b(3, 8, 128), k=b(3, 2, 128), v=b(3, 2, 128), pos=z(3), slots=z(3, torch.int64) - 1, q_out=b(3, 8, 128))
    wide = b(3, 12, 128)
    rows = pool.k.view(-1)[: 3 * 8 * 128]
    refused(lambda **k: H.hsq_page_write(ctx, pool, **k), w,
            dict(q_out=w["q"]), dict(q=wide[:, :8], k=wide[:, 8:10], v=wide[:, 10:], q_out=wide.view(-1)[8 * 128: 8 * 128 + 3 * 1024].view(3, 8, 128)),
            dict(q_out=rows.view(3, 8, 128)), dict(k=rows[: 3 * 256].view(3, 2, 128)), dict(v=pool.v.view(-1)[: 3 * 256].view(3, 2, 128)))
    with pytest.raises(H.HSQError):  # keys and values in one place
        H.hsq_page_write(ctx, H.PagePool(pool.k, pool.k), **w)
    n = H.hsq_shared_attn_workspace_size(ctx, 3, 1, 20, 3)
    big = torch.zeros(n + 3 * 8 * 128 * 2, dtype=torch.uint8, device="cuda")
    a = dict(q=b(3, 8, 128), q_start=z(2), lens=z(1), table=z((1, 2)), out=b(3, 8, 128), workspace=big[:n], prefix=z(2), prefix_len=20,
             max_new=3, lse=torch.zeros(3, 8, device="cuda"))
    refused(lambda **k: H.hsq_shared_attn(ctx, pool, **k), a,
            dict(out=a["q"]), dict(out=big[n - 256: n - 256 + 6144].view(torch.bfloat16).view(3, 8, 128)),
            dict(lse=big[n - 96: n].view(torch.float32).view(3, 8)), dict(out=rows.view(3, 8, 128)),
            dict(lse=a["out"].view(-1)[:48].view(torch.float32).view(1, 24).view(3, 8)),
            dict(table=big[256: 264].view(torch.int32).view(1, 2)), dict(prefix=big[512: 520].view(torch.int32)))
    both_kv = H.PagePool(pool.k, pool.k)  # read only: one tensor for keys and values is fine
    H.hsq_shared_attn(ctx, both_kv, **a)
    assert word(ctx) == set()


def test_numbers_that_no_c_int_holds_are_refused():
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    ctx = make(8, 2, 1, 512)
    pool = H.allocate_pages(ctx, 4, 16)
    z = lambda n, dt=torch.int32: torch.zeros(n, dtype=dt, device="cuda")  # noqa: E731
    t = dict(cached=z(1), fresh=z(1), free_ids=z(4), used=z(1), table=z((1, 2)), slots=z(1, torch.int64), pos=z(1),
             q_start=z(2), lens=z(1), used_out=z(1))
    q = torch.zeros((3, 8, 128), dtype=torch.bfloat16, device="cuda")
    a = dict(q=q, q_start=z(2), lens=z(1), table=z((1, 2)), out=torch.zeros_like(q), max_new=3,
             workspace=torch.empty(H.hsq_shared_attn_workspace_size(ctx, 3, 1, 0, 3), dtype=torch.uint8, device="cuda"))
    for big in (1 << 32, (1 << 32) + 3, -(1 << 32), 1 << 70):
        for call in (lambda: H.hsq_page_tables(ctx, pool, **t, base=big),
                     lambda: H.hsq_shared_attn(ctx, pool, **dict(a, max_new=big)),
                     lambda: H.hsq_shared_attn_workspace_size(ctx, big, 1, 0, 3), lambda: H.hsq_shared_attn_workspace_size(ctx, 3, big, 0, 3),
                     lambda: H.hsq_shared_attn_workspace_size(ctx, 3, 1, big, 3), lambda: H.hsq_shared_attn_workspace_size(ctx, 3, 1, 0, big)):
            with pytest.raises(H.HSQError) as e:
                call()
            assert e.value.status == 1
        if big < 0:
            with pytest.raises(H.HSQError):
                H.hsq_shared_attn(ctx, pool, **a, prefix_len=big)
    H.hsq_page_tables(ctx, pool, **t, base=7)
    H.hsq_shared_attn(ctx, pool, **a)
    assert word(ctx) == set()


def test_a_pool_keeps_its_tensors():
    """The library holds their addresses: another tensor put in their place would go unread, the old one's memory being free."""
    import dataclasses
    import hierarchical_kv_cache_hsq_gb300 as H
    pool = H.allocate_pages(make(8, 2), 4, 16)
    for name in ("k", "v"):
        with pytest.raises(dataclasses.FrozenInstanceError):
            setattr(pool, name, pool.k.clone())
    assert pool._c.k == pool.k.data_ptr() and pool._c.v == pool.v.data_ptr() and (pool.n_pages, pool.page_n) == (4, 16)
    assert pool == pool and pool != H.PagePool(pool.k, pool.v)


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (4, 4), (8, 1)])
@pytest.mark.parametrize("own,new,width,lens", [
    ([32, 20], [10, 1], 2, [40, 20]),         # request 0 has 30 tokens stored, two of the ten new ones fit
    ([32, 20], [10, 4], 2, [70, 23]),         # none of its rows' own tokens fits
    ([64, 64], [40, 3], 4, [70, 64]), ([64, 64], [40, 3], 4, [2 ** 31 - 1, 65]),
    ([160, 16], [150, 1], 10, [170, 16]), ([160, 16], [150, 1], 10, [160 + 150, 16]), ([160, 16], [150, 1], 10, [2 ** 31 - 1, 2 ** 30 + 5])])
def test_a_table_too_short_for_a_length_moves_no_row(own, new, width, lens, Hq, Hkv):
    x = attn_inputs(Hq, Hkv, 16, 50, own, new, pad=1, seed=sum(own) + Hq, stale=0.25)
    x["table"] = x["table"][:, :width].copy().clip(0)
    x["lens"] = np.array(lens, np.int64).astype(np.int32)
    out, lse, err = run_attn(x)
    assert err == {"LEN"}
    # (a length that puts every row past the table gives the same limits as any longer one; the bound of lse goes by it)
    check_attn(dict(x, lens=np.minimum(lens, 16 * width + np.asarray(new))), out, lse)


@pytest.mark.parametrize("rows,B,max_new,most", [(1255, 256, 1000, 200 << 20), (5095, 4096, 1000, 700 << 20), (256, 256, 1, 80 << 20)])
def test_the_workspace_goes_by_the_rows(rows, B, max_new, most):
    """Decodes with one chunk of 1000 among them: no room is kept for a tile's rows of every request."""
    import hierarchical_kv_cache_hsq_gb300 as H
    ctx = make(32, 8, 1)
    assert H.hsq_shared_attn_workspace_size(ctx, rows, B, 4096, max_new) <= most


@pytest.mark.parametrize("Hq,Hkv,own,new,prefix", [
    (8, 2, [40, 9, 700, 33, 5, 1500, 64], [32, 5, 17, 1, 5, 31, 6], 300), (8, 2, [3000, 17, 2500, 600], [17, 5, 6, 32], 0),
    (4, 4, [128, 17, 900, 19, 2000], [128, 17, 33, 2, 100], 77), (8, 1, [50, 3, 700, 900], [16, 3, 9, 140], 100),
    (5, 1, [25, 700, 4, 30], [25, 13, 4, 4], 2000), (8, 2, list(range(20, 220, 2)), [5 + i % 28 for i in range(100)], 40)])
def test_parts_of_requests_of_unequal_rows_stay_in_the_workspace(Hq, Hkv, own, new, prefix):
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    x = attn_inputs(Hq, Hkv, 16, prefix, np.maximum(own, new), new, pad=1, seed=sum(new))
    ctx = make(Hq, Hkv, len(own))
    n = H.hsq_shared_attn_workspace_size(ctx, x["q"].shape[0], len(own), prefix, x["max_new"])
    room = torch.full((n + (1 << 20),), 255, dtype=torch.uint8, device="cuda")
    out, lse, err = run_attn(x, ctx, workspace=room[:n])
    assert not err and (room[n:] == 255).all()
    check_attn(x, out, lse)


def test_the_calls_go_to_the_current_stream():
    """The binding takes the stream's bare handle from torch: it has to be the one that torch's public Stream gives."""
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    from hierarchical_kv_cache_hsq_gb300 import _binding
    pool = H.allocate_pages(make(8, 2), 4, 16)
    side = torch.cuda.Stream()
    assert _binding._stream_on(pool, None) == torch.cuda.current_stream().cuda_stream
    with torch.cuda.stream(side):
        assert _binding._stream_on(pool, None) == torch.cuda.current_stream().cuda_stream == side.cuda_stream
    assert _binding._stream_on(pool, side) == side.cuda_stream != torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (8, 1), (5, 1)])
@pytest.mark.parametrize("new", [[1, 1, 1, 0], [3, 1, 2, 7]])
@pytest.mark.parametrize("prefix", [0, 33])
def test_few_rows_over_long_contexts_of_their_own(Hq, Hkv, new, prefix):
    x = attn_inputs(Hq, Hkv, 32, prefix, [20011, 4096, 9, 12000], new, pad=1, seed=Hq + prefix)
    out, lse, err = run_attn(x)
    assert not err
    check_attn(x, out, lse)


def test_a_decode_step_of_rows_all_over_the_pool():
    """The new token of each of 16 requests: a page and a position of its own, slots as a table gives them."""
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    rng = np.random.default_rng(8)
    B, Hq, Hkv, page, max_pos = 16, 8, 2, 16, 1 << 15
    ctx = make(Hq, Hkv, B, max_pos)
    cached = rng.integers(0, 300, B)
    have, need = -(-cached // page), -(-(cached + 1) // page)
    ids = rng.permutation(int(need.sum()) + 3)
    table, at = np.full((B, 20), -1), 0
    for b in range(B):
        table[b, : have[b]] = ids[at: at + have[b]]
        at += have[b]
    pool = H.allocate_pages(ctx, len(ids), page)
    t = dict(table=i32(table), slots=i64([0] * B), pos=i32([0] * B), q_start=i32([0] * (B + 1)), lens=i32([0] * B), used_out=i32([0]))
    H.hsq_page_tables(ctx, pool, i32(cached), i32([1] * B), i32(ids), i32([at]), **t, base=max_pos - 400)
    x = torch.from_numpy(rng.standard_normal((B, Hq + 2 * Hkv, 128)).astype(np.float32)).cuda().bfloat16()
    q, k, v = x[:, :Hq], x[:, Hq: Hq + Hkv], x[:, Hq + Hkv:]
    rot = torch.zeros((B, Hq, 128), dtype=torch.bfloat16, device="cuda")
    H.hsq_page_write(ctx, pool, q, k, v, t["pos"], t["slots"], rot)
    assert word(ctx) == set()
    zero = np.zeros(tuple(pool.k.shape))
    slots = host(t["slots"])
    assert len(set(slots // page)) == B and (host(t["pos"]) == max_pos - 400 + cached).all()
    wq, wk, wv = P.page_write(zero, zero, host(q), host(k), host(v), host(t["pos"]), slots, THETA, max_pos)
    for got, want in ((host(rot), wq), (host(pool.k), wk), (host(pool.v), wv)):
        # one rounding to bf16, and cos and sin from float32 tables: under 8 roundings of 2^-24 of |lo| + |hi| <= 12
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 12 * 2.0 ** -21).all()
