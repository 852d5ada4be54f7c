"""What one row of the attention over selected pages holds, or one of its pages, is nothing to the others: rows of no
token, and keys that are no numbers."""

import numpy as np
import pytest

from hsq_harness import ensure_built
from oracle import paged as P
from test_gpu_paged import attn_inputs, host, i64, make
from test_gpu_selection import (check_page_attn, check_summaries, run_page_attn, run_select, selection_inputs, some_selection,
                                want_select, word)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


# the last tile's rows, its first warp's among them, are not all of a token: 70 tokens are two tiles of 32 and 6 of a third
@pytest.mark.parametrize("Hq,Hkv,page,new", [(8, 2, 16, 70), (8, 2, 64, 34), (16, 2, 16, 17), (5, 1, 32, 55), (2, 2, 128, 135)])
@pytest.mark.parametrize("rest", [float("nan"), float("inf"), 2.0e4])
def test_rows_behind_a_request_change_nothing(Hq, Hkv, page, new, rest):
    """A tile's load of queries goes on behind its request's last row, into padding or another request."""
    x = attn_inputs(Hq, Hkv, page, 0, [1500, 300], [new, 1], pad=40, seed=new)
    sel = some_selection(x, page, 1500 // page, seed=new)
    q = x["q"].clone()
    q[new:] = 0.0
    want, lse = run_page_attn(dict(x, q=q), sel)[:2]
    q = q.clone()
    q[new:] = rest
    x["q"] = q
    got, glse, err = run_page_attn(x, sel)
    assert not err
    np.testing.assert_array_equal(got[:new], want[:new])
    np.testing.assert_array_equal(glse[:new], lse[:new])
    assert (got[new + 1:] == 7.0).all()


@pytest.mark.parametrize("new", [50, 333])
def test_what_an_earlier_call_left_in_shared_memory_changes_nothing(new):
    """With 5 heads a KV head a tile has 125 rows: the places of the other three are whatever a call of 4 heads, whose tiles
    have 128, left there."""
    y = attn_inputs(4, 1, 16, 0, [2000] * 8, [1500] * 8, seed=1)
    ysel = some_selection(y, 16, 3, seed=2)
    x = attn_inputs(5, 1, 16, 0, [1500] * 8, [new] * 8, seed=3)
    sel = some_selection(x, 16, 90, seed=4)
    got = []
    for rest in (0.0, float("nan"), float("inf"), -3.0e38):
        y["q"] = y["q"].clone().fill_(rest)
        run_page_attn(y, ysel)
        got.append(run_page_attn(x, sel)[:2])
    for out, lse in got[1:]:
        np.testing.assert_array_equal(out, got[0][0])
        np.testing.assert_array_equal(lse, got[0][1])
    check_page_attn(x, sel, *got[0])


@pytest.mark.parametrize("new", [1, 4, 60, 333])
@pytest.mark.parametrize("Hq,Hkv,page", [(8, 2, 16), (5, 1, 32), (2, 2, 64), (16, 2, 128)])
@pytest.mark.parametrize("key", [float("nan"), float("inf"), -3.3e38])
def test_a_key_that_gives_no_numbers_shows_in_the_rows_that_take_its_page_alone(new, Hq, Hkv, page, key):
    """Neighbouring rows share a tile and its products, but a page that a row does not take is not there for it.  (-3.3e38: its
    logits pass fp32's range.)"""
    x = attn_inputs(Hq, Hkv, page, 3 * page, [40 * page] * 2, [new] * 2, pad=3, seed=new + page)
    rng = np.random.default_rng(new)
    rows, top, r = 2 * new, 12, Hq // Hkv
    whole = 43 - -(-new // page) - 1  # pages that every row sees all of
    sel = np.full((rows + 3, Hkv, top), -1, np.int32)
    for i in range(rows):
        for h in range(Hkv):
            n = int(rng.integers(1, top - 1))
            sel[i, h, :n] = np.sort(rng.permutation(whole - 2)[:n])
    # one row alone takes page whole - 1, and some take page 2, of the prefix
    sel[int(rng.integers(0, new)), 0, top - 1] = whole - 1
    k = x["k"].clone()
    k[int(x["table"][0][whole - 4]), 0, page // 2] = key
    k[int(x["prefix"][2]), Hkv - 1, 1] = key
    out, lse, err = run_page_attn(dict(x, k=k), sel)
    assert not err
    takers = np.zeros((rows + 3, Hq), bool)
    takers[:new, :r] |= (sel[:new, 0] == whole - 1).any(-1)[:, None]
    takers[:, (Hkv - 1) * r:] |= (sel[:, Hkv - 1] == 2).any(-1)[:, None]
    assert takers.any() and (new == 1 or not takers[:rows].all())
    if np.isnan(key):
        assert np.isnan(out[takers]).all() and np.isnan(lse[takers]).all()
    assert np.isfinite(out[:rows][~takers[:rows]]).all()
    # the others: the oracle's bounds with any other key there
    quiet = (np.arange(rows + 3) < rows) & ~takers.any(1)
    check_page_attn(x, sel, np.where(quiet[:, None, None], out, 7.0), np.where(quiet[:, None], lse, 7.0), quiet)


@pytest.mark.parametrize("most", [1, 5, 40])
@pytest.mark.parametrize("length", [-1, 10 ** 6])
def test_the_length_of_a_request_without_rows_is_looked_at_too(most, length):
    x = selection_inputs(8, 2, 16, 40, [200, 100, 90], [most, 0, most], 5, seed=most)
    sel, err = run_select(x)
    assert not err
    out, lse, err = run_page_attn(x, sel)
    assert not err
    x["lens"][1] = length
    sel2, err = run_select(x)
    assert err == {"LEN"}
    np.testing.assert_array_equal(sel2, sel)
    np.testing.assert_array_equal(sel, want_select(x)[0])
    out2, lse2, err = run_page_attn(x, sel)
    assert err == {"LEN"}
    np.testing.assert_array_equal(out2, out)
    np.testing.assert_array_equal(lse2, lse)


@pytest.mark.parametrize("repeat", [1, 400])
def test_a_page_that_a_step_names_in_two_places_gets_codes_of_the_two(repeat):
    """Its codes and scale may be of either (of a row before a negative slot, and of a later one); the others are as ever."""
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    rng = np.random.default_rng(repeat)
    Hkv, n = 8, 3 * repeat
    pool = H.PagePool(*[torch.from_numpy(rng.standard_normal((n, Hkv, 16, 128)).astype(np.float32)).cuda().bfloat16()] * 2)
    slots = np.concatenate([[48 * i + 3, -1, 48 * i + 5, 48 * i + 31, 48 * i + 9, 48 * i + 40] for i in range(repeat)])
    ctx, none = make(Hkv, Hkv, 1), (np.zeros((n, Hkv, 128), np.int8), np.zeros((n, Hkv), np.float32))
    sums = H.allocate_summaries(ctx, pool)
    H.hsq_page_summaries(ctx, pool, sums, i64(slots))
    assert word(ctx) == set()
    codes, scale = sums.codes.cpu().numpy(), host(sums.scale)
    k, apart = host(pool.k), np.arange(0, n, 3)
    ways = [P.page_summaries(k, 16 * apart + last, *none)[:2] for last in (3, 5, 9)]
    assert np.logical_or.reduce([codes[apart] == c[apart] for c, _ in ways]).all()
    near = [np.abs(scale[apart] - s[apart]) <= s[apart] * 2.0 ** -22 for _, s in ways]
    assert np.logical_or.reduce(near).all()
    rest = np.delete(np.arange(n), apart)
    want = P.page_summaries(k, slots, *none)
    check_summaries(codes[rest], scale[rest], want[0][rest], want[1][rest])
