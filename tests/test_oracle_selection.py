"""The long-context part of the paged oracle against hand-worked cases and
against the parts that it shares with others, the host calls of the rotation,
and the refusals that need no GPU."""

import ctypes

import numpy as np
import pytest

from hsq_harness import ensure_built
from oracle import paged as P
from oracle.hsq_oracle import rope


@pytest.fixture(scope="module")
def H():
    ensure_built()
    import hierarchical_kv_cache_hsq_gb300 as H
    H.load_library()
    return H


def test_rotation_of_the_whole_head_in_halves_is_the_contexts():
    x = np.random.default_rng(0).standard_normal((3, 128))
    w, amp = P.rope_frequencies(128, 1e6)
    for p in (0, 1, 777, 100000):
        np.testing.assert_allclose(P.rotate(x, p, w, amp, False), rope(x, np.full(3, p), 1e6), atol=1e-12)


def test_rotation_by_a_quarter_turn():
    x = np.arange(128.0)
    w = np.array([np.pi / 2, 0, 0, 0])
    y = P.rotate(x, 1, w, 2.0, False)
    assert np.allclose(y[[0, 4]], [-8, 0]) and np.allclose(y[[1, 5]], [2, 10]) and (y[8:] == x[8:]).all()
    y = P.rotate(x, 1, w, 1.0, True)
    assert np.allclose(y[:4], [-1, 0, 2, 3]) and (y[8:] == x[8:]).all()


@pytest.mark.parametrize("scaling", ["none", "linear", "base", "yarn"])
@pytest.mark.parametrize("dims", [8, 64, 96, 128])
@pytest.mark.parametrize("factor", [1.0, 4.0, 31.5])
def test_host_frequencies_match_the_oracle(H, scaling, dims, factor):
    got, amp = H.hsq_rope_frequencies(dims, 5e5, scaling, factor, 8192.0, 30.0, 2.0)
    want, wamp = P.rope_frequencies(dims, 5e5, scaling, factor, 8192.0, 30.0, 2.0)
    np.testing.assert_allclose(got, want, rtol=1e-13)
    assert abs(amp - wamp) < 1e-14
    if factor == 1.0:
        np.testing.assert_allclose(got, 5e5 ** (-2 * np.arange(dims // 2) / dims), rtol=1e-13)


def test_ramped_frequencies_keep_the_fast_and_divide_the_slow(H):
    w, _ = H.hsq_rope_frequencies(128, 1e6)
    y, amp = H.hsq_rope_frequencies(128, 1e6, "yarn", 4.0, 32768)
    turns = 32768 * w / (2 * np.pi)
    assert (y[turns >= 32] == w[turns >= 32]).all()
    np.testing.assert_allclose(y[turns <= 1], w[turns <= 1] / 4, rtol=1e-15)
    assert (np.diff(y) < 0).all() and abs(amp - 1.1386294361) < 1e-9


def test_rope_table_rows_make_every_angle(H):
    w, _ = H.hsq_rope_frequencies(64, 1e4, "linear", 2.0)
    t = H.hsq_rope_table(w, 1.25, 1000).astype(np.float64)
    assert t.shape == (256 + 4, 64)
    for p in (0, 1, 255, 256, 513, 999):
        hi, lo = t[256 + p // 256], t[p % 256]
        z = (hi[:32] + 1j * hi[32:]) * (lo[:32] + 1j * lo[32:])
        np.testing.assert_allclose(z, 1.25 * np.exp(1j * p * w), atol=4 * 2.0 ** -24)


def test_rope_refusals(H):
    for bad in (dict(dims=4), dict(dims=132), dict(dims=60), dict(dims=-8), dict(theta=0.0), dict(theta=float("inf")),
                dict(scaling="linear", factor=0.5), dict(scaling="base", factor=float("nan")),
                dict(scaling="yarn", factor=2.0), dict(scaling="yarn", factor=2.0, original=10.0, beta_fast=1.0)):
        with pytest.raises(H.HSQError):
            H.hsq_rope_frequencies(**bad)
    with pytest.raises(ValueError):
        H.hsq_rope_frequencies(scaling="other")
    for omega, amp, most in (([1.0] * 3, 1.0, 10), ([1.0] * 68, 1.0, 10), ([1.0] * 4, float("inf"), 10),
                             ([float("nan")] * 4, 1.0, 10), ([1.0] * 4, 1.0, 0), ([1.0] * 4, 1.0, (1 << 24) + 1)):
        with pytest.raises(H.HSQError):
            H.hsq_rope_table(omega, amp, most)


def test_summary_by_hand():
    k = np.zeros((2, 128))
    k[0, :3], k[1, :3] = [1, -2, 0.5], [3, 0, 0]  # sums 4, -2, 0.5
    codes, scale = P.summary(k)
    assert codes[:4].tolist() == [127, -64, 16, 0] and scale == 4 / 254  # -63.5 and 15.875
    assert P.summary(np.zeros((3, 128)))[1] == 0
    k[1, 7] = np.nan
    codes, scale = P.summary(k)
    assert (codes == 0).all() and scale == np.inf


def test_summaries_take_a_pages_last_row_of_the_step():
    rng = np.random.default_rng(1)
    k = rng.standard_normal((4, 2, 16, 128))
    codes, scale = np.full((4, 2, 128), 9), np.full((4, 2), 9.0)
    c, s, err = P.page_summaries(k, [14, 15, 48, 49, 50, -1, 1000], codes, scale)
    assert err == {"PAGE"} and (c[[1, 2]] == 9).all() and (s[[1, 2]] == 9).all()
    for h in range(2):
        assert (c[0, h] == P.summary(k[0, h])[0]).all() and (c[3, h] == P.summary(k[3, h, :3])[0]).all()


def test_selection_by_hand():
    # page p's summary points along dim 0 with weight p % 5; the query looks along it
    codes, scale = np.zeros((20, 1, 128), int), np.ones((20, 1))
    codes[:, 0, 0] = np.arange(20) % 5
    q = np.zeros((2, 2, 128), np.float32)
    q[:, :, 0] = 0.5
    table = np.arange(4, 20)[None, :]
    sel, err = P.page_select(codes, scale, q, [0, 2], [200], table, [0, 1, 2, 3], 60, 16, 6, 1, 2)
    # the second row sees 4 + 13 pages (0 .. 16), the first as many: of 1 .. 14 those of weight 4: 4, 9, 14
    assert not err and sel[1, 0].tolist() == [0, 4, 9, 14, 15, 16] and (sel[0] == sel[1]).all()
    sel, _ = P.page_select(codes, scale, q, [0, 2], [200], table, [0, 1, 2, 3], 60, 16, 7, 1, 2)
    assert sel[1, 0].tolist() == [0, 3, 4, 9, 14, 15, 16]  # a tie goes to the lower page
    sel, _ = P.page_select(codes, scale, q, [0, 2], [20], table, [0, 1, 2, 3], 60, 16, 7, 1, 2)
    assert sel[0, 0].tolist() == [0, 1, 2, 3, 4, 5, -1]
    scale[7] = np.inf
    codes[7] = 0
    sel, _ = P.page_select(codes, scale, q, [0, 2], [200], table, [0, 1, 2, 3], 60, 16, 4, 1, 2)
    assert sel[1, 0].tolist() == [0, 7, 15, 16]


def test_attention_over_all_pages_is_the_shared_one_and_entries_count_once():
    rng = np.random.default_rng(2)
    k, v = rng.standard_normal((2, 9, 2, 16, 128))
    q = rng.standard_normal((3, 4, 128))
    table = np.array([[2, 3, 8], [4, 5, 6]])
    args = (k, v, q, [0, 2, 3], [40, 33], table, [0, 1], 21)
    want = P.shared_attn(*args)
    sel = np.tile(np.arange(5), (3, 2, 1))
    got = P.page_attn(*args, sel)
    assert not got[4]
    for a, b in zip(got, want):
        np.testing.assert_allclose(a, b, rtol=1e-12)
    twice = np.tile([0, 1, 1, 2, 1, 2, 3, 4, 9, 4], (3, 2, 1))
    got = P.page_attn(*args, twice)
    assert got[4] == {"SEL"}
    np.testing.assert_allclose(got[0], want[0], rtol=1e-12)


def test_workspace_sizes_refuse(H):
    cfg = H.make_config(8, 2, 16, 1, 4, 16, 0, 64)
    lib, n = H.load_library(), ctypes.c_size_t(0)
    for fn in (lib.hsq_page_select_workspace_size, lib.hsq_page_attn_workspace_size):
        assert fn(None, 16, 1, 1, 1, 0, 1, 1, ctypes.byref(n)) == 1
    assert cfg.n_kv_heads == 2


def test_null_arguments_are_refused_before_any_gpu_call(H):
    from hierarchical_kv_cache_hsq_gb300 import _binding as B
    lib = H.load_library()
    pages, sums, rope_ = B.hsq_pages(), B.hsq_summaries(), B.hsq_rope()
    z = [None] * 9
    assert lib.hsq_page_write_rope(None, pages, rope_, 1, None, None, None, 0, 0, 0, 1, None, None, None, None) == 1
    assert lib.hsq_page_summaries(None, pages, sums, 1, None, None) == 1
    assert lib.hsq_page_select(None, pages, sums, *[1] * 8, *z[:7], 0, None) == 1
    assert lib.hsq_page_attn(None, pages, *[1] * 6, *z, 0, None) == 1
