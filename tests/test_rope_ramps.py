"""YaRN's ramp by the pair's index: against the oracle, numbers worked out by hand with 40 digits, and the ramp by turns;
the rotation that it makes, on the GPU; what make_rope and the tables refuse."""

import numpy as np
import pytest

from hsq_harness import ensure_built
from oracle import paged as P


@pytest.fixture(scope="module")
def H():
    ensure_built()
    import hierarchical_kv_cache_hsq_gb300 as H
    H.load_library()
    return H


# d(32) and d(1) of the two: 23.596 and 39.651, 10.472 and 22.513
@pytest.mark.parametrize("dims,theta,original,factor,first,last,ramp", [
    (128, 1e6, 32768, 4.0, 23, 40, {24: 0.005375321490790101503775, 30: 0.001064360981247001816321, 39: 6.490394320837028824360e-5}),
    (64, 1e4, 4096, 16.0, 10, 23, {11: 0.03912856978928671825664, 16: 0.005673076923076923076923, 22: 2.393837667360088386265e-4})])
def test_ramp_by_index_against_numbers_worked_out_by_hand(H, dims, theta, original, factor, first, last, ramp):
    w, _ = H.hsq_rope_frequencies(dims, theta)
    y, amp = H.hsq_rope_frequencies(dims, theta, "yarn_index", factor, original)
    assert (y[: first + 1] == w[: first + 1]).all()
    np.testing.assert_allclose(y[last:], w[last:] / factor, rtol=1e-15)
    for i, want in ramp.items():
        assert abs(y[i] / want - 1) < 1e-13
    assert abs(amp - (0.1 * np.log(factor) + 1)) < 1e-15
    turns, _ = H.hsq_rope_frequencies(dims, theta, "yarn", factor, original)
    differ = np.abs(y / turns - 1) > 1e-12
    assert (np.flatnonzero(differ) == np.arange(first + 1, last)).all()


@pytest.mark.parametrize("dims", [8, 64, 96, 128])
@pytest.mark.parametrize("factor", [1.0, 4.0, 31.5])
# (contexts so short or so long that the ramp lies at an end or past it, and one without width)
@pytest.mark.parametrize("theta,original,fast,slow", [(5e5, 8192.0, 30.0, 2.0), (1e4, 4.0, 32.0, 1.0), (10.0, 1e9, 32.0, 1.0),
                                                      (1e6, 100.0, 32.0, 1.0), (1e6, 32768.0, 2.0, 1.99)])
def test_ramp_by_index_matches_the_oracle(H, dims, factor, theta, original, fast, slow):
    got, amp = H.hsq_rope_frequencies(dims, theta, "yarn_index", factor, original, fast, slow)
    want, wamp = P.rope_frequencies(dims, theta, "yarn_index", factor, original, fast, slow)
    np.testing.assert_allclose(got, want, rtol=1e-13)
    assert abs(amp - wamp) < 1e-14


def test_ramp_by_index_refusals(H):
    ok = dict(scaling="yarn_index", factor=2.0, original=1000.0)
    H.hsq_rope_frequencies(**ok)
    for bad in (dict(theta=1.0), dict(theta=0.5), dict(beta_slow=0.0), dict(beta_slow=-1.0), dict(beta_slow=float("nan")),
                dict(beta_fast=1.0), dict(beta_fast=float("inf")), dict(original=0.0), dict(original=float("inf")), dict(factor=0.5)):
        with pytest.raises(H.HSQError):
            H.hsq_rope_frequencies(**dict(ok, **bad))


def test_frequencies_of_ones_own_go_with_no_scaling(H):
    """(they were taken, and the scaling, its factor and its amplitude dropped)"""
    for bad in (dict(scaling="yarn", factor=4.0, original=32768.0), dict(scaling="linear", factor=2.0), dict(factor=2.0),
                dict(theta=1e6), dict(original=10.0), dict(beta_fast=16.0), dict(beta_slow=2.0), dict(dims=128), dict(dims=4)):
        with pytest.raises(ValueError):
            H.make_rope(None, omega=[0.5, 0.25, 0.0, -1.0], max_pos=10, **bad)


def test_tables_without_numbers_are_refused(H):
    for omega, amp, most in (([1.0] * 4, 1e39, 10), ([1.0] * 4, -1e39, 10), ([1e305] * 4, 1.0, 1 << 24),
                             ([1.0, -1e308, 0.0, 1.0], 1.0, 1000)):
        with pytest.raises(H.HSQError):
            H.hsq_rope_table(omega, amp, most)
    assert np.isfinite(H.hsq_rope_table([1e300] * 4, 3e38, 1 << 20)).all()


@pytest.mark.gpu
def test_frequencies_of_ones_own(H):
    from test_gpu_paged import make
    for kw in (dict(), dict(dims=8)):
        rope = H.make_rope(make(4, 2, 1, 64), omega=np.array([0.5, 0.25, 0.0, -1.0]), max_pos=300, **kw)
        assert rope.dims == 8
        np.testing.assert_allclose(rope.table[1].cpu().numpy()[:4], np.cos([0.5, 0.25, 0.0, -1.0]), rtol=1e-6)
    assert H.make_rope(make(4, 2, 1, 64)).dims == 128


@pytest.mark.gpu
@pytest.mark.parametrize("dims,interleaved", [(128, False), (64, True)])
def test_write_with_the_ramp_by_index(H, dims, interleaved):
    import torch
    from test_gpu_paged import host, i32, i64, make
    from test_gpu_selection import word
    ctx = make(4, 2, 1, 64)
    kw = dict(dims=dims, theta=1e6, scaling="yarn_index", factor=4.0, original=32768.0)
    rope, (omega, amp) = H.make_rope(ctx, interleaved=interleaved, max_pos=131072, **kw), P.rope_frequencies(**kw)
    pos = np.array([0, 1, 300, 40000, 131071], np.int32)
    q, k = torch.randn(5, 4, 128, device="cuda"), torch.randn(5, 2, 128, device="cuda")
    pool, out = H.allocate_pages(ctx, 1, 16), torch.empty(5, 4, 128, dtype=torch.bfloat16, device="cuda")
    H.hsq_page_write(ctx, pool, q, k, k, i32(pos), i64(np.arange(5)), out, rope=rope)
    assert word(ctx) == set()
    for i, p in enumerate(pos):
        for got, x in ((host(out)[i], q), (host(pool.k)[0, :, i], k)):
            want = P.rotate(host(x)[i].astype(np.float64), int(p), omega, amp, interleaved)
            # one rounding to bf16, and under 8 roundings of 2^-24 of |a| + |b| <= 12, amp times
            assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + amp * 12 * 2.0 ** -21).all()
