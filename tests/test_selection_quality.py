"""What the score finds: the page of one token that a head looks at, among tokens that it does not, is selected once the
token's logit stands out from the others' by what the page's mean and the sum over the heads take away."""

import numpy as np
import pytest

from oracle import paged as P

TOKENS, TAKEN = 8192, 1024


def one_row(page, r, z, rng):
    """Keys whose logits against each of r queries are normal with spread 1, but for one, which has z against the first; the
    row's selection of TAKEN tokens' pages by the oracle, and that token's page."""
    n = TOKENS // page
    q = rng.standard_normal((1, r, 128))
    q = (q * np.sqrt(128) / np.linalg.norm(q, axis=2, keepdims=True)).astype(np.float32)
    k = rng.standard_normal((n, page, 128))
    at = int(rng.integers(1, n - 2))  # neither the first page nor of the last two, which are always taken
    one, look = k[at, int(rng.integers(0, page))], q[0, 0] / np.sqrt(128)
    one += look * (z - one @ look)
    codes, scale = np.zeros((n, 1, 128), int), np.zeros((n, 1))
    for i in range(n):
        codes[i, 0], scale[i, 0] = P.summary(k[i])
    sel, err = P.page_select(codes, scale, q, [0, 1], [TOKENS], np.arange(n)[None, :], [], 0, page, TAKEN // page, 1, 2)
    assert not err
    return sel[0, 0], at


@pytest.mark.parametrize("r", [1, 4])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_a_token_that_stands_out_is_found(page, r):
    """A page's mean logit, summed over the heads, has spread sqrt(r / page) where no token stands out, and the one token adds
    z / page, with z = 12 sqrt(page r) twelve spreads.  One page in eight is taken: those 1.2 spreads above the mean, 1.4 where five of 61
    are taken by score.  Less one for the rounding to 8 bits (0.02 of a spread) and the threshold's own noise, 9.6 are left.
    The page's noise is one spread, and the other heads' logits of the token are z times cosines of spread 1 / sqrt(128) each: with three
    of them 1.9 spreads, 2.1 in all, which takes 9.6 away once in 400000 rows; 12 are tried."""
    rng = np.random.default_rng(page + r)
    for _ in range(12):
        sel, at = one_row(page, r, 12 * np.sqrt(page * r), rng)
        assert at in sel


def test_a_token_that_a_pages_mean_hides_is_found_by_smaller_pages():
    """At 30 spreads the token has nearly all of the softmax's weight (e^30 against 8192 e^0.5).  Pages of 16 add it as 30 / 16, 7.5 of
    their spreads of 1 / 4, 6.3 above what is taken; pages of 128, summed over four heads, as 30 / sqrt(128 4) = 1.3 of theirs, where 1.4
    are asked for: one row in two is lost (none of 24: once in 2^24)."""
    found = {}
    for page, r in ((16, 1), (128, 4)):
        rng = np.random.default_rng(1)
        found[page] = [at in sel for sel, at in (one_row(page, r, 30.0, rng) for _ in range(24))]
    assert all(found[16]) and not all(found[128])
