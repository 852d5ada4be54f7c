"""The device error word as the tests read it: every bit of the header has its
name in the package, and a wait that ran out does not pass unseen."""

import re

import pytest

import hierarchical_kv_cache_hsq_gb300 as H
from hsq_harness import waits_checked


def test_every_bit_of_the_word_is_exported():
    from hierarchical_kv_cache_hsq_gb300 import _binding
    with open(_binding.HEADER) as f:
        bits = dict(re.findall(r"\b(HSQ_DEVERR_[A-Z0-9_]+) = (\d+)", f.read()))
    assert "HSQ_DEVERR_WAIT" in bits
    for name, value in bits.items():
        assert getattr(H, name) == int(value), name


def test_a_wait_that_ran_out_fails_the_test_that_reads_the_word():
    assert waits_checked(lambda ctx, stream: H.HSQ_DEVERR_PAGE)(None) == H.HSQ_DEVERR_PAGE
    with pytest.raises(AssertionError):
        waits_checked(lambda ctx, stream: H.HSQ_DEVERR_PAGE | H.HSQ_DEVERR_WAIT)(None)
