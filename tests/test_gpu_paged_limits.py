"""Paged serving where lengths, sizes and arguments go past what a step has
room for: what is refused, and what the calls do with the rest."""

import numpy as np
import pytest

from hsq_harness import ensure_built
from oracle import paged as P
from test_gpu_paged import i32, i64, make, run_tables, word

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
