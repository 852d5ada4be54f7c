"""The paged oracle against hand-worked cases, and the refusals of the paged
calls that need no GPU."""

import ctypes

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


def test_tables_by_hand():
    table = np.array([[7, -1, -1], [5, 6, -1], [-1, -1, -1]], np.int32)
    # 15 + 2 tokens: one new page; 32 + 1: one; 0 + 0: none
    got = P.page_tables([15, 32, 0], [2, 1, 0], [9, 3, 4, 8], 1, table, 5, 16, 10, base=100)
    assert got["table"].tolist() == [[7, 3, -1], [5, 6, 4], [-1, -1, -1]]
    assert got["q_start"].tolist() == [0, 2, 3, 3] and got["lens"].tolist() == [17, 33, 0]
    assert got["slots"].tolist() == [7 * 16 + 15, 3 * 16, 4 * 16, -1, -1]
    assert got["pos"].tolist() == [115, 116, 132, -1, -1] and got["used"] == 3 and not got["err"]


def test_tables_out_of_pages_and_rows():
    table = np.full((2, 2), -1, np.int32)
    got = P.page_tables([0, 0], [20, 3], [1, 99], 0, table, 22, 16, 4)
    assert got["table"].tolist() == [[1, -1], [-1, -1]] and got["used"] == 2
    assert got["err"] == {"PAGE", "LEN"} and got["q_start"].tolist() == [0, 20, 22]
    assert got["slots"][:16].tolist() == list(range(16, 32)) and (got["slots"][16:] == -1).all()


def test_attention_of_equal_scores_is_the_mean_and_of_nothing_is_zero():
    rng = np.random.default_rng(0)
    k, v = np.zeros((4, 2, 16, 128)), rng.standard_normal((4, 2, 16, 128))
    q = rng.standard_normal((3, 4, 128))
    table = np.array([[2, -1], [3, 9]], np.int32)
    out, lse, _, _ = P.shared_attn(k, v, q, [0, 2, 3], [3, 0], table, [1], 5)
    own = v[2, 0, :3]
    np.testing.assert_allclose(out[1, 0], np.concatenate([v[1, 0, :5], own]).mean(0))
    np.testing.assert_allclose(out[0, 0], np.concatenate([v[1, 0, :5], own[:2]]).mean(0))
    np.testing.assert_allclose(out[2, 3], v[1, 1, :5].mean(0))
    np.testing.assert_allclose(lse[:, 0], np.log([7, 8, 5]))
    out, lse, _, _ = P.shared_attn(k, v, q, [0, 2, 3], [2, 0], table, [], 0)
    assert (out[2] == 0).all() and np.isneginf(lse[2]).all()
    # a page outside the pool is not attended to
    out, lse, _, _ = P.shared_attn(k, v, q, [0, 0, 1], [0, 20], table, [], 0)
    np.testing.assert_allclose(lse[0], np.log(16))


def test_write_stores_rotated_keys_and_plain_values():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((2, 2, 128)), rng.standard_normal((2, 1, 128)), rng.standard_normal((2, 1, 128))
    pages = np.zeros((2, 1, 16, 128))
    q_out, pk, pv = P.page_write(pages, pages, q, k, v, [3, -1], [17, 2], 1e4, 100)
    np.testing.assert_array_equal(pv[1, 0, 1], v[0, 0])
    np.testing.assert_allclose(np.linalg.norm(pk[1, 0, 1]), np.linalg.norm(k[0, 0]))
    assert pk[0].any() == False and (q_out[1] == 0).all()  # noqa: E712
    c, s = np.cos(3.0), np.sin(3.0)  # frequency 0 turns by the position itself
    np.testing.assert_allclose(q_out[0, 1, [0, 64]], [q[0, 1, 0] * c - q[0, 1, 64] * s, q[0, 1, 64] * c + q[0, 1, 0] * s])


def test_null_context_is_refused(H):
    lib, p = H.load_library(), H._binding.hsq_pages(k=256, v=256, n_pages=1, page_n=16)
    ref, n = ctypes.byref(p), ctypes.c_size_t(0)
    assert lib.hsq_page_tables(None, ref, 1, 1, 1, 1, 0, *([None] * 11)) == 1
    assert lib.hsq_page_write(None, ref, 1, None, None, None, 0, 0, 0, 0, None, None, None, None) == 1
    assert lib.hsq_shared_attn(None, ref, 1, 1, 1, 0, 1, *([None] * 8), 0, None) == 1
    assert lib.hsq_shared_attn_workspace_size(None, 1, 1, 0, 1, ctypes.byref(n)) == 1
    assert b"context" in lib.hsq_last_error(None) or b"ctx" in lib.hsq_last_error(None)


def test_a_pool_off_the_gpu_is_refused(H):
    import torch
    x = torch.zeros(2, 1, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        H.PagePool(x, x)


def test_pages_struct_matches_the_header(tmp_path, H):
    from test_abi_layout import _c_layout
    cls = H._binding.hsq_pages
    names = [f[0] for f in cls._fields_]
    c = _c_layout(tmp_path, "hsq_pages", names)
    assert c["size"] == ctypes.sizeof(cls) and all(c[n] == getattr(cls, n).offset for n in names)
