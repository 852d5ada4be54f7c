"""What hsq_shared_attn does when a bounded wait of its main kernel runs out: it
ends, says so in the device error word, and leaves nothing behind that a later
call would meet."""

import time

import numpy as np
import pytest

from hsq_harness import ensure_built
from test_gpu_paged import attn_inputs, check_attn, make, run_attn

pytestmark = [pytest.mark.gpu, pytest.mark.expects_wait]

ROLES = ["LOAD", "MMA", "QUERY", "SOFTMAX", "FEW"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


@pytest.fixture
def fault():
    import hierarchical_kv_cache_hsq_gb300 as H
    yield H.hsq_debug_set_fault
    H.hsq_debug_set_fault(0)


def call(x, ctx):
    """-> out, lse, the whole device error word"""
    import hierarchical_kv_cache_hsq_gb300 as H
    words = []
    read = H.hsq_sync_status
    H.hsq_sync_status = lambda c, stream=None: words.append(read(c, stream)) or words[-1]
    try:
        out, lse, _ = run_attn(x, ctx)
    finally:
        H.hsq_sync_status = read
    return out, lse, words[-1]


# every kind of work at once; proposals over a prefix; decode; own tokens alone, in tiles that end inside 16 keys
SHAPES = [([300, 20, 60, 900, 2000], [200, 1, 9, 1, 70], 900), ([30, 77, 41], [3, 3, 3], 2000), ([700] * 20, [1] * 20, 517),
          ([333, 201], [300, 40], 0)]


@pytest.mark.parametrize("role", ROLES)
def test_a_wait_that_runs_out_ends_the_call_and_no_more(role, fault):
    import hierarchical_kv_cache_hsq_gb300 as H
    for own, new, prefix in SHAPES:
        x = attn_inputs(8, 2, 16, prefix, own, new, seed=len(own) + prefix)
        ctx = make(8, 2, len(own))
        tiles = prefix > 0 or max(new) > 4  # (a lone key tile goes to one of the two streams: QUERY then need not act)
        acts = {"LOAD": tiles, "QUERY": True if max(new) > 32 else None, "SOFTMAX": tiles, "MMA": max(new) > 32,
                "FEW": min(new) <= 4}[role]
        for _ in range(3):
            fault(getattr(H, "HSQ_FAULT_WAIT_" + role))
            t0 = time.monotonic()
            _, _, w = call(x, ctx)
            assert time.monotonic() - t0 < 20
            assert w in ([0, H.HSQ_DEVERR_WAIT] if acts is None else [H.HSQ_DEVERR_WAIT if acts else 0]), (own, new, prefix, w)
            fault(0)
            out, lse, w = call(x, ctx)
            assert w == 0
            check_attn(x, out, lse)


def test_all_of_them_at_once(fault):
    import hierarchical_kv_cache_hsq_gb300 as H
    own, new, prefix = SHAPES[0]
    x = attn_inputs(8, 2, 64, prefix, own, new, seed=5)
    ctx = make(8, 2, len(own))
    fault(sum(getattr(H, "HSQ_FAULT_WAIT_" + r) for r in ROLES))
    for _ in range(5):
        assert call(x, ctx)[2] == H.HSQ_DEVERR_WAIT
    fault(0)
    out, lse, w = call(x, ctx)
    assert w == 0
    check_attn(x, out, lse)


def test_a_graph_captured_without_a_fault_has_none(fault):
    import torch
    import hierarchical_kv_cache_hsq_gb300 as H
    from test_gpu_paged import host, i32
    x = attn_inputs(8, 2, 16, 300, [40, 9, 130], [1, 2, 100], seed=50)
    ctx = make(8, 2, 3)
    pool, out, lse = H.PagePool(x["k"], x["v"]), torch.zeros_like(x["q"]), torch.zeros(x["q"].shape[:2], device="cuda")
    n = H.hsq_shared_attn_workspace_size(ctx, x["q"].shape[0], 3, 300, 100)
    args = (i32(x["q_start"]), i32(x["lens"]), i32(x["table"]), out, torch.empty(n, dtype=torch.uint8, device="cuda"))
    prefix = i32(x["prefix"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        H.hsq_shared_attn(ctx, pool, x["q"], *args, prefix=prefix, prefix_len=300, max_new=100, lse=lse)
    fault(H.HSQ_FAULT_WAIT_LOAD)
    g.replay()
    assert H.hsq_sync_status(ctx) == 0
    check_attn(x, host(out), host(lse))
    assert np.isfinite(host(out)).all()
