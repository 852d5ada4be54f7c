import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built library")
    config.addinivalue_line("markers", "slow: full-size workload check (minutes on CPU)")
    config.addinivalue_line("markers", "expects_wait: the test makes a bounded wait run out")


@pytest.fixture(autouse=True)
def _no_wait_ran_out(request, monkeypatch):
    """A GPU test that reads the device error word fails when a bounded wait ran out, whichever bits it looks at itself."""
    if request.node.get_closest_marker("gpu") is None or request.node.get_closest_marker("expects_wait") is not None:
        return
    import hierarchical_kv_cache_hsq_gb300 as H
    from hsq_harness import waits_checked
    monkeypatch.setattr(H, "hsq_sync_status", waits_checked(H.hsq_sync_status))


GOLDEN = os.path.join(os.path.dirname(os.path.abspath(__file__)), "golden")


def golden_path(name: str) -> str:
    return os.path.join(GOLDEN, name)
