"""The ctypes mirrors of hsq_rope, hsq_summaries and hsq_pages have the C layout of include/hsq.h."""

import ctypes

import pytest

from hierarchical_kv_cache_hsq_gb300 import _binding as B
from test_abi_layout import _c_layout


@pytest.mark.parametrize("cls,struct", [(B.hsq_rope, "hsq_rope"), (B.hsq_summaries, "hsq_summaries"), (B.hsq_pages, "hsq_pages")])
def test_struct_matches_the_header(tmp_path, cls, struct):
    names = [f[0] for f in cls._fields_]
    c = _c_layout(tmp_path, struct, names)
    assert c["size"] == ctypes.sizeof(cls)
    for n in names:
        assert c[n] == getattr(cls, n).offset, n
