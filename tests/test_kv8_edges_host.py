"""Workspace sizes of the 8-bit KV cache attention (host side, nothing launched)."""
import os

import pytest

from long_context_sparse_09_b200 import binding as bd


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(bd.LIB_PATH):
        from long_context_sparse_09_b200 import build
        build.build_library()
    return bd.lib()


def test_a_plan_counts_units_in_32_bits():
    """1024 row tiles over 2^28 slots are 2^31 units of 128 slots: a plan (and the
    workspace of its pieces) for one tile less, a CTA a tile beyond."""
    p = bd.kv8_params(1, 1, 64, 128, 1 << 28, "bf16")
    assert bd.kv8_attend_workspace_bytes(p, 1, 1023 * 256) > 0
    assert bd.kv8_attend_workspace_bytes(p, 1, 1024 * 256) == 0
