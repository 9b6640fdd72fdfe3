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


@pytest.mark.parametrize("n_q,n_kv,d,block,N,B,Q", [
    (64, 8, 128, 64, 1 << 20, 1, 2048), (64, 8, 128, 16, 1 << 20, 1, 32768), (64, 8, 128, 64, 1 << 15, 1, 1 << 15),
    (64, 8, 64, 16, 1 << 17, 12, 300), (14, 2, 256, 32, 1 << 18, 3, 777), (64, 8, 128, 64, 1 << 16, 4096, 1)])
def test_workspace_of_accumulated_weights_is_bounded(n_q, n_kv, d, block, N, B, Q):
    """The numbers per query row and sub-block of 32 slots (16 for blocks of 16) that
    weights go through take 512 MB at most, however long the cache; the rest is small."""
    p = bd.kv8_params(n_q, n_kv, d, block, N, "bf16")
    assert bd.kv8_attend_workspace_bytes(p, B, Q, True) <= (512 << 20) + (160 << 20)
    assert B * Q * n_q * (N // min(block, 32)) * 4 > 512 << 20   # (it would be more in one)
