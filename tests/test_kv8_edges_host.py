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
    p = bd.kv8_params(1, 1, 64, 128, 1 << 28, "f32")
    assert bd.kv8_attend_workspace_bytes(p, 1, 1023 * 128) > 0
    assert bd.kv8_attend_workspace_bytes(p, 1, 1024 * 128) == 0


@pytest.mark.parametrize("d,N,B,Q", [(128, 1 << 16, 1, 200000), (64, 1 << 20, 300, 4096), (256, 1 << 17, 7, 33333),
                                     (128, 1 << 28, 1, 1 << 18)])
def test_workspace_of_long_prompts_does_not_grow_with_them(d, N, B, Q):
    """bf16 prompts over more than 32K slots: the sums of a plan's CTAs, whatever the
    number of row tiles."""
    p = bd.kv8_params(64, 8, d, 128, N, "bf16")
    assert 0 < bd.kv8_attend_workspace_bytes(p, B, Q) <= 160 << 20


@pytest.mark.parametrize("n_q,n_kv,d,block,N,B,Q", [
    (64, 8, 128, 64, 1 << 20, 1, 2048), (64, 8, 128, 16, 1 << 20, 1, 32768), (64, 8, 128, 64, 1 << 15, 1, 1 << 15),
    (64, 8, 64, 16, 1 << 17, 12, 300), (14, 2, 256, 32, 1 << 18, 3, 777), (64, 8, 128, 64, 1 << 16, 4096, 1)])
def test_workspace_of_accumulated_weights_is_bounded(n_q, n_kv, d, block, N, B, Q):
    """The numbers per query row and sub-block of 32 slots (16 for blocks of 16) that
    weights go through take 512 MB at most, however long the cache; the rest is small."""
    p = bd.kv8_params(n_q, n_kv, d, block, N, "bf16")
    assert bd.kv8_attend_workspace_bytes(p, B, Q, True) <= (512 << 20) + (160 << 20)
    assert B * Q * n_q * (N // min(block, 32)) * 4 > 512 << 20   # (it would be more in one)
