"""Edges of the 8-bit KV cache path."""
import numpy as np
import pytest
import torch

from oracle import kv8
from long_context_sparse_09_b200 import binding as bd
from gpu_util import DEV
from test_gpu_kv8 import _clean_status, random_cache  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------- evict --
@pytest.mark.parametrize("NB,keep", [(3, 2), (40, 17), (40, 36), (1200, 300)])
def test_evict_ties_of_both_zeros(NB, keep):
    """0 and -0 are equal: of tied blocks the lower index stays."""
    block, d, recent = 16, 64, 1
    acc = torch.zeros(1, 2, NB)
    acc[..., ::2] = -0.0
    acc[0, 1] = -acc[0, 1]
    acc[..., 5::7] = 1.0
    acc[..., -1] = 1.0
    codes, exps = random_cache(1, 2, NB * block, d, block, NB)
    p = bd.kv8_params(2, 2, d, block, NB * block, "bf16")
    dc, de, da = codes.to(DEV), exps.to(DEV), acc.to(DEV)
    n = torch.tensor([NB * block], dtype=torch.int32, device=DEV)
    kept = torch.full((1, 2, keep), -7, dtype=torch.int32, device=DEV)
    acc_out, n_out = torch.empty_like(da), torch.empty_like(n)
    bd.csa_kv8_evict(p, keep, recent, da, n, dc[0], de[0], dc[1], de[1], kept, acc_out, n_out)
    ref, ref_acc, _ = kv8.evict(acc.numpy(), [NB * block], keep, recent, block)
    assert np.array_equal(kept.cpu().numpy(), ref)
    assert np.array_equal(acc_out.cpu().numpy(), ref_acc)
    for h in range(2):
        was = codes[0, 0, h].view(NB, block, d)[torch.from_numpy(ref[0, h]).long()]
        assert torch.equal(dc[0, 0, h].cpu().view(NB, block, d)[:keep], was)
