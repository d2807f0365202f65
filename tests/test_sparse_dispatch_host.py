"""The PyTorch side of the block-sparse calls without a GPU."""
import pytest
import torch
from torch.autograd import forward_ad

from attention_kl_divergence_fwd_b200 import build as skl_build, sparse


@pytest.fixture(scope="module", autouse=True)
def built():
    skl_build.build()


def test_forward_mode_tangents_are_refused():
    t = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    idx = torch.zeros(1, 2, 8, 1, dtype=torch.int32)
    with forward_ad.dual_level():
        for j in range(3):
            args = [t, t, t]
            args[j] = forward_ad.make_dual(t.clone(), torch.ones_like(t))
            with pytest.raises(NotImplementedError, match="qkv"[j] + " carries a forward-mode tangent"):
                sparse.sparse_attention(*args, idx)
