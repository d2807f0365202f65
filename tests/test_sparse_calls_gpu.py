"""Ways of calling the block-sparse operators (needs a B200)."""
import pytest
import torch
from torch.autograd import forward_ad

import attention_kl_divergence_fwd_b200 as skl
from attention_kl_divergence_fwd_b200 import sparse
from test_sparse_gpu import inputs, lists

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from attention_kl_divergence_fwd_b200 import build
    build.build()
    skl.load_library()


def test_forward_mode_derivatives_are_refused():
    q, k, v, do = (t.cuda() for t in inputs(1, 4, 2, 20, 130, 64, seed=41))
    idx = lists(1, 2, 20, 130, 2, seed=41).cuda()
    with forward_ad.dual_level():
        for j in range(3):
            args = [q, k, v]
            args[j] = forward_ad.make_dual(args[j], torch.ones_like(args[j]))
            with pytest.raises(NotImplementedError, match="qkv"[j] + " carries a forward-mode tangent"):
                sparse.sparse_attention(*args, idx, causal=True)
            with torch.no_grad(), pytest.raises(NotImplementedError):
                sparse.sparse_attention(*args, idx, causal=True)
            args[j].requires_grad_()
            with pytest.raises(NotImplementedError):
                sparse.sparse_attention(*args, idx, causal=True)
        qg = q.clone().requires_grad_()
        out = sparse.sparse_attention(qg, k, v, idx, causal=True)
        with pytest.raises(NotImplementedError, match="dout carries a forward-mode tangent"):
            torch.autograd.grad(out, qg, forward_ad.make_dual(do, torch.ones_like(do)))
    # Beside a dual level, tensors without a tangent are as ever.
    assert torch.equal(out.detach(), sparse.sparse_attention(q, k, v, idx, causal=True))
