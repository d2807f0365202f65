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


@pytest.fixture
def apart(monkeypatch, tmp_path):
    """A copy of the module to spoil; nothing is compiled."""
    copy = tmp_path / "_sparse_dispatch.so"
    copy.write_bytes(open(sparse.DISPATCH_PATH, "rb").read())
    monkeypatch.setattr(sparse, "DISPATCH_PATH", str(copy))
    monkeypatch.setattr(skl_build, "DISPATCH", str(copy))
    monkeypatch.setattr(sparse, "_dispatch", None)
    compiled = []

    def run(cmd, **kw):
        compiled.append(cmd)
        raise FileNotFoundError(cmd[0])
    monkeypatch.setattr(skl_build.subprocess, "run", run)
    return copy, compiled


def test_the_library_is_built_without_the_dispatch_module(apart):
    copy, compiled = apart
    copy.unlink()
    with pytest.warns(UserWarning, match="block-sparse calls are not available"):
        assert skl_build.build() == skl_build.LIB
    assert [c[0] for c in compiled] == ["g++"]
    with pytest.raises(FileNotFoundError):
        skl_build.build_dispatch()
    t = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(OSError, match="not built"):
        sparse.block_mass(t, t)


def test_a_module_of_another_pytorch_is_not_used(apart, monkeypatch):
    copy, compiled = apart
    skl_build.build_dispatch()
    assert not compiled
    with pytest.raises(FileNotFoundError):
        skl_build.build_dispatch(force=True)
    assert copy.exists()  # still good
    monkeypatch.setattr(torch, "__version__", "2.0.0")
    t = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(OSError, match="not built for this PyTorch"):
        sparse.block_mass(t, t)
    with pytest.raises(FileNotFoundError):
        skl_build.build_dispatch()
    assert len(compiled) == 2 and not copy.exists()
