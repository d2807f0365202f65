"""Block-sparse attention without a GPU: refusals of the C entry points and of the Python
wrappers, and pins of the fp64 oracle (brute force, autograd, finite differences)."""
import math

import pytest
import torch

import attention_kl_divergence_fwd_b200 as skl
from attention_kl_divergence_fwd_b200 import build as skl_build, sparse
from oracle import (oracle_block_mass, oracle_block_select, oracle_fwd, oracle_sparse_attn,
                    selected_keys)

P = 1 << 12  # a fake, 16-byte aligned, non-null address: never dereferenced on these paths
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    skl_build.build()
    return skl.load_library()


def call_mass(lib, **kw):
    a = dict(q=P, k=P, lens=0, B=1, H=4, Hkv=2, nq=100, nk=200, d=64, scale=0.1, causal=1, lse=P,
             ws=0, wsb=0, mass=P, stream=0)
    a.update(kw)
    return lib.streamkl_block_mass(*a.values())


def call_select(lib, **kw):
    a = dict(mass=P, lens=0, B=1, Hs=2, nq=100, nk=200, causal=1, topk=4, first=1, last=1, idx=P,
             stream=0)
    a.update(kw)
    return lib.streamkl_block_select(*a.values())


def call_attn(lib, backward=False, **kw):
    head = dict(q=P, k=P, v=P)
    if backward:
        head.update(out=P, lse=P, dout=P)
    a = dict(idx=P, lens=0, B=1, H=4, Hkv=2, Hs=2, nq=100, nk=200, d=64, topk=4, scale=0.1,
             causal=1, ws=P, wsb=BIG)
    tail = dict(dq=P, dk=P, dv=P, stream=0) if backward else dict(out=P, lse=P, stream=0)
    args = {**head, **a}
    if not backward:
        args.update(tail)
        args.update(kw)
        return lib.streamkl_sparse_attn_fwd(*args.values())
    args.update({k: v for k, v in kw.items() if k in args})
    tail.update({k: v for k, v in kw.items() if k in tail})
    return lib.streamkl_sparse_attn_bwd(*args.values(), *tail.values())


def test_mass_refusals(lib):
    for kw in (dict(q=0), dict(k=0), dict(mass=0), dict(B=0), dict(nq=0), dict(nk=-1),
               dict(scale=float("nan")), dict(lse=0), dict(lse=0, ws=P, wsb=4 * 4 * 100 * 4 - 1)):
        assert call_mass(lib, **kw) == 1, kw
    for kw in (dict(d=96), dict(Hkv=3), dict(Hkv=0), dict(H=1 << 14, B=1 << 12, Hkv=1 << 10),
               dict(H=256, Hkv=1), dict(nk=1 << 30)):
        assert call_mass(lib, **kw) == 2, kw
    for kw in (dict(q=P + 8), dict(mass=P + 4), dict(lse=P + 4), dict(lens=P + 2)):
        assert call_mass(lib, **kw) == 3, kw


def test_select_refusals(lib):
    for kw in (dict(mass=0), dict(idx=0), dict(B=0), dict(nk=0), dict(topk=0), dict(first=-1),
               dict(last=-1), dict(first=3, last=2), dict(first=2 ** 31 - 1, last=2 ** 31 - 1)):
        assert call_select(lib, **kw) == 1, kw
    for kw in (dict(nk=524289), dict(topk=(1 << 20) + 1), dict(B=1 << 13, nq=1 << 18)):
        assert call_select(lib, **kw) == 2, kw
    assert call_select(lib, mass=P + 4) == 3
    assert call_select(lib, lens=P + 1) == 3


@pytest.mark.parametrize("backward", [False, True])
def test_attention_refusals(lib, backward):
    null = ["q", "k", "v", "idx", "out"] + (["lse", "dout", "dq", "dk", "dv"] if backward else [])
    for name in null:
        assert call_attn(lib, backward, **{name: 0}) == 1, name
    for kw in (dict(topk=0), dict(B=0), dict(scale=float("inf")), dict(ws=0), dict(wsb=16)):
        assert call_attn(lib, backward, **kw) == 1, kw
    for kw in (dict(d=32), dict(Hs=3), dict(H=12, Hkv=4, Hs=6), dict(H=512, Hkv=2, Hs=2),
               dict(topk=(1 << 20) + 1), dict(nk=1 << 30)):
        assert call_attn(lib, backward, **kw) == 2, kw
    for name in null:
        assert call_attn(lib, backward, **{name: P + 2}) == 3, name
    assert call_attn(lib, backward, lens=P + 2) == 3


def test_workspace_sizes(lib):
    ws = lib.streamkl_sparse_attn_workspace
    # The bit matrix: one bit per query, block and selection head, 32 queries to a word.
    assert ws(2, 16, 4, 4, 4096, 4096, 128, 16, 0) >= 2 * 4 * 4096 // 8 * 64
    assert ws(2, 16, 4, 4, 4096, 4096, 128, 16, 1) >= 2 * 4 * 4096 // 8 * 64 + 8 * 2 * 16 * 4096
    assert ws(1, 4, 2, 2, 1, 4096, 64, 4, 0) == 0
    assert ws(1, 4, 2, 2, 100, 200, 96, 4, 0) == -1
    assert lib.streamkl_block_mass_workspace(1, 4, 2, 100, 200, 64) == 4 * 4 * 100 * 4
    assert lib.streamkl_block_mass_workspace(1, 32, 8, 1, 8192, 64) == 0
    assert lib.streamkl_block_mass_workspace(64, 32, 8, 1, 8192, 64) == 4 * 64 * 32 * 128
    assert lib.streamkl_block_mass_workspace(1, 4, 2, 100, 200, 96) == -1
    assert ws(1, 4, 2, 2, 100, 200, 64, 0, 0) == -1


def test_wrappers_reject_cpu_and_wrong_tensors():
    q = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    idx = torch.zeros(1, 2, 8, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        sparse.sparse_attention(q, q, q, idx)
    with pytest.raises(ValueError):
        sparse.block_mass(q, q)
    with pytest.raises(ValueError):
        sparse.select_blocks(torch.zeros(1, 2, 8, 1), 8, 1)
    assert [sparse.num_blocks(n) for n in (1, 64, 65)] == [1, 1, 2]


def test_dispatch_raises_the_library_error():
    with pytest.raises(skl.StreamKLError) as e:
        sparse._ext().check(3, "some call")
    assert e.value.status == 3 and "some call" in str(e.value)
    sparse._ext().check(0, "some call")
    with pytest.raises(ValueError, match="mass has 3 blocks, n_k = 64 keys make 1"):
        sparse.select_blocks(torch.zeros(1, 1, 1, 3), 64, 1)


# ------------------------------------------------------------------ oracle pins


def _inputs(B, H, Hkv, nq, nk, d, seed=0):
    g = torch.Generator().manual_seed(seed)
    mk = lambda h, n: torch.randn(B, h, n, d, generator=g).to(torch.bfloat16)
    return mk(H, nq), mk(Hkv, nk), mk(Hkv, nk), mk(H, nq)


def test_oracle_mass_is_the_map_summed_by_blocks():
    q, k, _, _ = _inputs(2, 4, 2, 70, 200, 16)
    m = oracle_block_mass(q, k, 0.3, True)
    assert torch.allclose(m.sum(-1), torch.ones_like(m.sum(-1)), atol=1e-12)
    s = torch.einsum("bhid,bhjd->bhij", q.double(), k.double().repeat_interleave(2, 1)) * 0.3
    mask = torch.arange(200)[None, :] > torch.arange(70)[:, None] + 130
    p = s.masked_fill(mask, -math.inf).softmax(-1)
    ref = torch.stack([p[..., 64 * c:64 * c + 64].sum(-1) for c in range(4)], -1)
    assert torch.allclose(m, ref.view(2, 2, 2, 70, 4).mean(2), atol=1e-12)
    _, _, lse = oracle_fwd(q, k.repeat_interleave(2, 1), q, k.repeat_interleave(2, 1), 0.3, 0.3, True)
    assert torch.allclose(oracle_block_mass(q, k, 0.3, True, lse=lse), m, atol=1e-12)


def test_oracle_select_ties_and_forced():
    m = torch.tensor([[[[0.5, 0.1, 0.3, 0.3, 0.0, float("nan"), 0.3, 0.9]]]])
    sel = lambda **kw: oracle_block_select(m, 512, **{**dict(topk=3, causal=False, n_first=0, n_last=0), **kw})[0, 0, 0].tolist()
    assert sel() == [0, 2, 7]
    assert sel(topk=4) == [0, 2, 3, 7]
    assert sel(n_first=2, n_last=1) == [0, 1, 7]
    assert sel(topk=7) == [0, 1, 2, 3, 4, 6, 7]
    assert sel(topk=10) == [0, 1, 2, 3, 4, 5, 6, 7, -1, -1]


def test_oracle_attention_with_every_block_is_dense_attention():
    q, k, v, do = _inputs(1, 4, 2, 50, 130, 16)
    idx = torch.tensor([2, 0, 1, 1, -1], dtype=torch.int32).expand(1, 2, 50, 5)
    out, lse, dq, dk, dv = oracle_sparse_attn(q, k, v, idx, 0.25, True, dout=do)
    a = [t.double().requires_grad_() for t in (q, k, v)]
    kk, vv = (t.repeat_interleave(2, 1) for t in a[1:])
    s = a[0] @ kk.transpose(-1, -2) * 0.25
    s = s.masked_fill(torch.arange(130)[None, :] > torch.arange(50)[:, None] + 80, -math.inf)
    ref = s.softmax(-1) @ vv
    g = torch.autograd.grad(ref, a, do.double())
    assert torch.allclose(out, ref, atol=1e-12)
    assert torch.allclose(lse, s.logsumexp(-1), atol=1e-12)
    for x, y in zip((dq, dk, dv), g):
        assert torch.allclose(x, y, atol=1e-12)


def test_oracle_gradients_against_differences():
    q, k, v, do = _inputs(1, 2, 1, 6, 150, 8, seed=3)
    idx = torch.tensor([[0, 2], [1, -1], [-1, -1], [2, 2], [0, 1], [9, 1]], dtype=torch.int32)
    idx = idx.view(1, 1, 6, 2)
    q, k, v = (t.double() for t in (q, k, v))
    f = lambda: (oracle_sparse_attn(q, k, v, idx, 0.4, True)[0] * do.double()).sum().item()
    _, _, dq, dk, dv = oracle_sparse_attn(q, k, v, idx, 0.4, True, dout=do)
    for t, grad in ((q, dq), (k, dk), (v, dv)):
        for at in range(0, t.numel(), max(1, t.numel() // 12)):
            x, h = t.view(-1), 1e-5
            keep = x[at].item()
            x[at] = keep + h
            up = f()
            x[at] = keep - h
            down = f()
            x[at] = keep
            assert abs((up - down) / (2 * h) - grad.reshape(-1)[at].item()) < 1e-7


def test_oracle_empty_rows_and_padding():
    q, k, v, do = _inputs(2, 2, 2, 5, 100, 8)
    k[1, :, 30:], v[1, :, 30:] = float("nan"), float("inf")
    idx = torch.zeros(2, 2, 5, 1, dtype=torch.int32)
    idx[0, 0, 3] = -1
    out, lse, dq, dk, dv = oracle_sparse_attn(q, k, v, idx, 0.4, True, torch.tensor([100, 30]), do)
    assert (out[0, 0, 3] == 0).all() and lse[0, 0, 3] == -math.inf and (dq[0, 0, 3] == 0).all()
    for t in (out, dq, dk, dv):
        assert torch.isfinite(t).all()
    assert (dk[1, :, 30:] == 0).all() and (dv[1, :, 30:] == 0).all()
    assert selected_keys(idx, 100)[0, 0, 0].sum() == 64
    m = oracle_block_mass(q, k, 0.4, True, torch.tensor([100, 3]))
    assert (m[1, :, :2] == 0).all() and torch.isfinite(m).all()
