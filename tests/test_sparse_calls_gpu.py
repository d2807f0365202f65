"""Ways of calling the block-sparse operators (needs a B200)."""
import ctypes

import pytest
import torch
from torch.autograd import forward_ad

import attention_kl_divergence_fwd_b200 as skl
from attention_kl_divergence_fwd_b200 import sparse
from attention_kl_divergence_fwd_b200.autograd import set_check_status
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


@pytest.mark.parametrize("d", [64, 128])
def test_every_call_reads_its_own_selection(d):
    """The forward starts beside the kernel that writes its bit matrix, into memory that still holds
    another call's: few and many tiles, lists of one row and of all blocks in turn, eager and in a
    captured graph."""
    for B, H, Hkv, nq, nk in ((1, 2, 1, 2, 5000), (2, 16, 16, 700, 900), (1, 8, 2, 3000, 3000)):
        q, k, v, do = (t.cuda() for t in inputs(B, H, Hkv, nq, nk, d, seed=nq))
        nb = sparse.num_blocks(nk)
        g = torch.Generator().manual_seed(d)
        picks = [torch.rand(B, Hkv, nq, nb, generator=g).argsort(-1)[..., :6].int().cuda()
                 for _ in range(3)]
        picks.append(torch.full_like(picks[0], -1))
        alone = []
        for idx in picks:
            alone.append(sparse.streamkl_sparse_attn_fwd(q, k, v, idx, 0.125, True))
            torch.cuda.synchronize()  # and its workspace goes to the next call
        assert (alone[3][0] == 0).all() and not torch.equal(alone[0][0], alone[1][0])
        for _ in range(8):
            got = [sparse.streamkl_sparse_attn_fwd(q, k, v, idx, 0.125, True) for idx in picks]
            torch.cuda.synchronize()
            for want, have in zip(alone, got):
                assert all(torch.equal(a, b) for a, b in zip(want, have))
        # One workspace for every replay; the selection changes under it.
        idx, graph = picks[0].clone(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out, lse = sparse.streamkl_sparse_attn_fwd(q, k, v, idx, 0.125, True)
            grads = sparse.streamkl_sparse_attn_bwd(q, k, v, out, lse, do, idx, 0.125, True)
        for want, new in zip(alone * 3, picks * 3):
            idx.copy_(new)
            graph.replay()
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
            ref = sparse.streamkl_sparse_attn_bwd(q, k, v, *want, do, new, 0.125, True)
            assert all(torch.equal(a, b) for a, b in zip(grads, ref))
    assert skl.device_status() == 0


def test_other_python_threads_run_during_a_call():
    """Launches and the wait of a status check happen without the interpreter lock, which work queued
    before them may need. The library's functions are replaced by one that says whether its
    caller holds the lock; as a status, 1 is an error."""
    q, k, v, do = (t.cuda() for t in inputs(1, 4, 2, 20, 130, 64, seed=43))
    idx = lists(1, 2, 20, 130, 2, seed=43).cuda()
    mass = torch.zeros(1, 2, 20, 3, device="cuda")
    leaf = q.clone().requires_grad_()
    calls = [lambda: sparse.block_mass(q, k), lambda: sparse.select_blocks(mass, 130, 2),
             lambda: sparse.sparse_attention(q, k, v, idx),
             lambda: torch.autograd.grad(sparse.sparse_attention(leaf, k, v, idx), leaf, do)]
    ext = sparse._ext()
    at = lambda f: ctypes.cast(f, ctypes.c_void_p).value
    lib = skl.load_library()
    real = [at(getattr(lib, "streamkl_" + n)) for n in (
        "block_mass", "block_mass_workspace", "block_select", "sparse_attn_workspace",
        "sparse_attn_fwd", "sparse_attn_bwd", "status_string", "device_status")]
    held = at(ctypes.pythonapi.PyGILState_Check)
    try:
        set_check_status(True)
        # Every launch, then every status check.
        for fake in ([held if j in (0, 2, 4, 5) else a for j, a in enumerate(real)],
                     real[:7] + [held]):
            ext.bind(fake)
            for call in calls:
                call()
    finally:
        ext.bind(real)
        set_check_status(False)
    torch.cuda.synchronize()
    assert skl.device_status() == 0


def odd(t):
    """The same values behind one element of the same storage: contiguous, at an address that is no
    multiple of 16."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    flat[1:] = t.reshape(-1)
    r = flat[1:].view(t.shape)
    assert r.is_contiguous() and r.data_ptr() % 16
    return r


def test_contiguous_views_at_any_address():
    """Laid out by the call, as other strides are."""
    q, k, v, do = (t.cuda() for t in inputs(2, 4, 2, 70, 300, 64, seed=42))
    idx = lists(2, 2, 70, 300, 4, seed=42).cuda()
    lse = sparse.streamkl_sparse_attn_fwd(q, k, torch.zeros_like(k),
                                          torch.arange(5, dtype=torch.int32, device="cuda")
                                          .expand(2, 2, 70, 5).contiguous(), 0.125, True)[1]
    mass = sparse.block_mass(q, k, causal=True, lse=lse)
    assert torch.equal(sparse.block_mass(odd(q), k, causal=True, lse=odd(lse)), mass)
    assert torch.equal(sparse.block_mass(q, odd(k), causal=True),
                       sparse.block_mass(q, k, causal=True))
    sel = sparse.select_blocks(mass, 300, 3, True)
    assert torch.equal(sparse.select_blocks(odd(mass), 300, 3, True), sel)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    out = sparse.sparse_attention(*leaves, idx, causal=True)
    ref = torch.autograd.grad(out, leaves, do)
    moved = [odd(t).requires_grad_() for t in (q, k, v)]
    got = sparse.sparse_attention(*moved, odd(idx), causal=True)
    assert torch.equal(got, out)
    for a, b in zip(torch.autograd.grad(got, moved, odd(do)), ref):
        assert torch.equal(a, b)
    # One sequence of a batch of single-token masses: 65 blocks of one head.
    m = torch.rand(3, 1, 1, 65, device="cuda")
    for b in range(3):
        assert torch.equal(sparse.select_blocks(m[b:b + 1], 65 * 64, 4),
                           sparse.select_blocks(m[b:b + 1].clone(), 65 * 64, 4))
    assert skl.device_status() == 0


def test_captured_backward_of_inputs_computed_before():
    """The captured forward of a tensor that eager code computed is sound, its captured backward would
    go on into the eager part: refused, and the capture is as good as before."""
    q, k, v, do = (t.cuda() for t in inputs(1, 4, 2, 70, 300, 64, seed=44))
    idx = lists(1, 2, 70, 300, 4, seed=44).cuda()
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    made = [t * 1 for t in leaves]  # on the default stream, with a gradient function
    plain = [t.clone().requires_grad_() for t in (q, k, v)]
    out = sparse.sparse_attention(*plain, idx, causal=True)
    ref = torch.autograd.grad(out, plain, do)
    want = out.detach().clone()
    del out
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = []
        for j in range(3):
            args = [t.detach().requires_grad_() for t in made]
            args[j] = made[j]
            kept.append(sparse.sparse_attention(*args, idx, causal=True))
            for inputs_ in ([leaves[j]], [made[j]]):
                with pytest.raises(RuntimeError, match="qkv"[j] + " is part of a graph made on the default"):
                    torch.autograd.grad(kept[j], inputs_, do, retain_graph=True)
        args = [t.detach().requires_grad_() for t in made]
        kept.append(sparse.sparse_attention(*args, idx, causal=True))
        grads = torch.autograd.grad(kept[3], args, do)
    for t in (*kept, *grads):
        t.detach().zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(t, want) for t in kept)
    assert all(torch.equal(a, b) for a, b in zip(grads, ref))
    # Eager again.
    eager = torch.autograd.grad(sparse.sparse_attention(*made, idx, causal=True), leaves, do)
    assert all(torch.equal(a, b) for a, b in zip(eager, ref))
    assert skl.device_status() == 0
