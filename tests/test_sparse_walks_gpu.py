"""Block-sparse kernels on the launch shapes of long prompts and training steps, against the fp64
oracle (needs a B200): tiles that one CTA walks alone, many steps through every ring of buffers,
and every width that the selection is compiled for. Bounds as in test_sparse_gpu."""
import math

import pytest
import torch

import attention_kl_divergence_fwd_b200 as skl
from attention_kl_divergence_fwd_b200 import sparse
from oracle import oracle_block_mass, oracle_block_select, oracle_sparse_attn
from oracle.sparse_oracle import _allowed, _f64, _scores
from test_sparse_gpu import NAN, close, inputs, lists, pad_nan

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from attention_kl_divergence_fwd_b200 import build
    build.build()
    skl.load_library()


def sm_count():
    return torch.cuda.get_device_properties(0).multi_processor_count


def tile_queries(H, packs, nq):
    """Queries of a 128-row tile: the power of two that fits with the pack's heads."""
    n = 1
    while n * 2 * (H // packs) <= 128 and n < nq:
        n *= 2
    return n


def shared_lists(B, Hs, nq, nk, topk, run=100):
    """Lists that runs of queries share (runs end inside tiles): blocks that all rows of a tile list
    beside blocks that some do."""
    nb = (nk + 63) // 64
    g = torch.Generator().manual_seed(nq + nk)
    pick = torch.rand(B, Hs, (nq + run - 1) // run, nb, generator=g).argsort(-1)[..., :topk]
    return pick.repeat_interleave(run, 2)[:, :, :nq].int().contiguous()


# B, H, Hkv, Hsel, nq, nk, d, causal, topk, padded lengths
WALKS = [
    (2, 16, 16, 16, 700, 1500, 64, True, 5, [1500, 1111]),
    (2, 16, 16, 16, 700, 1500, 128, True, 5, [1111, 1500]),
    (1, 32, 8, 2, 700, 1300, 128, True, 6, None),
    (1, 32, 8, 8, 645, 1200, 64, True, 6, None),
    (2, 16, 16, 1, 650, 1010, 128, False, 9, [1010, 650]),
    (1, 39, 13, 13, 700, 700, 64, True, 11, None),
    (5, 32, 8, 8, 133, 1290, 128, True, 4, [1290, 1200, 133, 700, 1000]),
]


@pytest.mark.parametrize("case", WALKS, ids=str)
@pytest.mark.parametrize("shared", [False, True], ids=["unrelated", "shared"])
def test_tiles_of_one_cta_with_long_lists(case, shared):
    B, H, Hkv, Hs, nq, nk, d, causal, topk, lens = case
    P = max(Hkv, Hs)
    qn = tile_queries(H, P, nq)
    # One CTA per tile (the planner splits a list only while two CTAs per SM are not taken), rows
    # for all four warps of a tile, and lists longer than every ring of buffers.
    assert 2 * sm_count() // (B * P * ((nq + qn - 1) // qn)) < 2 and qn * H // P > 32
    idx = (shared_lists if shared else lists)(B, Hs, nq, nk, topk)
    if not shared:
        tile = idx[0, 0, :qn]
        assert len(set(tile[(tile >= 0) & (tile < nk // 64)].tolist())) > 8
    q, k, v, do = inputs(B, H, Hkv, nq, nk, d, seed=nq + topk)
    if lens:
        k, v = pad_nan(k, lens), pad_nan(v, lens)
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    tol = {}
    out, lse, dq, dk, dv = oracle_sparse_attn(q, k, v, idx, 0.125, causal, lt, do, tol)
    qg, kg, vg = (t.cuda().requires_grad_() for t in (q, k, v))
    got, got_lse = sparse.sparse_attention(qg, kg, vg, idx.cuda(), 0.125, causal,
                                           None if lt is None else lt.cuda(), return_lse=True)
    grads = torch.autograd.grad(got, (qg, kg, vg), do.cuda())
    assert skl.device_status() == 0
    empty = lse == -math.inf
    assert torch.equal(got_lse.cpu() == -math.inf, empty)
    close(torch.where(empty, 0.0, got_lse.detach().cpu()), torch.where(empty, 0.0, lse),
          tol["lse"], "lse")
    close(got.detach(), out, tol["out"], "out")
    for name, x, ref in zip(("dq", "dk", "dv"), grads, (dq, dk, dv)):
        close(x, ref, tol[name], name)


# B, H, Hkv, nq, nk, d, causal, padded lengths
LONG_MASS = [
    (2, 10, 10, 4229, 4229, 64, True, [4229, 4170]),
    (1, 600, 300, 70, 4229, 128, False, None),
    (1, 300, 300, 130, 4500, 64, True, None),
    (3, 206, 103, 65, 4300, 128, True, [4300, 2111, 65]),
]


@pytest.mark.parametrize("case", LONG_MASS, ids=str)
@pytest.mark.parametrize("given", [False, True])
def test_mass_of_ctas_with_many_steps(case, given):
    B, H, Hkv, nq, nk, d, causal, lens = case
    qn, nb = tile_queries(H, Hkv, nq), (nk + 63) // 64
    # A CTA takes all blocks of its tile: more than two groups of 32 staged blocks.
    assert 8 * sm_count() // (B * Hkv * ((nq + qn - 1) // qn)) < 2 and nb > 64
    assert qn * H // Hkv > 32
    q, k, _, _ = inputs(B, H, Hkv, nq, nk, d, seed=nk)
    if lens:
        k = pad_nan(k, lens)
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    scale = 0.125
    lse = None
    if given:
        lse = torch.empty(B, H, nq)
        for b in range(B):
            ok = _allowed(nq, nk, nk if lens is None else lens[b], causal)
            for h in range(H):
                s = _scores(_f64(q[b, h]), _f64(k[b, h // (H // Hkv)]), scale, ok)
                lse[b, h] = torch.logsumexp(s, -1).float()
    ref = oracle_block_mass(q, k, scale, causal, lt, lse)
    got = sparse.block_mass(q.cuda(), k.cuda(), scale, causal, None if lse is None else lse.cuda(),
                            None if lt is None else lt.cuda())
    assert skl.device_status() == 0
    # mass_tol of test_sparse_gpu with |q| |k| (Cauchy-Schwarz) for the largest sum_d |q_d k_d|.
    reach = (q.double().norm(dim=-1).max() * k.double().nan_to_num(0, 0, 0).norm(dim=-1).max()) * scale
    e = d * reach * 2.0 ** -23 + 8 * 2.0 ** -23 * (1 + 2 * reach) + 2.0 ** -21 + 64 * 2.0 ** -24
    close(got, ref, 3 * e * ref + 1e-30, "mass")
    assert (got.cpu()[ref == 0] == 0).all()


# One warp per row of up to 256 blocks, its registers by what the row sees; of up to 1024 blocks
# with 16 rows per SM or more; lengths set how many blocks the rows of a sequence see.
@pytest.mark.parametrize("nq,nk,lens", [(300, 16384, [16384, 9000]), (300, 16320, [12280, 4000]),
                                        (65, 12288, [8192, 8193]), (900, 9000, None),
                                        (450, 20000, [20000, 5000]), (450, 65536, [65536, 12100]),
                                        (420, 40001, [16500, 16300])], ids=str)
@pytest.mark.parametrize("topk,first,last", [(16, 1, 2), (48, 0, 0), (32, 2, 30), (5, 0, 1)])
def test_selection_of_every_width(nq, nk, lens, topk, first, last):
    B, Hs, nb = 2, 3, (nk + 63) // 64
    assert nb <= 256 or (nb <= 1024 and B * Hs * nq >= 16 * sm_count())
    g = torch.Generator().manual_seed(nk + topk)
    pool = torch.tensor([0.0, -0.0, 0.25, 0.25, 0.5, 1.0, -1.0, math.inf, -math.inf, NAN, 1e-40])
    mass = torch.rand(B, Hs, nq, nb, generator=g)
    mass[:, 0] = pool[torch.randint(0, len(pool), (B, nq, nb), generator=g)]  # ties
    mass[:, 1, ::2] = (mass[:, 1, ::2] * 4).floor() / 4
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    got = sparse.select_blocks(mass.cuda(), nk, topk, True, first, last,
                               None if lt is None else lt.cuda())
    assert torch.equal(got.cpu(), oracle_block_select(mass, nk, topk, True, first, last, lt))
    assert skl.device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_gradients_of_queries_and_keys_against_differences(d):
    """Central differences of the kernel's forward, along steps of one query (one key) that bf16
    holds exactly, against its gradient. Bound: the outputs' and the gradient's own (oracle), and
    what the oracle says the quotient differs from the derivative by."""
    nq, nk, scale = 40, 150, 0.25
    q, k, v, do = inputs(1, 2, 1, nq, nk, d, seed=45)
    grid = lambda t: (t.float().clamp(-3, 3) * 16).round() / 16  # 7 bits with a step
    q, k, v = (grid(t).to(torch.bfloat16) for t in (q, k, v))
    # One output entry, of values of either sign: its derivatives are well above the bound.
    do = torch.zeros_like(do)
    do[0, 1, 30, 0] = 1
    v[..., 0] = torch.where(torch.arange(nk) % 2 == 0, 3, -3)
    idx = torch.arange(3, dtype=torch.int32).expand(1, 1, nq, 3).contiguous()
    tol = {}
    _, _, dq, dk, _ = oracle_sparse_attn(q, k, v, idx, scale, True, None, do, tol)
    key = int(dk[0, 0].norm(dim=-1).argmax())
    leaves = [t.cuda().requires_grad_() for t in (q, k, v)]
    grads = torch.autograd.grad(sparse.sparse_attention(*leaves, idx.cuda(), scale, True), leaves,
                                do.cuda())
    for which, at, exact, name in ((0, (0, 1, 30), dq, "dq"), (1, (0, 0, key), dk, "dk")):
        step = torch.zeros_like((q, k)[which])
        step[at] = torch.sign(exact[at]).to(torch.bfloat16) / 16
        value, oracle, bound = [], [], 0.0
        for s in (1, -1):
            args = [q, k]
            args[which] = args[which] + s * step
            assert torch.equal(args[which].double(), (q, k)[which].double() + s * step.double())
            t = {}
            out, _ = oracle_sparse_attn(*args, v, idx, scale, True, bounds=t)
            oracle.append((out * do.double()).sum().item())
            bound += (t["out"] * do.double().abs()).sum().item() / 2
            got = sparse.sparse_attention(*(x.cuda() for x in (*args, v)), idx.cuda(), scale, True)
            value.append((got.cpu().double() * do.double()).sum().item())
        along = (grads[which].cpu().double() * step.double()).sum().item()
        truth = (exact * step.double()).sum().item()
        bound += abs((oracle[0] - oracle[1]) / 2 - truth) + (tol[name] * step.double().abs()).sum().item()
        assert abs((value[0] - value[1]) / 2 - along) <= bound
        assert bound < truth / 2  # the test can tell
