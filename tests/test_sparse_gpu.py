"""Block-sparse attention on the GPU against the fp64 oracle (needs a B200).

Tolerances are elementwise bounds computed with the oracle's own magnitudes (oracle_sparse_attn's
``bounds``): bf16 roundings of P, dS, out and the gradients at half a step (2^-8) each, fp32 sums
and exponents at their steps. Masses are fp32: a score's error (d products at 2^-23 of their
absolute sum, the exponent's argument at 4 steps) moves a mass by that relative amount. Lists
are compared exactly."""
import math
import threading

import pytest
import torch

import attention_kl_divergence_fwd_b200 as skl
from attention_kl_divergence_fwd_b200 import sparse
from attention_kl_divergence_fwd_b200.autograd import attention_kl_loss, set_check_status
from oracle import oracle_block_mass, oracle_block_select, oracle_sparse_attn

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    from attention_kl_divergence_fwd_b200 import build
    build.build()
    skl.load_library()


def inputs(B, H, Hkv, nq, nk, d, seed=0, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    mk = lambda h, n: (torch.randn(B, h, n, d, generator=g) * spread).to(torch.bfloat16)
    return mk(H, nq), mk(Hkv, nk), mk(Hkv, nk), mk(H, nq)


def lists(B, Hs, nq, nk, topk, seed=0, wild=True):
    """Random lists: unsorted, with repeats, -1 in any place, entries beyond the blocks, and every
    fifth query without any."""
    g = torch.Generator().manual_seed(seed + 100)
    nb = (nk + 63) // 64
    idx = torch.randint(-1, nb + (2 if wild else 0), (B, Hs, nq, topk), generator=g, dtype=torch.int32)
    if wild:
        idx[torch.rand(B, Hs, nq, generator=g) < 0.2] = -1
        idx[:, :, :, 0][idx[:, :, :, 0] == nb] = 2 ** 31 - 1
        idx[:, :, :, 0][idx[:, :, :, 0] == -1] = -2 ** 31
    return idx


def pad_nan(t, lens):
    t = t.clone()
    for b, n in enumerate(lens):
        t[b, :, n:] = NAN
        if n < t.shape[2]:
            t[b, :, n, 0] = math.inf
    return t


def close(got, ref, tol, what):
    got = got.cpu().double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = ((got - ref).abs() - tol).max().item()
    assert over <= 0, f"{what}: over its bound by {over:.3e}"


def mass_tol(q, k, scale, ref, causal):
    d = q.shape[-1]
    reach = (q.double().abs().amax(-1).amax() * 0 +
             (q.double().abs() @ k.double().nan_to_num(0, 0, 0).abs()
              .repeat_interleave(q.shape[1] // k.shape[1], 1).transpose(-1, -2)).amax()) * abs(scale)
    e = d * reach * 2.0 ** -23 + 8 * 2.0 ** -23 * (1 + 2 * reach) + 2.0 ** -21 + 64 * 2.0 ** -24
    return 3 * e * ref + 1e-30


# B, H, Hkv, nq, nk, d, causal, padded lengths
MASS = [
    (1, 1, 1, 1, 1, 64, True, None),
    (1, 4, 1, 1, 64, 128, False, None),
    (2, 8, 2, 1, 1000, 64, True, [1000, 1]),
    (2, 3, 1, 5, 333, 128, True, [333, 70]),
    (1, 2, 2, 130, 130, 64, True, None),
    (1, 6, 2, 200, 2200, 64, False, None),
    (1, 12, 2, 70, 70, 128, True, None),
    (2, 8, 2, 257, 300, 128, True, [300, 257]),
    (1, 5, 5, 300, 100, 64, True, None),       # the first queries see no key
    (3, 4, 4, 40, 190, 64, True, [190, 0, 41]),
    (1, 128, 1, 3, 129, 64, False, None),
    (1, 8, 2, 2, 5000, 128, True, [4700]),     # few rows: a cluster normalises on chip
    (40, 8, 4, 1, 900, 64, True, [900 - 22 * b for b in range(40)]),  # many: two kernels
]


@pytest.mark.parametrize("case", MASS, ids=str)
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("scale", [0.125, -0.3, 0.0])
def test_block_mass(case, given, scale):
    B, H, Hkv, nq, nk, d, causal, lens = case
    q, k, _, _ = inputs(B, H, Hkv, nq, nk, d, seed=nq)
    if lens:
        k = pad_nan(k, lens)
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    ref = oracle_block_mass(q, k, scale, causal, lt)
    lse = None
    if given:
        from oracle.sparse_oracle import _allowed, _f64, _scores
        lse = torch.empty(B, H, nq)
        for b in range(B):
            ok = _allowed(nq, nk, nk if lens is None else lens[b], causal)
            for h in range(H):
                s = _scores(_f64(q[b, h]), _f64(k[b, h // (H // Hkv)]), scale, ok)
                lse[b, h] = torch.logsumexp(s, -1).float()
        ref = oracle_block_mass(q, k, scale, causal, lt, lse)
    got = sparse.block_mass(q.cuda(), k.cuda(), scale, causal, None if lse is None else lse.cuda(),
                            None if lt is None else lt.cuda())
    assert got.shape == ref.shape and skl.device_status() == 0
    close(got, ref, mass_tol(q, k, scale, ref, causal), "mass")
    assert (got.cpu()[ref == 0] == 0).all()


@pytest.mark.parametrize("nq,nk,topk,first,last,causal,lens", [
    (1, 1, 1, 0, 0, True, None), (1, 64, 3, 1, 1, True, None), (5, 700, 4, 1, 2, True, [700, 300]),
    (300, 300, 3, 0, 0, True, None), (33, 4200, 16, 2, 2, False, [4200, 64]),
    (3, 16500, 40, 1, 1, True, [16500, 9000]), (2, 65536, 64, 0, 3, False, None),
    (2, 70000, 17, 1, 1, True, [70000, 0]), (1, 524288, 100, 3, 3, True, None),
    (40, 500, 20, 4, 8, True, None), (9, 5, 2, 1, 1, True, None)], ids=str)
def test_block_select(nq, nk, topk, first, last, causal, lens):
    B, Hs, nb = 2, 3, (nk + 63) // 64
    g = torch.Generator().manual_seed(nk)
    # Few distinct values (many ties), negative ones, both zeros, infinities and NaN among them.
    pool = torch.tensor([0.0, -0.0, 0.25, 0.25, 0.5, 1.0, -1.0, math.inf, -math.inf, NAN, 1e-40])
    mass = pool[torch.randint(0, len(pool), (B, Hs, nq, nb), generator=g)]
    mass[0] = torch.rand(Hs, nq, nb, generator=g)
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    got = sparse.select_blocks(mass.cuda(), nk, topk, causal, first, last,
                               None if lt is None else lt.cuda())
    ref = oracle_block_select(mass, nk, topk, causal, first, last, lt)
    assert torch.equal(got.cpu(), ref) and skl.device_status() == 0


# B, H, Hkv, Hsel, nq, nk, d, causal, topk, padded lengths
ATTN = [
    (1, 1, 1, 1, 1, 1, 64, True, 1, None),
    (1, 4, 1, 1, 1, 200, 128, True, 3, None),
    (3, 8, 2, 2, 1, 1000, 128, True, 16, [1000, 1, 65]),
    (2, 8, 8, 2, 1, 700, 64, False, 40, [700, 0]),
    (1, 6, 2, 1, 2, 300, 64, True, 5, None),
    (2, 3, 1, 1, 5, 333, 128, True, 4, [333, 70]),
    (1, 2, 2, 2, 130, 130, 64, True, 2, None),
    (1, 8, 2, 4, 70, 450, 128, False, 3, None),     # finer selection than K heads
    (1, 8, 2, 1, 200, 260, 64, True, 3, None),
    (2, 12, 2, 2, 129, 300, 128, True, 4, [300, 129]),
    (1, 5, 5, 5, 300, 100, 64, True, 2, None),      # the first queries see no key
    (1, 1, 1, 1, 513, 700, 128, True, 6, None),
    (1, 70, 1, 1, 3, 129, 64, False, 2, None),
    (1, 128, 1, 1, 2, 190, 128, True, 3, None),
    (2, 4, 4, 1, 33, 1100, 128, True, 9, [1100, 40]),
    (1, 4, 1, 1, 1200, 1200, 128, True, 4, None),   # few K heads: blocks split over clusters
    (1, 4, 1, 1, 1100, 1250, 64, True, 4, [1190]),
    (2, 40, 2, 1, 1, 700, 64, True, 5, [700, 65]),  # one query, more heads than a copied tile holds
    (1, 8, 2, 2, 1, 1300, 128, True, 600, None),    # one query, a list longer than the blocks
    (2, 16, 16, 16, 4, 800, 64, False, 3, [800, 3]),
]


@pytest.mark.parametrize("case", ATTN, ids=str)
@pytest.mark.parametrize("scale", [0.125, -0.2, 0.0])
def test_sparse_attention(case, scale):
    B, H, Hkv, Hs, nq, nk, d, causal, topk, lens = case
    q, k, v, do = inputs(B, H, Hkv, nq, nk, d, seed=nq + d)
    if lens:
        k, v = pad_nan(k, lens), pad_nan(v, lens)
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    idx = lists(B, Hs, nq, nk, topk, seed=nk)
    tol = {}
    out, lse, dq, dk, dv = oracle_sparse_attn(q, k, v, idx, scale, causal, lt, do, tol)
    dev = dict(scale=scale, causal=causal, seqlens_k=None if lt is None else lt.cuda())
    qg, kg, vg = (t.cuda().requires_grad_() for t in (q, k, v))
    got, got_lse = sparse.sparse_attention(qg, kg, vg, idx.cuda(), return_lse=True, **dev)
    grads = torch.autograd.grad(got, (qg, kg, vg), do.cuda())
    assert skl.device_status() == 0
    empty = lse == -math.inf
    assert torch.equal(got_lse.cpu() == -math.inf, empty)
    assert (got.detach().cpu()[empty] == 0).all() and (grads[0].cpu()[empty] == 0).all()
    close(torch.where(empty, 0.0, got_lse.detach().cpu()), torch.where(empty, 0.0, lse),
          tol["lse"], "lse")
    close(got.detach(), out, tol["out"], "out")
    for name, x, ref in zip(("dq", "dk", "dv"), grads, (dq, dk, dv)):
        close(x, ref, tol[name], name)
    # The inference call and a second run give the same bits.
    again = sparse.sparse_attention(q.cuda(), k.cuda(), v.cuda(), idx.cuda(), **dev)
    assert torch.equal(again, got)
    grads2 = torch.autograd.grad(sparse.sparse_attention(qg, kg, vg, idx.cuda(), **dev),
                                 (qg, kg, vg), do.cuda())
    assert all(torch.equal(a, b) for a, b in zip(grads, grads2))


def test_large_scores_and_rising_maxima():
    """Scores up to several hundred, rising along the keys, so the running reference moves."""
    q, k, v, do = inputs(1, 4, 2, 100, 640, 64, seed=5, spread=2.0)
    k = (k.float() * torch.linspace(0.2, 6, 640)[:, None]).to(torch.bfloat16)
    idx = torch.arange(10, dtype=torch.int32).expand(1, 2, 100, 10).contiguous()
    tol = {}
    out, lse, dq, dk, dv = oracle_sparse_attn(q, k, v, idx, 1.0, False, None, do, tol)
    qg, kg, vg = (t.cuda().requires_grad_() for t in (q, k, v))
    got, got_lse = sparse.sparse_attention(qg, kg, vg, idx.cuda(), 1.0, False, return_lse=True)
    close(got_lse.detach(), lse, tol["lse"], "lse")
    close(got.detach(), out, tol["out"], "out")
    for name, x, ref in zip(("dq", "dk", "dv"), torch.autograd.grad(got, (qg, kg, vg), do.cuda()),
                            (dq, dk, dv)):
        close(x, ref, tol[name], name)


@pytest.mark.parametrize("nq,nk,splitting", [(1, 9000, True), (3, 5000, True), (2000, 2300, False)])
def test_longer_lists(nq, nk, splitting):
    q, k, v, _ = inputs(1, 4, 2, nq, nk, 128, seed=9)
    nb = (nk + 63) // 64
    idx = torch.stack([torch.randperm(nb, generator=torch.Generator().manual_seed(i))[:24]
                       for i in range(2 * nq)]).view(1, 2, nq, 24).int()
    tol = {}
    out, lse = oracle_sparse_attn(q, k, v, idx, 0.088, True, bounds=tol)
    got, got_lse = sparse.sparse_attention(q.cuda(), k.cuda(), v.cuda(), idx.cuda(), 0.088, True,
                                           return_lse=True)
    close(got, out, tol["out"], "out")
    fin = lse > -math.inf
    close(got_lse.cpu()[fin], lse[fin], tol["lse"][fin], "lse")


def test_tokens_with_several_key_tiles_and_padded_ends():
    """More tiles than CTAs take at once, so that each walks several pairs of blocks of one list
    and reaches the padded end with earlier pairs still in flight."""
    B, Hkv, nk = 40, 8, 900
    q, k, v, _ = inputs(B, 16, Hkv, 1, nk, 128, seed=12)
    lens = torch.arange(B, dtype=torch.int32) * 22 + 30
    k, v = pad_nan(k, lens.tolist()), pad_nan(v, lens.tolist())
    idx = torch.arange(15, dtype=torch.int32).expand(B, Hkv, 1, 15).contiguous()
    tol = {}
    out, lse = oracle_sparse_attn(q, k, v, idx, 0.088, True, lens, bounds=tol)
    for _ in range(20):
        got, got_lse = sparse.sparse_attention(q.cuda(), k.cuda(), v.cuda(), idx.cuda(), 0.088, True,
                                               lens.cuda(), return_lse=True)
        close(got, out, tol["out"], "out")
        close(got_lse, lse, tol["lse"], "lse")


def test_gradient_against_differences():
    """Directional derivatives of the CUDA forward against its gradients. With out linear in v
    the difference quotient of v is exact up to rounding: bf16 outputs, 2^-8 of |out| each."""
    q, k, v, do = (t.cuda() for t in inputs(1, 4, 2, 64, 200, 64, seed=2))
    idx = lists(1, 2, 64, 200, 3, seed=4).cuda()
    vg = v.clone().requires_grad_()
    out = sparse.sparse_attention(q, k, vg, idx, causal=True)
    dv, = torch.autograd.grad(out, vg, do)
    step = torch.randn_like(v)
    moved = sparse.sparse_attention(q, k, step, idx, causal=True)
    lhs = (moved.double() * do.double()).sum()
    rhs = (dv.double() * step.double()).sum()
    bound = 2 * 2.0 ** -8 * ((moved.double() * do.double()).abs().sum() * 8 +
                             (dv.double() * step.double()).abs().sum())
    assert (lhs - rhs).abs() <= bound


def test_as_a_user_trains_and_serves():
    """Divergence, block masses from its log-sum-exps, selection and attention in one step with
    both gradients; then single tokens against a padded cache."""
    B, H, Hkv, n, d, ds = 2, 8, 2, 384, 128, 64
    q, k, v, do = inputs(B, H, Hkv, n, n, d, seed=1)
    qs, ks, _, _ = inputs(B, H, Hkv, n, n, ds, seed=2)
    qg, kg, vg, qsg, ksg = (t.cuda().requires_grad_() for t in (q, k, v, qs, ks))
    loss = attention_kl_loss(qg.detach(), kg.detach(), qsg, ksg, causal=True)
    _, _, lse_s = skl.streamkl_fwd_gqa(qg.detach(), kg.detach(), qsg.detach(), ksg.detach(),
                                       d ** -0.5, ds ** -0.5, True)
    out, idx = sparse.student_sparse_attention(qg, kg, vg, qsg, ksg, 3, causal=True, lse_s=lse_s)
    (loss + (out.float() * do.cuda().float()).sum()).backward()
    assert all(torch.isfinite(t.grad).all() for t in (qg, kg, vg, qsg, ksg))
    mass = oracle_block_mass(qs, ks, ds ** -0.5, True)
    picked = torch.zeros_like(mass).scatter_(-1, idx.cpu().long().clamp(min=0), 1.0)
    assert (picked[..., 0] == 1).all()
    # Every list carries as much mass as the oracle's best list, up to the masses' tolerance.
    best = oracle_block_select(mass, n, 3, True, 1, 1)
    ref_pick = torch.zeros_like(mass).scatter_(-1, best.long().clamp(min=0), 1.0)
    assert ((mass * picked).sum(-1) - (mass * ref_pick).sum(-1)).abs().max() < 1e-4
    tol = {}
    ref = oracle_sparse_attn(q, k, v, idx.cpu(), d ** -0.5, True, None, do, tol)
    for name, x, r in zip(("out", "dq", "dk", "dv"), (out.detach(), qg.grad, kg.grad, vg.grad),
                          (ref[0],) + ref[2:]):
        close(x, r, tol[name], name)
    # One new token of each sequence, with 300 and 77 keys in the cache.
    lens = torch.tensor([300, 77], dtype=torch.int32)
    kc, vc, ksc = (pad_nan(t, lens.tolist()) for t in (k, v, ks))
    tok, idx1 = sparse.student_sparse_attention(q[:, :, :1].cuda(), kc.cuda(), vc.cuda(),
                                                qs[:, :, :1].cuda(), ksc.cuda(), 3, causal=True,
                                                seqlens_k=lens.cuda())
    tol = {}
    r, _ = oracle_sparse_attn(q[:, :, :1], kc, vc, idx1.cpu(), d ** -0.5, True, lens, bounds=tol)
    close(tok, r, tol["out"], "token")


@pytest.mark.parametrize("nq,nk,causal,lens", [(64, 64, True, None), (40, 70, True, None),
                                               (150, 60, False, None), (90, 300, True, [300, 64]),
                                               (200, 150, True, [20, 150])], ids=str)
def test_gradients_of_queries_with_few_keys(nq, nk, causal, lens):
    """Rows that see one block at most take sum_d out dout from their keys: dS is then good to its
    own rounding, which the bounds require of these rows. Large values make that rounding of out
    the larger part otherwise."""
    B, Hs = 2, 1
    q, k, v, do = inputs(B, 6, 3, nq, nk, 64, seed=21)
    v = (v.float() + 4).to(torch.bfloat16)  # out and dout share a direction: D is large
    do = (do.float() + 2).to(torch.bfloat16)
    if lens:
        k, v = pad_nan(k, lens), pad_nan(v, lens)
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    idx = lists(B, Hs, nq, nk, 3, seed=3, wild=False)
    idx[..., 0] = 0
    idx[0, 0, 5] = -1
    tol = {}
    ref = oracle_sparse_attn(q, k, v, idx, 0.125, causal, lt, do, tol)
    qg, kg, vg = (t.cuda().requires_grad_() for t in (q, k, v))
    out = sparse.sparse_attention(qg, kg, vg, idx.cuda(), 0.125, causal, None if lt is None else lt.cuda())
    for name, x, r in zip(("dq", "dk", "dv"), torch.autograd.grad(out, (qg, kg, vg), do.cuda()), ref[2:]):
        close(x, r, tol[name], name)


def test_graph_capture_streams_and_other_layouts():
    q, k, v, do = (t.cuda() for t in inputs(2, 4, 2, 70, 300, 64, seed=8))
    idx = lists(2, 2, 70, 300, 4, seed=8).cuda()
    out, lse = skl.sparse.streamkl_sparse_attn_fwd(q, k, v, idx, 0.125, True)
    ref = skl.sparse.streamkl_sparse_attn_bwd(q, k, v, out, lse, do, idx, 0.125, True)
    # Another stream.
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o2, l2 = skl.sparse.streamkl_sparse_attn_fwd(q, k, v, idx, 0.125, True, stream=s)
    s.synchronize()
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    # Two captured graphs (each with its own workspace) replayed in turn on new inputs.
    qs = [q.clone(), q.flip(2).contiguous()]
    graphs, outs = [], []
    for x in qs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o, l = skl.sparse.streamkl_sparse_attn_fwd(x, k, v, idx, 0.125, True)
            grads = skl.sparse.streamkl_sparse_attn_bwd(x, k, v, o, l, do, idx, 0.125, True)
            m = skl.sparse.streamkl_block_mass(x, k, 0.125, True)
        graphs.append(g)
        outs.append((o, *grads, m))
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], out)
    assert all(torch.equal(a, b) for a, b in zip(outs[0][1:4], ref))
    assert torch.equal(outs[1][4], sparse.block_mass(qs[1], k, 0.125, True))
    # Transposed views are laid out by the call; an expanded gradient too.
    qt = q.transpose(1, 2).contiguous().transpose(1, 2).requires_grad_()
    o3 = sparse.sparse_attention(qt, k, v, idx, 0.125, True)
    assert torch.equal(o3, out)
    o3.sum().backward()
    ones = torch.ones_like(out)
    assert torch.equal(qt.grad, skl.sparse.streamkl_sparse_attn_bwd(q, k, v, out, lse, ones, idx,
                                                                    0.125, True)[0])
    assert skl.device_status() == 0


def test_calls_on_two_streams_at_once():
    streams = [torch.cuda.Stream() for _ in range(2)]
    jobs = []
    for j in range(2):
        q, k, v, do = (t.cuda() for t in inputs(1, 8, 2, 600, 900, 128, seed=30 + j))
        idx = lists(1, 2, 600, 900, 6, seed=j).cuda()
        jobs.append((q, k, v, do, idx))

    def run(q, k, v, do, idx, stream=None):
        out, lse = sparse.streamkl_sparse_attn_fwd(q, k, v, idx, 0.1, True, stream=stream)
        g = sparse.streamkl_sparse_attn_bwd(q, k, v, out, lse, do, idx, 0.1, True, stream=stream)
        m = sparse.streamkl_block_mass(q, k, 0.1, True, stream=stream)
        i = sparse.streamkl_block_select(m, 900, True, 5, stream=stream)
        return [out, lse, *g, m, i]

    alone = [run(*job) for job in jobs]
    torch.cuda.synchronize()
    for _ in range(5):
        both = [run(*job, stream=s) for job, s in zip(jobs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(alone, both):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert skl.device_status() == 0


def test_offsets_past_32_bits():
    """A cache whose last heads lie beyond 2^31 elements: token attention with its gradients, block
    masses and selection of the last head against the oracle on that head alone."""
    H, n, d = 128, 132000, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    k = torch.empty(1, H, n, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    v = torch.empty_like(k).normal_(generator=g)
    assert k.numel() > 2 ** 31
    q = torch.empty(1, H, 1, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    do = torch.empty_like(q).normal_(generator=g)
    mass = sparse.block_mass(q, k, 0.088, True)
    idx = sparse.select_blocks(mass, n, 6, True, 1, 2)
    last = [t[:, -1:].cpu() for t in (q, k, v, do, idx, mass)]
    ref_mass = oracle_block_mass(last[0], last[1], 0.088, True)
    close(last[5], ref_mass, mass_tol(last[0], last[1], 0.088, ref_mass, True), "mass")
    assert torch.equal(last[4], oracle_block_select(last[5], n, 6, True, 1, 2))
    out, lse = sparse.streamkl_sparse_attn_fwd(q, k, v, idx, 0.088, True)
    tol = {}
    ref = oracle_sparse_attn(*last[:3], last[4], 0.088, True, None, last[3], tol)
    close(out[:, -1:], ref[0], tol["out"], "out")
    dq, dk, dv = sparse.streamkl_sparse_attn_bwd(q, k, v, out, lse, do, idx, 0.088, True)
    for name, x, r in zip(("dq", "dk", "dv"), (dq, dk, dv), ref[2:]):
        close(x[:, -1:], r, tol[name], name)
    assert skl.device_status() == 0


def test_bad_lengths_are_reported_and_read_as_empty():
    q, k, v, _ = (t.cuda() for t in inputs(2, 4, 2, 3, 130, 64, seed=8))
    idx = torch.zeros(2, 2, 3, 1, dtype=torch.int32, device="cuda")
    for bad in (-1, 131):
        lens = torch.tensor([130, bad], dtype=torch.int32, device="cuda")
        out, lse = sparse.sparse_attention(q, k, v, idx, causal=True, seqlens_k=lens, return_lse=True)
        assert skl.device_status() == 1
        assert (out[1] == 0).all() and (lse[1] == -math.inf).all() and torch.isfinite(lse[0]).all()
        assert (sparse.block_mass(q, k, seqlens_k=lens)[1] == 0).all()
        assert skl.device_status() == 1
    with pytest.raises(ValueError):
        sparse.sparse_attention(q, k, v, idx.long())
    with pytest.raises(ValueError):
        sparse.sparse_attention(q, k, v.float(), idx)
    with pytest.raises(ValueError):
        sparse.select_blocks(torch.zeros(1, 1, 1, 3, device="cuda"), 64, 1)
    with pytest.raises(skl.StreamKLError):
        sparse.select_blocks(torch.zeros(1, 1, 1, 1, device="cuda"), 64, 1, n_first=1, n_last=1)


def test_backward_reports_a_length_that_went_bad_after_the_forward():
    q, k, v, do = (t.cuda() for t in inputs(2, 4, 2, 3, 130, 64, seed=9))
    idx = torch.zeros(2, 2, 3, 1, dtype=torch.int32, device="cuda")
    lens = torch.tensor([130, 70], dtype=torch.int32, device="cuda")
    leaves = [t.requires_grad_() for t in (q, k, v)]
    try:
        set_check_status(True)
        out = sparse.sparse_attention(*leaves, idx, causal=True, seqlens_k=lens)
        lens.data.fill_(131)
        with pytest.raises(skl.StreamKLError, match="backward"):
            out.backward(do)
    finally:
        set_check_status(False)
    assert all(t.grad is None for t in leaves) and skl.device_status() == 0


def test_captured_step_of_a_user():
    q, k, v, do = (t.cuda() for t in inputs(1, 4, 2, 70, 300, 64, seed=11))
    idx = lists(1, 2, 70, 300, 4, seed=11).cuda()
    eager = [t.clone().requires_grad_() for t in (q, k, v)]
    out = sparse.sparse_attention(*eager, idx, causal=True)
    ref = torch.autograd.grad(out, eager, do, retain_graph=True)
    fresh = [t.clone().requires_grad_() for t in (q, k, v)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        # The leaves of the graph that still lives are refused, its detached ones are not.
        with pytest.raises(RuntimeError, match="q is part of a graph made on the default stream"):
            sparse.sparse_attention(*eager, idx, causal=True)
        with pytest.raises(RuntimeError, match="v is part of a graph"):
            sparse.sparse_attention(*fresh[:2], eager[2], idx, causal=True)
        o = sparse.sparse_attention(*fresh, idx, causal=True)
        d = torch.autograd.grad(o, fresh, do)
    for t in (o, *d):
        t.detach().zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, out) and all(torch.equal(a, b) for a, b in zip(d, ref))
    assert skl.device_status() == 0


def test_gradients_are_not_differentiated_again():
    q, k, v, do = (t.cuda() for t in inputs(1, 4, 2, 20, 130, 64, seed=12))
    idx = lists(1, 2, 20, 130, 2, seed=12).cuda()
    leaves = [t.requires_grad_() for t in (q, k, v)]
    out = sparse.sparse_attention(*leaves, idx, causal=True)
    once = torch.autograd.grad(out, leaves, do, retain_graph=True)
    kept = torch.autograd.grad(out, leaves, do, create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(once, kept))
    with pytest.raises(RuntimeError, match="differentiable once"):
        kept[0].sum().backward()


def test_calls_on_a_fresh_thread():
    """A serving thread's first CUDA work may be a single-token call."""
    q, k, v, _ = (t.cuda() for t in inputs(2, 4, 2, 1, 300, 64, seed=13))
    idx = lists(2, 2, 1, 300, 3, seed=13).cuda()
    lse = sparse.streamkl_sparse_attn_fwd(q, k, v, idx, 0.125, True)[1]
    calls = [lambda: sparse.sparse_attention(q, k, v, idx, causal=True),
             lambda: sparse.block_mass(q, k, causal=True),
             lambda: sparse.block_mass(q, k, causal=True, lse=lse),
             lambda: sparse.select_blocks(torch.zeros(1, 1, 1, 5, device="cuda"), 300, 3)]
    for call in calls:
        want = call()
        torch.cuda.synchronize()
        got = []
        thread = threading.Thread(target=lambda: got.append(call()))
        thread.start()
        thread.join()
        torch.cuda.synchronize()
        assert got and torch.equal(got[0], want)


def test_what_follows_in_the_stream_follows_every_kernel_of_the_call():
    """Kernels of a call overlap: one block that every query lists keeps dK and dV busy long after
    dQ is done, and one query that lists every block keeps the last tile of dQ busy."""
    q, k, v, do = (t.cuda() for t in inputs(1, 4, 1, 6000, 6000, 128, seed=14))
    one = torch.zeros(1, 1, 6000, 94, dtype=torch.int32, device="cuda")
    all_ = torch.arange(94, dtype=torch.int32, device="cuda").expand(1, 1, 6000, 94).contiguous()
    idx = torch.empty_like(one)
    wants = []
    for lists_ in (one, all_):
        out, lse = sparse.streamkl_sparse_attn_fwd(q, k, v, lists_, 0.1, False)
        g = sparse.streamkl_sparse_attn_bwd(q, k, v, out, lse, do, lists_, 0.1, False)
        torch.cuda.synchronize()
        wants.append([out, lse, *g])
    for _ in range(3):
        for lists_, want in zip((one, all_), wants):
            idx.copy_(lists_)  # a kernel right before the call writes what it reads
            out, lse = sparse.streamkl_sparse_attn_fwd(q, k, v, idx, 0.1, False)
            grads = [torch.full_like(t, NAN) for t in (q, k, v)]
            sparse.streamkl_sparse_attn_bwd(q, k, v, out, lse, do, idx, 0.1, False, dq=grads[0],
                                            dk=grads[1], dv=grads[2])
            early = [t.clone() for t in (out, lse, *grads)]  # and kernels right after read it
            idx.fill_(-1)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(early, want))
    assert skl.device_status() == 0
