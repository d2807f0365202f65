"""Measured cases of the block-sparse attention operators, with their plain forms.

A distilled student map picks, for every query, the blocks of 64 keys that the full
attention then reads:

  mass    probability mass of the student's attention map on each key block, averaged over
          the query heads that share a K head;
  select  the blocks each query reads: the first ones, the last visible ones, and the
          heaviest of the rest, ascending, -1 behind the last;
  attn    softmax attention over the selected blocks (forward);
  train   the same with its gradients dQ, dK, dV.

`run` computes a case in elementary torch operations in fp32 (``own = False``) or through the
package's entry points (``own = True``).
"""
import math

import torch

own = False

BLOCK = 64
DEV = "cuda"


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def listed():
    return [
        # One training step's student map (batch 2, 16 heads in groups of four, 4096 tokens):
        # the log-sum-exps are at hand from the divergence's forward.
        dict(name="mass_step_4096", op="mass", B=2, H=16, Hkv=4, nq=4096, nk=4096, d=128, causal=True,
             lse=True, ragged=False),
        # Long-context distillation, one sequence of 16384 tokens with a 64-wide student.
        dict(name="mass_long_16384", op="mass", B=1, H=32, Hkv=8, nq=16384, nk=16384, d=64, causal=True,
             lse=True, ragged=False),
        # Serving: one new token of each of 16 sequences against a padded student key cache.
        dict(name="mass_token_b16", op="mass", B=16, H=32, Hkv=8, nq=1, nk=32768, d=64, causal=True,
             lse=False, ragged=True),
        # Serving, one short sequence: latency.
        dict(name="mass_token_b1", op="mass", B=1, H=8, Hkv=2, nq=1, nk=4097, d=64, causal=True,
             lse=False, ragged=False),
        # Selection for every token of a 16384-token sequence and 8 K heads.
        dict(name="select_long_16384", op="select", B=1, Hs=8, nq=16384, nk=16384, causal=True, topk=16,
             first=1, last=2, ragged=False),
        # Selection for one new token of 64 sequences of up to 65536 tokens.
        dict(name="select_token_b64", op="select", B=64, Hs=8, nq=1, nk=65536, causal=True, topk=32,
             first=1, last=2, ragged=True),
        # Prompt processing: 16384 tokens, 32 heads over 8 K heads, 32 blocks per query.
        dict(name="attn_prompt_16384", op="attn", B=1, H=32, Hkv=8, Hs=8, nq=16384, nk=16384, d=128,
             causal=True, topk=32, own_pct=15, ragged=False),
        # Serving: one new token of 32 sequences against padded caches.
        dict(name="attn_token_b32", op="attn", B=32, H=32, Hkv=8, Hs=8, nq=1, nk=16384, d=128,
             causal=True, topk=16, own_pct=15, ragged=True),
        # Serving, one long sequence: latency.
        dict(name="attn_token_b1", op="attn", B=1, H=32, Hkv=8, Hs=8, nq=1, nk=65536, d=128,
             causal=True, topk=32, own_pct=15, ragged=False),
        # A training step at batch 2, 16 heads, 4096 tokens.
        dict(name="train_step_4096", op="train", B=2, H=16, Hkv=4, Hs=4, nq=4096, nk=4096, d=128,
             causal=True, topk=16, own_pct=15, ragged=False),
        # A short odd-sized step, one K head per query head, narrow heads, keys before the queries.
        dict(name="train_odd_1337", op="train", B=2, H=8, Hkv=8, Hs=8, nq=1337, nk=2001, d=64,
             causal=True, topk=8, own_pct=15, ragged=False),
        # Long-context training.
        dict(name="train_long_16384", op="train", B=1, H=16, Hkv=4, Hs=4, nq=16384, nk=16384, d=128,
             causal=True, topk=32, own_pct=15, ragged=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["mass", "mass", "select", "attn", "attn", "train", "train"])
    token = op != "train" and rng.random() < 0.4
    if op == "select":
        c = dict(op=op, Hs=rng.choice([1, 2, 4, 8]), causal=rng.random() < 0.8, topk=rng.randint(1, 64),
                 first=0, last=0, ragged=rng.random() < 0.5)
        c["first"] = rng.randint(0, min(2, c["topk"]))
        c["last"] = rng.randint(0, min(3, c["topk"] - c["first"]))
        if token:
            return c | dict(B=_log_int(rng, 1, 64), nq=1, nk=_log_int(rng, 64, 131072))
        nq = _log_int(rng, 32, 16384)
        nk = nq + rng.choice([0, rng.randint(0, 4096)])
        return c | dict(B=rng.randint(1, 2) if nq < 8192 else 1, nq=nq, nk=nk)
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 4, 6, 8])
    c = dict(op=op, H=Hkv * G, Hkv=Hkv, d=rng.choice([64, 128]), causal=rng.random() < 0.8)
    if token:
        c |= dict(B=_log_int(rng, 1, 32), nq=rng.choice([1, 1, 1, 2, 5]), nk=_log_int(rng, 64, 32768),
                  ragged=rng.random() < 0.7)
    else:
        nq = _log_int(rng, 100, 6000)
        nk = nq if rng.random() < 0.5 else nq + rng.randint(1, 2000)
        c |= dict(B=1 if nq > 3000 else rng.randint(1, 3), nq=nq, nk=nk, ragged=rng.random() < 0.2)
    if op == "mass":
        return c | dict(lse=not token)
    return c | dict(Hs=rng.choice([Hkv, Hkv, 1]), topk=_log_int(rng, 2, 48), own_pct=rng.choice([0, 15, 50]))


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _lens(case, g):
    """Key counts of a padded batch: between a quarter of the cache and all of it."""
    if not case["ragged"]:
        return None
    n = case["nk"]
    lo = max(1, n // 4, min(n, case["nq"]))
    return torch.randint(lo, n + 1, (case["B"],), generator=g, device=DEV, dtype=torch.int32)


def _normal(shape, g, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _last_key(case, lens):
    """[B, nq] index of the last key each query may read (-1: none)."""
    nk = torch.full((case["B"],), case["nk"], device=DEV) if lens is None else lens.long()
    i = torch.arange(case["nq"], device=DEV)
    if case["causal"]:
        return (i[None, :] + (nk - case["nq"])[:, None]).clamp(min=-1)
    return (nk - 1)[:, None].expand(-1, case["nq"])


def prepare(case, seed):
    g = _gen(seed)
    lens = _lens(case, g)
    last = _last_key(case, lens)
    s = dict(case=case, lens=lens)
    B, nq, nk = case["B"], case["nq"], case["nk"]
    if case["op"] == "select":
        # Masses of a peaked map: exponentials of normal scores, normalised over the blocks.
        m = torch.randn((B, case["Hs"], nq, _blocks(nk)), generator=g, device=DEV).mul_(1.5).exp_()
        vis = torch.arange(_blocks(nk), device=DEV) * BLOCK <= last[:, None, :, None]
        m *= vis
        s["mass"] = m / m.sum(-1, keepdim=True).clamp_(min=1e-30)
        return s
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    s["q"] = _normal((B, H, nq, d), g)
    s["k"] = _normal((B, Hkv, nk, d), g)
    s["scale"] = 1.0 / math.sqrt(d)
    if case["op"] == "mass":
        s["lse"] = torch.empty(B, H, nq, device=DEV) if case["lse"] else None
        for bh in range(B * H if case["lse"] else 0):  # one head's map at a time
            b, h = divmod(bh, H)
            t = (s["q"][b, h].float() @ s["k"][b, h // (H // Hkv)].float().T).mul_(s["scale"])
            t.masked_fill_(torch.arange(nk, device=DEV) > last[b][:, None], -math.inf)
            s["lse"][b, h] = torch.logsumexp(t, -1)
        return s
    s["v"] = _normal((B, Hkv, nk, d), g)
    if case["op"] == "train":
        s["dout"] = _normal((B, H, nq, d), g)
    # Selections as a distilled map gives them: the first block, the last two visible ones, and
    # blocks that neighbouring queries largely share (own_pct: how far a query's own choice moves).
    nb = _blocks(nk)
    seg = torch.rand((B, case["Hs"], (nq + 127) // 128, nb), generator=g, device=DEV)
    score = seg.repeat_interleave(128, 2)[:, :, :nq]
    score = score + case["own_pct"] / 100 * torch.rand(score.shape, generator=g, device=DEV)
    c = torch.arange(nb, device=DEV)
    top = (torch.div(last, BLOCK, rounding_mode="floor"))[:, None, :, None]
    score = score + 4 * ((c == 0) | (c > top - 2))
    score = score.masked_fill_(c > top, -math.inf)
    val, idx = score.topk(min(case["topk"], nb), -1)
    idx = torch.where(val > -math.inf, idx, nb).sort(-1).values
    s["idx"] = torch.where(idx < nb, idx, -1).int()
    if s["idx"].shape[-1] < case["topk"]:
        s["idx"] = torch.nn.functional.pad(s["idx"], (0, case["topk"] - s["idx"].shape[-1]), value=-1)
    s["idx"] = s["idx"].contiguous()
    return s


# ------------------------------------------------------------------ plain forms


def _plain_mass(s):
    c = s["case"]
    B, H, Hkv, nq, nk = c["B"], c["H"], c["Hkv"], c["nq"], c["nk"]
    q = s["q"].float().view(B, Hkv, (H // Hkv) * nq, -1)
    p = torch.matmul(q, s["k"].float().transpose(-1, -2)).mul_(s["scale"]).view(B, H, nq, nk)
    hide = torch.arange(nk, device=DEV) > _last_key(c, s["lens"])[:, None, :, None]
    p.masked_fill_(hide, -math.inf)
    lse = s["lse"] if s["lse"] is not None else torch.logsumexp(p, -1)
    p.sub_(torch.where(lse > -math.inf, lse, 0.0)[..., None]).exp_()
    if nk % BLOCK:
        p = torch.nn.functional.pad(p, (0, -nk % BLOCK))
    p = p.view(B, H, nq, -1, BLOCK).sum(-1)
    return p.view(B, Hkv, H // Hkv, nq, -1).mean(2)


def _plain_select(s):
    c, m = s["case"], s["mass"]
    nb, k = m.shape[-1], c["topk"]
    i = torch.arange(nb, device=DEV)
    vis = (torch.div(_last_key(c, s["lens"]), BLOCK, rounding_mode="floor") + 1)[:, None, :, None]
    forced = (i < c["first"]) | (i >= vis - c["last"])
    key = torch.where(forced, math.inf, m).masked_fill(i >= vis, -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :k]
    order = torch.where(order < vis, order, nb).sort(-1).values
    order = torch.where(order < nb, order, -1).int()
    return torch.nn.functional.pad(order, (0, k - order.shape[-1]), value=-1)


def _hidden(s):
    """[B, Hkv, 1, nq, nk] True where a query does not read a key."""
    c = s["case"]
    B, Hkv, Hs, nq, nk = c["B"], c["Hkv"], c["Hs"], c["nq"], c["nk"]
    nb = _blocks(nk)
    idx = s["idx"].long()
    sel = torch.zeros(B, Hs, nq, nb + 1, dtype=torch.bool, device=DEV)
    sel.scatter_(-1, torch.where(idx >= 0, idx, nb), True)
    hide = ~sel[..., :nb].repeat_interleave(BLOCK, -1)[..., :nk]
    hide |= torch.arange(nk, device=DEV) > _last_key(c, s["lens"])[:, None, :, None]
    return hide.repeat_interleave(Hkv // Hs, 1)[:, :, None]


def _softmax_(p):
    """In-place softmax of the last axis; rows without a finite entry become 0."""
    m = p.amax(-1, keepdim=True)
    p.sub_(torch.where(m > -math.inf, m, 0.0)).exp_()
    return p.div_(p.sum(-1, keepdim=True).clamp_(min=1e-30))


def _plain_token(s):
    """Forward of single tokens: only the selected keys are gathered."""
    c = s["case"]
    B, H, Hkv, nk = c["B"], c["H"], c["Hkv"], c["nk"]
    idx = s["idx"][:, :, 0].long().repeat_interleave(Hkv // c["Hs"], 1)
    key = (idx[..., None] * BLOCK + torch.arange(BLOCK, device=DEV)).flatten(2)
    hide = (key < 0) | (key > _last_key(c, s["lens"])[:, None, :])
    at = key.clamp(0, nk - 1)[..., None].expand(-1, -1, -1, c["d"])
    k, v = s["k"].gather(2, at).float(), s["v"].gather(2, at).float()
    q = s["q"].float().view(B, Hkv, H // Hkv, -1)
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])
    p = _softmax_(p.masked_fill_(hide[:, :, None], -math.inf))
    return torch.matmul(p, v).view(B, H, 1, -1).to(torch.bfloat16)


def _plain_attn(s):
    c = s["case"]
    if c["nq"] == 1 and c["op"] == "attn":
        return _plain_token(s)
    B, H, Hkv, nq, nk, d = c["B"], c["H"], c["Hkv"], c["nq"], c["nk"], c["d"]
    G = H // Hkv
    q = s["q"].float().view(B, Hkv, G * nq, d)
    k, v = s["k"].float(), s["v"].float()
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])
    p.view(B, Hkv, G, nq, nk).masked_fill_(_hidden(s), -math.inf)
    p = _softmax_(p)
    o = torch.matmul(p, v)
    out = o.view(B, H, nq, d).to(torch.bfloat16)
    if c["op"] == "attn":
        return out
    do = s["dout"].float().view(B, Hkv, G * nq, d)
    dv = torch.matmul(p.transpose(-1, -2), do)
    ds = torch.matmul(do, v.transpose(-1, -2))
    ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    del p
    dq = torch.matmul(ds, k).mul_(s["scale"]).view(B, H, nq, d)
    dk = torch.matmul(ds.transpose(-1, -2), q).mul_(s["scale"])
    return dict(out=out, dq=dq.to(torch.bfloat16), dk=dk.to(torch.bfloat16), dv=dv.to(torch.bfloat16))


def run(state):
    c = state["case"]
    if not own:
        return {"mass": _plain_mass, "select": _plain_select}.get(c["op"], _plain_attn)(state)
    from attention_kl_divergence_fwd_b200 import sparse
    if c["op"] == "mass":
        return sparse.block_mass(state["q"], state["k"], scale=state["scale"], causal=c["causal"],
                                 lse=state["lse"], seqlens_k=state["lens"])
    if c["op"] == "select":
        return sparse.select_blocks(state["mass"], c["nk"], c["topk"], causal=c["causal"],
                                    n_first=c["first"], n_last=c["last"], seqlens_k=state["lens"])
    if c["op"] == "attn":
        return sparse.sparse_attention(state["q"], state["k"], state["v"], state["idx"],
                                       scale=state["scale"], causal=c["causal"],
                                       seqlens_k=state["lens"])
    q, k, v = (state[n].detach().requires_grad_() for n in "qkv")
    out = sparse.sparse_attention(q, k, v, state["idx"], scale=state["scale"], causal=c["causal"],
                                  seqlens_k=state["lens"])
    dq, dk, dv = torch.autograd.grad(out, (q, k, v), state["dout"])
    return dict(out=out, dq=dq, dk=dk, dv=dv)


# ------------------------------------------------------- least work and exact values


def work(case):
    """Each input read once and each output written once (of a cache, the selected blocks when
    they are fewer), and the products of the pairs that are read. Padded batches count as full."""
    B, nq, nk = case["B"], case["nq"], case["nk"]
    nb = _blocks(nk)
    off = nk - nq
    seen = [max(0, min(nk, i + off + 1)) if case["causal"] else nk for i in range(nq)]
    if case["op"] == "select":
        vis = sum(_blocks(n) for n in seen)
        return dict(bytes=4.0 * B * case["Hs"] * (vis + nq * case["topk"]), flops=0)
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    qb, kb = 2.0 * B * H * nq * d, 2.0 * B * Hkv * nk * d
    if case["op"] == "mass":
        out = 4.0 * B * Hkv * nq * nb
        return dict(bytes=qb + kb + out + (4.0 * B * H * nq if case["lse"] else 0),
                    flops=2.0 * d * B * H * sum(seen))
    pairs = float(B * H * sum(min(n, case["topk"] * BLOCK) for n in seen))
    ib = 4.0 * B * case["Hs"] * nq * case["topk"]
    kb = min(kb, 2.0 * B * Hkv * nq * case["topk"] * BLOCK * d)
    if case["op"] == "attn":
        return dict(bytes=2 * qb + 2 * kb + ib, flops=4.0 * d * pairs)
    return dict(bytes=4 * qb + 4 * kb + ib, flops=14.0 * d * pairs)


def exact(case, seed):
    """The definition in fp64, one head at a time, from the same inputs."""
    if case["op"] == "select":
        return None
    s = prepare(case, seed)
    B, H, Hkv, nq, nk, d = (case[n] for n in ("B", "H", "Hkv", "nq", "nk", "d"))
    G, nb = H // Hkv, _blocks(nk)
    j = torch.arange(nk, device=DEV)
    lens = [nk] * B if s["lens"] is None else s["lens"].tolist()
    row = torch.arange(nq, device=DEV)[:, None]
    if case["op"] == "mass":
        out = torch.zeros(B, Hkv, nq, nb, dtype=torch.float64, device=DEV)
    else:
        out = torch.zeros(B, H, nq, d, dtype=torch.float64, device=DEV)
        dq, dk, dv = torch.zeros_like(out), *(torch.zeros(B, Hkv, nk, d, dtype=torch.float64, device=DEV)
                                              for _ in range(2))
    for b in range(B):
        n = lens[b]
        ok = j[None, :n] <= (row + n - nq if case["causal"] else n + 0 * row)
        for h in range(H):
            g = h // G
            q, k = s["q"][b, h].double(), s["k"][b, g, :n].double()
            allowed = ok
            if case["op"] != "mass":
                idx = s["idx"][b, g // (Hkv // case["Hs"])].long()
                pick = torch.zeros(nq, nb + 1, device=DEV)
                pick[row.expand_as(idx), torch.where(idx < 0, nb, idx)] = 1
                allowed = ok & (pick[:, torch.div(j[:n], BLOCK, rounding_mode="floor")] > 0)
            t = (q @ k.T) * s["scale"]
            e = torch.where(allowed, t, torch.full_like(t, -math.inf))
            if case["op"] == "mass":
                if s["lse"] is None:
                    p = torch.softmax(e, -1).nan_to_num_(0.0)
                else:
                    p = torch.where(allowed, (e - s["lse"][b, h].double()[:, None]).exp(), 0.0)
                at = torch.div(j[:n], BLOCK, rounding_mode="floor").expand(nq, n)
                out[b, g].scatter_add_(1, at, p / G)
                continue
            p = torch.softmax(e, -1).nan_to_num_(0.0)
            v = s["v"][b, g, :n].double()
            out[b, h] = p @ v
            if case["op"] == "train":
                do = s["dout"][b, h].double()
                dv[b, g, :n] += p.T @ do
                ds = p * (do @ v.T - (do * out[b, h]).sum(-1, keepdim=True)) * s["scale"]
                dq[b, h] = ds @ k
                dk[b, g, :n] += ds.T @ q
    if case["op"] != "train":
        return out
    return dict(out=out, dq=dq, dk=dk, dv=dv)
