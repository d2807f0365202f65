"""fp64 CPU oracle of the block-sparse attention operators (test infrastructure only).

Everything is materialised per head in float64 from the inputs as they are; no code is shared
with the CUDA library. ``seqlens_k`` gives the keys of each padded sequence; blocks are 64 keys.

    mass[b, hk, i, c] = mean over the heads of a K head of sum_{j in block c} P[h, i, j]
    out[b, h, i]      = softmax over the allowed keys of the listed blocks, times V
"""
from __future__ import annotations

import torch

F64 = torch.float64
BLOCK = 64


def _f64(t):
    return t.detach().cpu().to(F64)


def _lens(seqlens_k, B, n_k):
    return [n_k] * B if seqlens_k is None else [int(n) for n in seqlens_k]


def _allowed(n_q, n_k, n, causal):
    """[n_q, n_k] keys each query may read of a sequence with n of n_k keys."""
    i, j = torch.arange(n_q)[:, None], torch.arange(n_k)[None, :]
    ok = (j < n).expand(n_q, n_k)
    return ok & (j <= i + n - n_q) if causal else ok


def _scores(q, k, scale, ok):
    """Scores with -inf where not allowed; K rows that no query may read count as 0 (they may
    hold anything)."""
    k = torch.where(ok.any(0)[:, None], k, torch.zeros_like(k))
    return torch.where(ok, (q @ k.T) * scale, torch.full(ok.shape, float("-inf"), dtype=F64))


def _softmax(s):
    """Row softmax and log-sum-exp; a row without keys is all 0 and -inf."""
    lse = torch.logsumexp(s, -1)
    p = (s - torch.where(lse > float("-inf"), lse, torch.zeros_like(lse))[:, None]).exp()
    return p, lse


def oracle_block_mass(q, k, scale, causal, seqlens_k=None, lse=None):
    B, H, n_q, _ = q.shape
    h_kv, n_k = k.shape[1], k.shape[2]
    nb, G = (n_k + BLOCK - 1) // BLOCK, H // k.shape[1]
    out = torch.zeros(B, h_kv, n_q, nb, dtype=F64)
    for b, n in enumerate(_lens(seqlens_k, B, n_k)):
        ok = _allowed(n_q, n_k, n, causal)
        for h in range(H):
            s = _scores(_f64(q[b, h]), _f64(k[b, h // G]), scale, ok)
            p, own = _softmax(s)
            if lse is not None:
                given = _f64(lse[b, h])
                p = torch.where((given > float("-inf"))[:, None], (s - given[:, None]).exp(),
                                torch.zeros_like(s))
            p = torch.nn.functional.pad(p, (0, nb * BLOCK - n_k)).view(n_q, nb, BLOCK).sum(-1)
            out[b, h // G] += p / G
    return out


def oracle_block_select(mass, n_k, topk, causal, n_first, n_last, seqlens_k=None):
    """One row at a time, by sorting Python tuples."""
    B, Hs, n_q, nb = mass.shape
    out = torch.full((B, Hs, n_q, topk), -1, dtype=torch.int32)
    for b, n in enumerate(_lens(seqlens_k, B, n_k)):
        for i in range(n_q):
            last = min(n - 1, i + n - n_q) if causal else n - 1
            vis = last // BLOCK + 1 if last >= 0 else 0
            for h in range(Hs):
                row = mass[b, h, i].tolist()
                rank = []
                for c in range(vis):
                    x = row[c]
                    first = 0 if c < n_first or c >= vis - n_last else (2 if x != x else 1)
                    rank.append((first, -x if first == 1 else 0.0, c))
                pick = sorted(c for _, _, c in sorted(rank)[:topk])
                out[b, h, i, :len(pick)] = torch.tensor(pick, dtype=torch.int32)
    return out


def selected_keys(block_idx, n_k):
    """Boolean [..., n_k] from lists of blocks: a set, entries outside the blocks ignored."""
    nb = (n_k + BLOCK - 1) // BLOCK
    idx = block_idx.cpu().long()
    idx = torch.where((idx >= 0) & (idx < nb), idx, torch.full_like(idx, nb))
    sel = torch.zeros(*idx.shape[:-1], nb + 1, dtype=torch.bool)
    sel.scatter_(-1, idx, True)
    return sel[..., :nb].repeat_interleave(BLOCK, -1)[..., :n_k]


def oracle_sparse_attn(q, k, v, block_idx, scale, causal, seqlens_k=None, dout=None, bounds=None):
    """out, lse and, given dout, dq, dk, dv. ``bounds`` (a dict) receives, per result, a bound on
    the error of a computation that rounds P and dS to bf16 for the products, out and the
    gradients to bf16 once, and keeps everything else in fp32 (see below)."""
    B, H, n_q, d = q.shape
    h_kv, n_k = k.shape[1], k.shape[2]
    G, Gs = H // h_kv, H // block_idx.shape[1]
    sel = selected_keys(block_idx, n_k)
    out, lse = torch.zeros(B, H, n_q, d, dtype=F64), torch.zeros(B, H, n_q, dtype=F64)
    dq = torch.zeros_like(out)
    dk, dv = torch.zeros(B, h_kv, n_k, d, dtype=F64), torch.zeros(B, h_kv, n_k, d, dtype=F64)
    tol = {n: torch.zeros_like(t) for n, t in
           (("out", out), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv))}
    half, tiny = 2.0 ** -8, 2.0 ** -126  # half a step of bf16, relative; least fp32 normal
    for b, n in enumerate(_lens(seqlens_k, B, n_k)):
        base = _allowed(n_q, n_k, n, causal)
        live = (torch.arange(n_k) < n)[:, None]
        for h in range(H):
            qq = _f64(q[b, h])
            kk = torch.where(live, _f64(k[b, h // G]), torch.zeros(1, dtype=F64))
            vv = torch.where(live, _f64(v[b, h // G]), torch.zeros(1, dtype=F64))
            ok = base & sel[b, h // Gs]
            s = _scores(qq, kk, scale, ok)
            p, l = _softmax(s)
            o = p @ vv
            out[b, h], lse[b, h] = o, l
            # A score's fp32 error: d products and sums of at most 2^-23 of their absolute sum
            # (tensor cores truncate, hence a whole step), and the exponent's argument, product
            # with log2 e included, to 4 steps of its size; 2^-21 for the exponential and sums.
            mag = (qq.abs() @ kk.abs().T) * abs(scale)
            reach = torch.where(ok, mag, torch.zeros_like(mag)).amax(-1)
            e_s = (d * reach * 2.0 ** -23 + 8 * 2.0 ** -23 * (1 + 2 * reach) + 2.0 ** -21
                   + n_k * 2.0 ** -24)
            tol["lse"][b, h] = e_s
            # Rounded probabilities: relative, and, as fp32 flushes what lies below its least
            # normal number 2^-126, that much in absolute terms; so for dS and every result.
            e_p = (half + 3 * e_s)[:, None] * p + tiny
            e_o = e_p @ vv.abs() + half * o.abs() + tiny
            tol["out"][b, h] = e_o
            if dout is None:
                continue
            do = _f64(dout[b, h])
            dP = do @ vv.T
            D = (do * o).sum(-1, keepdim=True)
            ds = p * (dP - D)
            dv[b, h // G] += p.T @ do
            dq[b, h] = ds @ kk * scale
            dk[b, h // G] += ds.T @ qq * scale
            # dS: its rounding, the relative error of p, fp32 errors of dP and D, and D formed
            # from the rounded out, except where a query sees one block at most (D from its keys).
            e_d = (do.abs() * e_o).sum(-1, keepdim=True)
            own = 3 * e_s[:, None] * (p * dP.abs()).sum(-1, keepdim=True)
            e_d = torch.where(base.sum(-1, keepdim=True) <= BLOCK, own, e_d)
            f32 = d * 2.0 ** -23 * (do.abs() @ vv.abs().T + (do * o).abs().sum(-1, keepdim=True))
            e_ds = half * ds.abs() + 3 * e_s[:, None] * p * (dP.abs() + D.abs()) \
                + (1 + half) * p * (e_d + f32) + tiny * (1 + dP.abs() + D.abs())
            tol["dv"][b, h // G] += e_p.T @ do.abs() + tiny
            tol["dq"][b, h] = e_ds @ kk.abs() * abs(scale) + half * dq[b, h].abs() + tiny
            tol["dk"][b, h // G] += e_ds.T @ qq.abs() * abs(scale) + tiny
    tol["dk"] += half * dk.abs()
    tol["dv"] += half * dv.abs()
    if bounds is not None:
        bounds.update(tol)
    return (out, lse) if dout is None else (out, lse, dq, dk, dv)
