"""Block-sparse attention steered by a distilled attention map.

The divergence of ``attention_kl`` trains a student map towards a teacher's. Cut into blocks of
64 keys, the student map then says which keys full attention has to read:

    kl, _, lse_s = streamkl_fwd(q_t, k_t, q_s, k_s, ...)            # training: the map's loss
    mass = block_mass(q_s, k_s, causal=True, lse=lse_s)             # [B, H_kv, N_Q, NB] fp32
    idx = select_blocks(mass, n_k, topk=16, causal=True)            # [B, H_kv, N_Q, 16] int32
    out = sparse_attention(q, k, v, idx, causal=True)               # differentiable in q, k, v

and, serving one token against a padded cache (``seqlens_k``: keys of each sequence), the same
calls with ``N_Q = 1`` and without ``lse``; ``student_sparse_attention`` makes the three in a row.

Tensors are bf16 [B, heads, N, d] on one CUDA device, d in {64, 128}; K heads may be shared by a
group of query heads, and one selection may serve several K heads. Views that are not contiguous or
begin at no multiple of 16 bytes are copied by the call (the raw ``streamkl_*`` calls refuse them).
The first ``seqlens_k`` (or N_K) keys and values, and all queries and output gradients, have to be
finite: queries are computed in tiles, and a NaN or infinity in a block that one query of a tile
lists can reach the tile's others. What a padded cache holds behind them may be anything. Calls run
on the current (or the given) stream and allocate outputs and workspace from PyTorch's allocator,
which makes them safe to capture into a CUDA graph (a backward through ``torch.autograd.grad``:
``.backward()`` accumulates into leaves on the stream where eager code first used them; leaves whose
eager graph from the default stream still lives are refused while capturing, and so is the captured
backward of inputs that eager code computed there). With status checks on
(``autograd.set_check_status``, read by the forward for its backward too) every call waits for its
kernels and raises their errors. The selection has no gradient, the attention's gradients are not
differentiable again, and forward-mode derivatives (``torch.autograd.forward_ad``) through the
attention are refused.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import inspect
import math
import os
import sys
from typing import Optional

import torch

from . import LIB_PATH, StreamKLError, _check, autograd, load_library

BLOCK = 64  # keys per block
DISPATCH_PATH = os.path.join(os.path.dirname(LIB_PATH), "_sparse_dispatch.so")


_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
# The raw lookups behind torch.cuda.current_device() and current_stream().cuda_stream.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _on_device(fn):
    """Runs an entry point on the device of its first tensor, made current when it is not.
    Single-token calls take a few microseconds on the GPU, so the common path costs one lookup."""
    name = next(iter(inspect.signature(fn).parameters))

    @functools.wraps(fn)
    def wrapper(*args, **kwargs):
        dev = (args[0] if args else kwargs[name]).get_device()
        if dev < 0:
            raise ValueError(f"{fn.__name__}: tensors must be on a CUDA device")
        if dev == _current_device():
            return fn(*args, **kwargs)
        with torch.cuda.device(dev):
            return fn(*args, **kwargs)
    return wrapper


def _stream_ptr(stream, dev):
    if stream is None:
        return _current_stream(dev)
    if stream.device_index != dev:
        raise ValueError(f"stream on {stream.device}, tensors on cuda:{dev}")
    return stream.cuda_stream


def num_blocks(n_k: int) -> int:
    """Blocks that n_k keys make up."""
    return (int(n_k) + BLOCK - 1) // BLOCK


def _bf16(name, t, dev, like=None):
    if t.dtype is not _BF16 or t.get_device() != dev or t.dim() != 4 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 4-D bf16 tensor [B, heads, N, d] on cuda:{dev}")
    if like is not None and t.shape != like:
        raise ValueError(f"{name} must have shape {tuple(like)}, got {tuple(t.shape)}")


def _typed(name, t, dev, dtype, shape):
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous() or t.shape != shape:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on "
                         f"cuda:{dev}")
    return t


def _lens(seqlens_k, dev, B):
    if seqlens_k is None:
        return 0
    return _typed("seqlens_k", seqlens_k, dev, _I32, (B,)).data_ptr()


def _new(t, stream):
    """Memory that a call allocates: on another stream than the current one it is not handed out
    again before that stream is past the call."""
    if stream is not None:
        t.record_stream(stream)
    return t


def _workspace(nbytes, like, stream):
    if nbytes <= 0:
        return None, 0
    ws = _new(like.new_empty(nbytes, dtype=torch.uint8), stream)
    return ws, ws.data_ptr()


def _qk_shape(q, k, dev):
    _bf16("q", q, dev)
    _bf16("k", k, dev)
    B, H, n_q, d = q.shape
    Bk, h_kv, n_k, dk = k.shape
    if Bk != B or dk != d:
        raise ValueError("inconsistent shapes of q and k")
    return B, H, h_kv, n_q, n_k, d


def _qkv_shape(q, k, v, block_idx, dev):
    B, H, h_kv, n_q, n_k, d = _qk_shape(q, k, dev)
    _bf16("v", v, dev, k.shape)
    if block_idx.dim() != 4:
        raise ValueError("block_idx must be [B, H_sel, N_Q, topk]")
    _, h_sel, _, topk = block_idx.shape
    _typed("block_idx", block_idx, dev, _I32, (B, h_sel, n_q, topk))
    return B, H, h_kv, h_sel, n_q, n_k, d, topk


@_on_device
def streamkl_block_mass(q_s, k_s, scale_S: float, causal: bool, lse_s=None, seqlens_k=None,
                        mass=None, stream=None):
    """Mass of the map softmax(scale <q_s, k_s>) on every block of 64 keys, averaged over the
    query heads of each K head: fp32 [B, H_kv, N_Q, ceil(N_K / 64)]."""
    dev = q_s.get_device()
    B, H, h_kv, n_q, n_k, d = _qk_shape(q_s, k_s, dev)
    nb = num_blocks(n_k)
    if mass is None:
        mass = _new(q_s.new_empty((B, h_kv, n_q, nb), dtype=_F32), stream)
    else:
        _typed("mass", mass, dev, _F32, (B, h_kv, n_q, nb))
    lib = load_library()
    nbytes = ws = lse = 0
    keep = None
    if lse_s is None:
        nbytes = lib.streamkl_block_mass_workspace(B, H, h_kv, n_q, n_k, d)
        keep, ws = _workspace(nbytes, q_s, stream)
    else:
        lse = _typed("lse_s", lse_s, dev, _F32, (B, H, n_q)).data_ptr()
    st = lib.streamkl_block_mass(
        q_s.data_ptr(), k_s.data_ptr(), _lens(seqlens_k, dev, B), B, H, h_kv, n_q, n_k, d,
        scale_S, bool(causal), lse, ws, nbytes, mass.data_ptr(), _stream_ptr(stream, dev))
    _check(st, "streamkl_block_mass")
    return mass


@_on_device
def streamkl_block_select(mass, n_k: int, causal: bool, topk: int, n_first: int = 1,
                          n_last: int = 1, seqlens_k=None, block_idx=None, stream=None):
    """The blocks each query reads: int32 [B, H_sel, N_Q, topk], ascending, -1 behind the last."""
    if mass.dim() != 4:
        raise ValueError("mass must be [B, H_sel, N_Q, NB]")
    dev = mass.get_device()
    B, h_sel, n_q, nb = mass.shape
    _typed("mass", mass, dev, _F32, (B, h_sel, n_q, nb))
    n_k, topk = int(n_k), int(topk)
    if num_blocks(n_k) != nb:
        raise ValueError(f"mass has {nb} blocks, n_k = {n_k} keys make {num_blocks(n_k)}")
    if block_idx is None:
        block_idx = _new(mass.new_empty((B, h_sel, n_q, max(topk, 0)), dtype=_I32), stream)
    else:
        _typed("block_idx", block_idx, dev, _I32, (B, h_sel, n_q, topk))
    st = load_library().streamkl_block_select(
        mass.data_ptr(), _lens(seqlens_k, dev, B), B, h_sel, n_q, n_k, bool(causal), topk,
        int(n_first), int(n_last), block_idx.data_ptr(), _stream_ptr(stream, dev))
    _check(st, "streamkl_block_select")
    return block_idx


@_on_device
def streamkl_sparse_attn_fwd(q, k, v, block_idx, scale: float, causal: bool, seqlens_k=None,
                             out=None, lse=None, stream=None):
    """Attention of every query over its listed blocks: out bf16 [B, H, N_Q, d] and the
    log-sum-exps fp32 [B, H, N_Q]."""
    dev = q.get_device()
    B, H, h_kv, h_sel, n_q, n_k, d, topk = _qkv_shape(q, k, v, block_idx, dev)
    if out is None:
        out = _new(torch.empty_like(q), stream)
    else:
        _bf16("out", out, dev, q.shape)
    if lse is None:
        lse = _new(q.new_empty((B, H, n_q), dtype=_F32), stream)
    else:
        _typed("lse", lse, dev, _F32, (B, H, n_q))
    lib = load_library()
    nbytes = lib.streamkl_sparse_attn_workspace(B, H, h_kv, h_sel, n_q, n_k, d, topk, 0)
    keep, ws = _workspace(nbytes, q, stream)
    st = lib.streamkl_sparse_attn_fwd(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), block_idx.data_ptr(), _lens(seqlens_k, dev, B), B,
        H, h_kv, h_sel, n_q, n_k, d, topk, scale, bool(causal), ws, nbytes, out.data_ptr(),
        lse.data_ptr(), _stream_ptr(stream, dev))
    _check(st, "streamkl_sparse_attn_fwd")
    return out, lse


@_on_device
def streamkl_sparse_attn_bwd(q, k, v, out, lse, dout, block_idx, scale: float, causal: bool,
                             seqlens_k=None, dq=None, dk=None, dv=None, stream=None):
    """dQ, dK, dV (bf16, the shapes of q, k, v) from the forward's out and lse."""
    dev = q.get_device()
    B, H, h_kv, h_sel, n_q, n_k, d, topk = _qkv_shape(q, k, v, block_idx, dev)
    _bf16("out", out, dev, q.shape)
    _bf16("dout", dout, dev, q.shape)
    _typed("lse", lse, dev, _F32, (B, H, n_q))
    grads = []
    for name, g, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if g is None:
            g = _new(torch.empty_like(like), stream)
        else:
            _bf16(name, g, dev, like.shape)
        grads.append(g)
    dq, dk, dv = grads
    lib = load_library()
    nbytes = lib.streamkl_sparse_attn_workspace(B, H, h_kv, h_sel, n_q, n_k, d, topk, 1)
    keep, ws = _workspace(nbytes, q, stream)
    st = lib.streamkl_sparse_attn_bwd(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), dout.data_ptr(),
        block_idx.data_ptr(), _lens(seqlens_k, dev, B), B, H, h_kv, h_sel, n_q, n_k, d, topk,
        scale, bool(causal), ws, nbytes, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
        _stream_ptr(stream, dev))
    _check(st, "streamkl_sparse_attn_bwd")
    return dq, dk, dv


_dispatch = None


def dispatch_marker() -> str:
    """What a dispatch module has to be built for: its interface to PyTorch and Python is theirs."""
    return f"block-sparse dispatch for PyTorch {torch.__version__}, Python {sys.version_info[:2]}."


def dispatch_current() -> bool:
    """Whether the dispatch module that is there was built for this PyTorch and Python."""
    if not os.path.exists(DISPATCH_PATH):
        return False
    with open(DISPATCH_PATH, "rb") as f:
        return dispatch_marker().encode() in f.read()


def _ext():
    """The C++ side of the calls below (raises OSError if it has not been built for this PyTorch and
    Python): checks, allocations and the autograd node without Python's share of a short call."""
    global _dispatch
    if _dispatch is None:
        lib = load_library()
        if not dispatch_current():
            raise OSError(f"block-sparse dispatch not built for this PyTorch: {DISPATCH_PATH} "
                          "(run python -m attention_kl_divergence_fwd_b200.build)")
        spec = importlib.util.spec_from_file_location("_sparse_dispatch", DISPATCH_PATH)
        ext = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(ext)
        ext.bind([ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.streamkl_block_mass, lib.streamkl_block_mass_workspace, lib.streamkl_block_select,
            lib.streamkl_sparse_attn_workspace, lib.streamkl_sparse_attn_fwd,
            lib.streamkl_sparse_attn_bwd, lib.streamkl_status_string, lib.streamkl_device_status)])
        ext.raise_as(StreamKLError)
        _dispatch = ext
    return _dispatch


def _lens_arg(seqlens_k):
    if seqlens_k is None or (seqlens_k.dtype == torch.int32 and seqlens_k.is_contiguous()):
        return seqlens_k
    return seqlens_k.to(torch.int32).contiguous()


def block_mass(q_s, k_s, scale: Optional[float] = None, causal: bool = False, lse=None,
               seqlens_k=None):
    """Mass of the student map on every block of 64 keys, averaged over the query heads that
    share a K head: fp32 [B, H_kv, N_Q, NB]; a row sums to 1.

    ``lse`` are the map's row log-sum-exps [B, H, N_Q] (``streamkl_fwd``'s lse_s) when they are
    at hand; without them the rows are normalised by their own sums. The default scale is
    1/sqrt(d). Not differentiable: the map is trained by its divergence."""
    if scale is None:
        scale = 1.0 / math.sqrt(q_s.shape[-1])
    if lse is not None:
        lse = lse.detach()
    return _ext().block_mass(q_s.detach(), k_s.detach(), scale, causal, lse, _lens_arg(seqlens_k),
                             autograd._check_status)


def select_blocks(mass, n_k: int, topk: int, causal: bool = False, n_first: int = 1,
                  n_last: int = 1, seqlens_k=None):
    """Of the blocks a query sees: the first ``n_first``, the last ``n_last`` and the heaviest of
    the rest, ``topk`` in all: int32 [B, H_sel, N_Q, topk], ascending, -1 behind the last.
    Equal masses go to the lower index, NaN ranks below every number."""
    return _ext().select_blocks(mass, n_k, topk, causal, n_first, n_last,
                                _lens_arg(seqlens_k), autograd._check_status)


def sparse_attention(q, k, v, block_idx, scale: Optional[float] = None, causal: bool = False,
                     seqlens_k=None, return_lse: bool = False):
    """Softmax attention of every query over the keys of its listed blocks, differentiable in q,
    k and v: bf16 [B, H, N_Q, d] (and the log-sum-exps fp32 [B, H, N_Q] with ``return_lse``,
    without gradient).

    block_idx int32 [B, H_sel, N_Q, topk]: a set per query (order and repeats do not matter,
    entries outside 0 .. NB-1 select nothing); query head h reads list h // (H // H_sel). A query
    with nothing to read gets 0 (log-sum-exp -inf) and passes no gradient."""
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    out, lse = _ext().sparse_attention(q, k, v, block_idx, _lens_arg(seqlens_k), scale, causal,
                                       return_lse, autograd._check_status)
    return (out, lse) if return_lse else out


def student_sparse_attention(q, k, v, q_s, k_s, topk: int, scale: Optional[float] = None,
                             scale_s: Optional[float] = None, causal: bool = False, lse_s=None,
                             n_first: int = 1, n_last: int = 1, seqlens_k=None):
    """Attention over the blocks that the student map of (q_s, k_s) puts most mass on:
    ``block_mass``, ``select_blocks`` and ``sparse_attention`` in a row.

    The student's K heads are the selection heads: their number and k's have to divide one
    another. Gradients flow to q, k and v only. Returns (out, block_idx)."""
    lens = _lens_arg(seqlens_k)
    mass = block_mass(q_s, k_s, scale_s, causal, lse_s, lens)
    idx = select_blocks(mass, k_s.shape[2], topk, causal, n_first, n_last, lens)
    return sparse_attention(q, k, v, idx, scale, causal, lens), idx
