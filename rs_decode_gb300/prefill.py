"""What goes ahead of ``Layer.prefill``: the plan of a ragged batch and the
norms of its query and key heads.

    ragged = Ragged(R, tokens_cap, block=512, max_blocks=64, n_free=free.numel())
    ragged.plan(lengths, context, free)                       # once per batch
    q, k = qk_norm(q, k, norm="l2", scale_q=N ** -0.5)        # per layer
    y = layer.prefill(ragged, q, k, v, alpha, beta, max_len=longest, start=start, pool=pool)

Each call is one call of the binding and only enqueues work on the stream.
"""
from __future__ import annotations

import torch

from . import binding as rb
from .layer import BF16, packed_stride

NORMS = {"none": rb.NORM_NONE, "l2": rb.NORM_L2, "rms": rb.NORM_RMS}


class Ragged:
    """Owner of one batch plan's device arrays (see ``rs_ragged`` in include/rs.h)."""

    def __init__(self, R: int, tokens_cap: int, block: int = 0, max_blocks: int = 0, n_free: int = 0, device="cuda"):
        self.desc = rb.RaggedDesc(R, tokens_cap, block, max_blocks, n_free)
        sz = rb.rs_ragged_bytes_for(self.desc)
        dev = torch.device(device)
        z = lambda n: torch.zeros(n // 4, dtype=torch.int32, device=dev)
        self.cu_tokens, self.cu_chunks, self.cu_blocks = z(sz.cu_tokens), z(sz.cu_chunks), z(sz.cu_blocks)
        self.token_req, self.token_pos = z(sz.token_req), z(sz.token_pos)
        self.chunks = z(sz.chunks).view(-1, 4)
        self.block_table = torch.full((R, max_blocks), -1, dtype=torch.int32, device=dev) if block else None
        self.counts = z(sz.counts)
        self.status_word = torch.zeros(1, dtype=torch.int32, device=dev)
        self.arrays = rb.RaggedArrays(*(rb._ptr(getattr(self, n)) for n in rb._RAGGED))

    def plan(self, lengths: torch.Tensor, context: torch.Tensor | None = None,
             free_blocks: torch.Tensor | None = None, stream=None) -> None:
        """lengths, context: int32 [R]; free_blocks: int32, at least n_free slots."""
        d, dev = self.desc, self.counts.get_device()
        for t, name in ((lengths, "lengths"), (context, "context")):
            if t is not None and (t.dtype is not torch.int32 or t.numel() != d.R or t.get_device() != dev or dev < 0):
                raise ValueError(f"{name} must be int32 [{d.R}] on the plan's CUDA device")
        if d.block and d.n_free and (free_blocks is None or free_blocks.dtype is not torch.int32
                                     or free_blocks.numel() < d.n_free or free_blocks.get_device() != dev):
            raise ValueError(f"free_blocks must be int32 [{d.n_free}] on the plan's CUDA device")
        rb.rs_ragged_plan(d, lengths, context, free_blocks, self.arrays, self.status_word, stream)

    def status(self, clear: bool = True) -> int:
        """RS_DEV_* bits that plan() set; synchronises."""
        bits = int(self.status_word.item()) & 0xffffffff
        if clear:
            self.status_word.zero_()
        return bits


def _empty(like: torch.Tensor, shape: tuple) -> torch.Tensor:
    if like.dtype is torch.bfloat16:
        return torch.empty_like(like)  # contiguous: like's heads lie side by side
    return torch.empty(shape, dtype=torch.bfloat16, device=like.device)


def qk_norm(q: torch.Tensor | None, k: torch.Tensor | None, *, norm: str = "l2", eps: float = 1e-6,
            wq: torch.Tensor | None = None, wk: torch.Tensor | None = None, weight_offset: float = 0.0,
            scale_q: float = 1.0, scale_k: float = 1.0, positions: torch.Tensor | None = None,
            inv_freq: torch.Tensor | None = None, interleaved: bool = False,
            out: tuple | None = None, stream=None) -> tuple:
    """Norms every head of q [T, Hq, D] and k [T, Hk, D] (bf16, rows at any
    stride; either may be None) and rotates its first 2 * len(inv_freq)
    channels by positions (int32 [T]) * inv_freq (float32).  Returns the two
    results, torch.bfloat16, in ``out`` if given (in place: out=(q, k)).
    Without out they are allocated on the current stream, which then has to be
    the one the call runs on.

    Delta-rule layers norm by x / sqrt(sum(x^2) + e): norm="rms" with
    eps=e / D and scales of D ** -0.5 (times the query's own)."""
    kind = NORMS.get(norm)
    if kind is None:
        raise ValueError(f"unknown norm {norm!r}")
    one = q if q is not None else k
    shape = one.shape if one is not None else ()
    dev = one.get_device() if one is not None else -1
    if len(shape) != 3 or dev < 0:
        raise ValueError("q or k must be a CUDA [T, heads, D] tensor")
    T, _, D = shape
    qo, ko = out if out is not None else (None, None)
    for t in (k, wq, wk, positions, inv_freq, qo, ko):
        if t is not None and t.get_device() != dev:
            raise ValueError(f"all tensors must be on one CUDA device, got {t.device} beside {one.device}")
    rot = 0
    if inv_freq is not None:
        if positions is None:
            raise ValueError("positions and inv_freq go together")
        rot = 2 * inv_freq.numel()
        if inv_freq.dtype is not torch.float32 or positions.dtype is not torch.int32 or positions.numel() != T:
            raise ValueError(f"inv_freq must be float32 and positions int32 [{T}]")
    elif positions is not None:
        raise ValueError("positions and inv_freq go together")
    for w in (wq, wk):
        if w is not None and (w.dtype not in BF16 or w.numel() != D):
            raise ValueError(f"weights must be bf16 [{D}], got {w.dtype} {tuple(w.shape)}")
    Hq = Hk = ld_q = ld_k = ld_qo = ld_ko = 0
    pq = pk = pqo = pko = None
    if q is not None:
        Hq = shape[1]
        ld_q = packed_stride(q, T, Hq, D, "q")
        if qo is None:
            qo = _empty(q, (T, Hq, D))
            ld_qo = Hq * D
        else:
            ld_qo = packed_stride(qo, T, Hq, D, "out[0]")
        pq, pqo = q.data_ptr(), qo.data_ptr()
    if k is not None:
        Hk = k.shape[1]
        ld_k = packed_stride(k, T, Hk, D, "k")
        if ko is None:
            ko = _empty(k, (T, Hk, D))
            ld_ko = Hk * D
        else:
            ld_ko = packed_stride(ko, T, Hk, D, "out[1]")
        pk, pko = k.data_ptr(), ko.data_ptr()
    d = rb.QkDesc(T, Hq, Hk, D, kind, rot, interleaved, eps, weight_offset, scale_q, scale_k, ld_q, ld_k, ld_qo, ld_ko)
    rb.rs_qk_norm(d, pq, pk, wq, wk, inv_freq, positions, pqo, pko, stream)
    return qo, ko
