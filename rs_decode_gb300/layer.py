"""Convenience owner of one layer's librs state, allocated as torch tensors.

The library allocates nothing; this class sizes every state array with
``rs_state_bytes_for`` and keeps the tensors alive.  Each method is one call
of the binding (which is one C entry point).  bf16 arrays are carried as int16
tensors holding the raw bit patterns.
"""
from __future__ import annotations

import numpy as np
import torch

from . import binding as rb


def to_device(d: dict, device="cuda", non_blocking: bool = False) -> dict:
    """numpy inputs (uint16 = bf16 bits, float32, int32) -> device tensors."""
    out = {}
    for k, v in d.items():
        a = np.ascontiguousarray(v)
        if a.dtype == np.uint16:
            a = a.view(np.int16)
        out[k] = torch.from_numpy(a).to(device, non_blocking=non_blocking)
    return out


BF16 = (torch.bfloat16, torch.int16)  # values, or their bit patterns


def packed_stride(t: torch.Tensor, rows: int, heads: int, d: int, name: str) -> int:
    """Row stride in elements of a packed [rows, heads, d] bf16 tensor whose heads lie side by side."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != d or shape[0] < rows or t.dtype not in BF16:
        raise ValueError(f"{name} must be bf16 [{rows}, {heads}, {d}], got {t.dtype} {tuple(shape)}")
    ld, head, one = t.stride()
    if one != 1 or (head != d and heads > 1):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    return ld if shape[0] > 1 else heads * d


class Layer:
    def __init__(self, kind: str, B: int, H: int, G: int, P: int, N: int, L: int, T_max: int = 0,
                 capacity: int | None = None, precision: int = rb.PREC_FP32, device="cuda"):
        if kind not in ("mamba2", "gdn", "kda"):
            raise ValueError(f"librs has no kernels for layer kind {kind!r}")
        self.kind = kind
        k = {"mamba2": rb.MAMBA2, "gdn": rb.GDN, "kda": rb.KDA}[kind]
        self.desc = rb.make_desc(k, B, H, G, P, N, L, T_max, capacity, precision)
        sz = rb.rs_state_bytes_for(self.desc)
        self.B, self.H, self.G, self.P, self.N, self.L, self.T_max = B, H, G, P, N, L, T_max
        self.cap = self.desc.capacity
        self._prefill_size = (None, 0)  # the last plan shape and its workspace bytes
        dev = torch.device(device)
        z = lambda n, dt: torch.zeros(n, dtype=dt, device=dev) if n else None
        self.ckpt_hp = z(sz.ckpt_hp // 4, torch.float32)
        self.ckpt_lp = z(sz.ckpt_lp // 2, torch.int16)
        self.buf_v = z(sz.buf_v, torch.uint8)
        self.buf_k = z(sz.buf_k // 2, torch.int16)
        self.buf_a = z(sz.buf_a // 4, torch.float32)
        self.buf_s = z(sz.buf_s // 4, torch.float32)
        self.base = z(B, torch.int32)
        self.h = z(B, torch.int32)
        self.nd = z(B, torch.int32)
        self.arrive = z(sz.arrive // 4, torch.int32)
        self.status_word = z(1, torch.int32)
        p = lambda t: t.data_ptr() if t is not None else None
        self.state = rb.State(p(self.ckpt_hp), p(self.ckpt_lp), p(self.buf_v), p(self.buf_k), p(self.buf_a),
                              p(self.buf_s), p(self.base), p(self.h), p(self.nd), p(self.arrive),
                              p(self.status_word))
        self.shape = (B, H, N, P)

    # ------------------------------------------------------------------ calls
    def init(self, S0: torch.Tensor | None = None, stream=None):
        """S0: fp32 [B, H, N, P] device tensor (key-major slabs) or None for zeros."""
        rb.rs_init(self.desc, self.state, S0, stream)

    def decode(self, d: dict, params: dict, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        if y is None:
            y = torch.empty(self.B, self.H, self.P, dtype=torch.float32, device=self.base.device)
        if self.kind == "mamba2":
            rb.rs_decode_mamba2(self.desc, self.state, d["x"], d["dt"], params["A"], d["Bm"], d["Cm"],
                                params.get("D"), y, stream)
        else:
            fn = rb.rs_decode_gdn if self.kind == "gdn" else rb.rs_decode_kda
            fn(self.desc, self.state, d["q"], d["k"], d["v"], d["alpha"], d["beta"], y, stream)
        return y

    def inputs(self, d: dict, params: dict) -> rb.Inputs:
        if self.kind == "mamba2":
            return rb.make_inputs(x=d["x"], dt=d["dt"], A=params["A"], Bm=d["Bm"], Cm=d.get("Cm"),
                                  D=params.get("D"))
        return rb.make_inputs(q=d["q"], k=d["k"], v=d["v"], alpha=d["alpha"], beta=d["beta"])

    def verify(self, T: int, d: dict, params: dict, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        if y is None:
            y = torch.empty(self.B, T, self.H, self.P, dtype=torch.float32, device=self.base.device)
        rb.rs_verify(self.desc, self.state, T, self.inputs(d, params), y, stream)
        return y

    def commit(self, accepted: torch.Tensor, stream=None):
        rb.rs_commit(self.desc, self.state, accepted, stream)

    def rollback(self, stream=None):
        rb.rs_rollback(self.desc, self.state, stream)

    def append(self, n: int, d: dict, params: dict, stream=None):
        rb.rs_append(self.desc, self.state, n, self.inputs(d, params), stream)

    def flush(self, stream=None):
        rb.rs_flush(self.desc, self.state, stream)

    def materialize(self, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        if out is None:
            out = torch.empty(self.shape, dtype=torch.float32, device=self.base.device)
        rb.rs_materialize(self.desc, self.state, out, stream)
        return out

    # ---------------------------------------------------------------- prefill
    def _prefill_bytes(self, rd, max_len: int) -> int:
        key = (rd.R, rd.tokens_cap, rd.block, rd.max_blocks, rd.n_free, max_len)
        if self._prefill_size[0] != key:
            self._prefill_size = (key, rb.rs_prefill_bytes_for(self.desc, rd, max_len))
        return self._prefill_size[1]

    def prefill_workspace(self, ragged, max_len: int) -> torch.Tensor | None:
        """Scratch of ``prefill`` for this plan shape; may serve many calls, one after another."""
        n = self._prefill_bytes(ragged.desc, max_len)
        return torch.empty(n, dtype=torch.uint8, device=self.base.device) if n else None

    def prefill(self, ragged, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, alpha: torch.Tensor,
                beta: torch.Tensor, *, max_len: int, rows: torch.Tensor | None = None,
                start: torch.Tensor | None = None, pool: torch.Tensor | None = None, y: torch.Tensor | None = None,
                work: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """The gated delta rule over a planned batch (``prefill.Ragged``), into this layer's state.

        q, k [rows, G, N], v [rows, H, P] bf16 (torch.bfloat16, or int16 bit
        patterns), each head contiguous, rows at any stride; alpha, beta fp32
        [rows, H].  rows, start: int32 [R] (see include/rs.h); pool
        [n, H, N, P], fp32 or, for a shared-bf16 layer, bf16.  Returns y
        torch.bfloat16 [rows, H, P].  Without y and work they are allocated
        on the current stream, which then has to be the one the call runs on."""
        rd = ragged.desc
        T, R, H, G, N, P = rd.tokens_cap, rd.R, self.H, self.G, self.N, self.P
        dev = self.base.get_device()
        for t, name in ((q, "q"), (k, "k"), (v, "v"), (alpha, "alpha"), (beta, "beta"), (rows, "rows"), (start, "start"),
                        (pool, "pool"), (y, "y"), (work, "work"), (ragged.counts, "the plan")):
            if t is not None and (dev < 0 or t.get_device() != dev):
                raise ValueError(f"{name} must be on the layer's CUDA device")
        ld_q, ld_k, ld_v = packed_stride(q, T, G, N, "q"), packed_stride(k, T, G, N, "k"), packed_stride(v, T, H, P, "v")
        for t, name in ((alpha, "alpha"), (beta, "beta")):
            shape = t.shape
            if t.dtype is not torch.float32 or len(shape) != 2 or shape[0] < T or shape[1] != H:
                raise ValueError(f"{name} must be float32 [{T}, {H}], got {t.dtype} {tuple(t.shape)}")
        for t, name in ((rows, "rows"), (start, "start")):
            if t is not None and (t.dtype is not torch.int32 or t.shape != (R,)):
                raise ValueError(f"{name} must be int32 [{R}]")
        n_pool = 0
        if pool is not None:
            types = BF16 if self.desc.precision & 0xf == rb.PREC_SHARED_BF16 else (torch.float32,)
            n_pool = pool.size(0)
            if pool.shape != (n_pool, H, N, P) or pool.dtype not in types:
                raise ValueError(f"pool must be {types[0]} [n, {H}, {N}, {P}], got {pool.dtype} {tuple(pool.shape)}")
        if y is None:
            y = torch.empty((T, H, P), dtype=torch.bfloat16, device=self.base.device)
        elif y.dtype not in BF16 or y.shape[1:] != (H, P) or y.shape[0] < T:
            raise ValueError(f"y must be bf16 [{T}, {H}, {P}], got {y.dtype} {tuple(y.shape)}")
        if work is None:
            work = self.prefill_workspace(ragged, max_len)
        elif work.nbytes < self._prefill_bytes(rd, max_len):
            raise ValueError("work is smaller than prefill_workspace() of this plan")
        p = rb._ptr
        args = rb.Prefill(q.data_ptr(), k.data_ptr(), v.data_ptr(), p(alpha), p(beta), ld_q, ld_k, ld_v, p(rows), p(start),
                          p(pool), n_pool, max_len)
        rb.rs_prefill_gdn(self.desc, self.state, rd, ragged.arrays, args, y, work, stream)
        return y

    def status(self, clear: bool = True, stream=None) -> int:
        return rb.rs_get_status(self.state, clear, stream)

    def pointers(self) -> dict:
        return {"base": self.base.cpu().numpy(), "h": self.h.cpu().numpy(), "nd": self.nd.cpu().numpy()}

    def checkpoint_hp(self) -> torch.Tensor | None:
        return None if self.ckpt_hp is None else self.ckpt_hp.view(self.shape)

    def checkpoint_lp_f32(self) -> torch.Tensor | None:
        if self.ckpt_lp is None:
            return None
        return (self.ckpt_lp.to(torch.int32) << 16).view(torch.float32).view(self.shape)
