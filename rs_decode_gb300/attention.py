"""The attention layers between the recurrent ones: a paged cache of keys and
values, and causal attention over it, for the batches that ``Ragged`` plans.

    cache = KVCache(Hq, Hk, D, n_pages, max_pages, page=64, type="e4m3")   # per layer
    ragged.plan(lengths, context)                          # once per batch
    plan = cache.plan(ragged, longest)                     # once per batch, for all layers of this shape
    q, k = qk_norm(q, k, norm="rms", wq=wq, wk=wk, positions=ragged.token_pos, inv_freq=inv_freq)
    cache.write(ragged, k, v, pages)                       # per layer
    y = cache.attend(ragged, q, pages, plan, max_len=longest)

Each call is one call of the binding and only enqueues work on the stream.
"""
from __future__ import annotations

import torch

from . import binding as rb
from .layer import BF16, packed_stride

TYPES = {"bf16": rb.KV_BF16, "e4m3": rb.KV_E4M3}


class KVCache:
    """Owner of one attention layer's cache (see ``rs_kv`` in include/rs.h).

    Hq query heads read Hk key and value heads of D channels; n_pages pages of
    ``page`` tokens.  ``pages``, given to the calls, is int32 [R, max_pages]: the
    page of a request's tokens page * j .. page * j + page - 1, for each j."""

    def __init__(self, Hq: int, Hk: int, D: int, n_pages: int, max_pages: int, page: int = 64, type: str = "bf16",
                 device="cuda"):
        if type not in TYPES:
            raise ValueError(f"unknown cache type {type!r}")
        self.desc = rb.KvDesc(Hq, Hk, D, TYPES[type], page, n_pages, max_pages)
        rb.rs_kv_bytes_for(self.desc)
        self.Hq, self.Hk, self.D, self.max_pages = Hq, Hk, D, max_pages
        self._sizes = (None, None)  # the last plan shape and its bytes
        dev = torch.device(device)
        e4m3 = type == "e4m3"
        shape = (n_pages, Hk, page)
        z = lambda s, dt: torch.zeros(s, dtype=dt, device=dev)
        self.k, self.v = (z((*shape, D), torch.uint8 if e4m3 else torch.bfloat16) for _ in range(2))
        self.k_exp, self.v_exp = (z(shape, torch.uint8) if e4m3 else None for _ in range(2))
        self.status_word = z(1, torch.int32)
        self._dev = self.status_word.get_device()
        self.kv = rb.Kv(*(rb._ptr(t) for t in (self.k, self.v, self.k_exp, self.v_exp)))

    # ------------------------------------------------------------------ checks
    def _on_device(self, names: str, *tensors) -> None:
        dev = self._dev
        for t in tensors:
            if t is not None and (dev < 0 or t.get_device() != dev):
                which = names.split()[next(i for i, x in enumerate(tensors) if x is t)]
                raise ValueError(f"{which} must be on the cache's CUDA device")
        if rb._current_device() != dev:  # the library launches on it
            raise ValueError(f"the cache's CUDA device ({dev}) must be the current one")

    def _pages(self, ragged, pages: torch.Tensor) -> None:
        if pages.dtype is not torch.int32 or pages.shape != (ragged.desc.R, self.max_pages):
            raise ValueError(f"pages must be int32 [{ragged.desc.R}, {self.max_pages}], got {pages.dtype} {tuple(pages.shape)}")

    def _bytes(self, rd, max_len: int) -> rb.AttnBytes:
        key = (rd.R, rd.tokens_cap, max_len)
        sizes = self._sizes  # read once: another thread may put another shape's there
        if sizes[0] != key:
            self._sizes = sizes = (key, rb.rs_attn_bytes_for(self.desc, rd, max_len))
        return sizes[1]

    # ------------------------------------------------------------------ calls
    def write(self, ragged, k: torch.Tensor, v: torch.Tensor, pages: torch.Tensor, stream=None) -> None:
        """The planned rows' keys and values, [rows, Hk, D] bf16 (torch.bfloat16, or int16 bit
        patterns; rows at any stride), to their places in the cache."""
        rd = ragged.desc
        self._on_device("k v pages ragged", k, v, pages, ragged.counts)
        self._pages(ragged, pages)
        T, Hk, D = rd.tokens_cap, self.Hk, self.D
        ld_k, ld_v = packed_stride(k, T, Hk, D, "k"), packed_stride(v, T, Hk, D, "v")
        rb.rs_kv_write(self.desc, self.kv, rd, ragged.arrays, pages, k.data_ptr(), v.data_ptr(), ld_k, ld_v,
                       self.status_word, stream)

    def read(self, ragged, pages: torch.Tensor, out: tuple | None = None, stream=None) -> tuple:
        """The planned rows' keys and values out of the cache again, torch.bfloat16
        [tokens_cap, Hk, D], in ``out`` if given; an e4m3 cache's as code times power of two.
        Without out they are allocated on the current stream, which then has to be the one
        the call runs on; rows that the batch does not fill are then undefined."""
        rd = ragged.desc
        shape = (rd.tokens_cap, self.Hk, self.D)
        if out is None:
            k, v = torch.empty((2, *shape), dtype=torch.bfloat16, device=self.status_word.device).unbind(0)
        else:
            k, v = out
            for t in out:
                if t.dtype not in BF16 or t.shape[1:] != shape[1:] or t.shape[0] < shape[0]:
                    raise ValueError(f"out must be bf16 {list(shape)}, got {t.dtype} {tuple(t.shape)}")
        self._on_device("out[0] out[1] pages ragged", k, v, pages, ragged.counts)
        self._pages(ragged, pages)
        rb.rs_kv_read(self.desc, self.kv, rd, ragged.arrays, pages, k, v, self.status_word, stream)
        return k, v

    def plan(self, ragged, max_len: int, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Shares of a planned batch's attention, in ``out`` if given (an earlier plan of the
        same shape); for all layers with these heads, this type and page tables of this size.  No
        request of the batch may bring more than max_len rows."""
        n = self._bytes(ragged.desc, max_len).plan
        if out is None:
            out = torch.empty(n, dtype=torch.uint8, device=self.status_word.device)
        self._on_device("out ragged", out, ragged.counts)
        if out.nbytes < n:
            raise ValueError("out is smaller than a plan of this batch")
        rb.rs_attn_plan(self.desc, ragged.desc, ragged.arrays, max_len, out, self.status_word, stream)
        return out

    def workspace(self, ragged, max_len: int) -> torch.Tensor:
        """Scratch of ``attend`` for this plan shape; may serve many calls, one after another."""
        return torch.empty(self._bytes(ragged.desc, max_len).work, dtype=torch.uint8, device=self.status_word.device)

    def attend(self, ragged, q: torch.Tensor, pages: torch.Tensor, plan: torch.Tensor, *, max_len: int,
               scale: float | None = None, y: torch.Tensor | None = None, work: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
        """Causal attention of the planned rows, q [rows, Hq, D] bf16 (rows at any stride), over
        their requests' cached keys, the batch's own among them (``write`` comes first).  scale
        is D ** -0.5 unless given.  Returns y torch.bfloat16 [rows, Hq, D].  Without y and work
        they are allocated on the current stream, which then has to be the one the call runs on;
        rows that the batch does not fill are then undefined.  The batch is the plan's: after
        another ``ragged.plan`` it has to be made anew."""
        rd = ragged.desc
        T, Hq, D = rd.tokens_cap, self.Hq, self.D
        self._on_device("q pages plan ragged y work", q, pages, plan, ragged.counts, y, work)
        self._pages(ragged, pages)
        ld_q = packed_stride(q, T, Hq, D, "q")
        sizes = self._bytes(rd, max_len)
        if plan.nbytes < sizes.plan:
            raise ValueError("plan is smaller than plan() of this batch")
        if y is None:
            y = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=self.status_word.device)
        elif y.dtype not in BF16 or y.shape[1:] != (Hq, D) or y.shape[0] < T:
            raise ValueError(f"y must be bf16 [{T}, {Hq}, {D}], got {y.dtype} {tuple(y.shape)}")
        if work is None:
            work = self.workspace(ragged, max_len)
        elif work.nbytes < sizes.work:
            raise ValueError("work is smaller than workspace() of this batch")
        attn = rb.Attn(q.data_ptr(), ld_q, rb._ptr(pages), D ** -0.5 if scale is None else scale, max_len)
        rb.rs_attend(self.desc, self.kv, rd, ragged.arrays, attn, plan, y, work, self.status_word, stream)
        return y

    def status(self, clear: bool = True) -> int:
        """RS_DEV_* bits that the calls set; synchronises."""
        bits = int(self.status_word.item()) & 0xffffffff
        if clear:
            self.status_word.zero_()
        return bits
