"""Thin ctypes binding of librs (include/rs.h).

Argument marshalling only: every function here turns torch tensors into raw
pointers, passes the current CUDA stream, calls the C entry point of the same
name, and raises ``RsError`` on a non-zero status.  All arithmetic runs in the
library's CUDA kernels; there is no fallback of any kind, and loading fails
loudly when librs.so has not been built.
"""
from __future__ import annotations

import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "librs.so")

MAMBA2, GDN, KDA = 0, 1, 2
PREC_FP32, PREC_TWO, PREC_SHARED_BF16 = 0, 1, 2
U_BF16 = 0x10  # flag: GDN records keep u in bf16
DEV_CAPACITY, DEV_ACCEPT, DEV_DRAFTS_PENDING = 0x1, 0x2, 0x4
DEV_TIMEOUT, DEV_LENGTH, DEV_BLOCKS, DEV_RECORDS, DEV_SLOT, DEV_GATE = 0x8, 0x10, 0x20, 0x40, 0x80, 0x100
NORM_NONE, NORM_L2, NORM_RMS = 0, 1, 2
CHUNK = 64  # rows of a chunk of the ragged prefill
KV_BF16, KV_E4M3 = 0, 1
STATUS = {0: "RS_OK", 1: "RS_ERR_INVALID_ARG", 2: "RS_ERR_UNSUPPORTED", 3: "RS_ERR_CAPACITY",
          4: "RS_ERR_CUDA", 5: "RS_ERR_DEVICE", 6: "RS_ERR_STATIC_LIMIT"}
STATIC_MAX_SEQS = 4096

_c_i32 = ctypes.c_int32
_vp = ctypes.c_void_p


class LayerDesc(ctypes.Structure):
    _fields_ = [(n, _c_i32) for n in ("kind", "B", "H", "G", "P", "N", "L", "T_max", "capacity",
                                       "precision")]


class State(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("ckpt_hp", "ckpt_lp", "buf_v", "buf_k", "buf_a", "buf_s", "base",
                                    "h", "nd", "arrive", "status")]


class StateBytes(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("ckpt_hp", "ckpt_lp", "buf_v", "buf_k", "buf_a",
                                                "buf_s", "base", "h", "nd", "arrive", "status")]


class Inputs(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("x", "dt", "A", "Bm", "Cm", "D", "q", "k", "v", "alpha", "beta")]


class RaggedDesc(ctypes.Structure):
    _fields_ = [(n, _c_i32) for n in ("R", "tokens_cap", "block", "max_blocks", "n_free")]


_RAGGED = ("cu_tokens", "cu_chunks", "cu_blocks", "token_req", "token_pos", "chunks", "block_table", "counts")


class RaggedArrays(ctypes.Structure):
    _fields_ = [(n, _vp) for n in _RAGGED]


class RaggedBytes(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in _RAGGED]


class QkDesc(ctypes.Structure):
    _fields_ = [(n, _c_i32) for n in ("T", "Hq", "Hk", "D", "norm", "rot", "interleaved")] + \
               [(n, ctypes.c_float) for n in ("eps", "weight_offset", "scale_q", "scale_k")] + \
               [(n, ctypes.c_int64) for n in ("ld_q", "ld_k", "ld_qo", "ld_ko")]


class Prefill(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("q", "k", "v", "alpha", "beta")] + \
               [(n, ctypes.c_int64) for n in ("ld_q", "ld_k", "ld_v")] + \
               [(n, _vp) for n in ("rows", "start", "pool")] + [("n_pool", _c_i32), ("max_len", _c_i32)]


class KvDesc(ctypes.Structure):
    _fields_ = [(n, _c_i32) for n in ("Hq", "Hk", "D", "type", "page", "n_pages", "max_pages")]


class Kv(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("k", "v", "ks", "vs")]


class KvBytes(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("k", "v", "ks", "vs")]


class AttnBytes(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("plan", "work")]


class Attn(ctypes.Structure):
    _fields_ = [("q", _vp), ("ld_q", ctypes.c_int64), ("pages", _vp), ("scale", ctypes.c_float), ("max_len", _c_i32)]


# name -> argtypes (restype is rs_status = int unless listed in _RESTYPE)
_SIGS = {
    "rs_status_string": [ctypes.c_int],
    "rs_version": [],
    "rs_last_cuda_error": [],
    "rs_state_bytes_for": [ctypes.POINTER(LayerDesc), ctypes.POINTER(StateBytes)],
    "rs_init": [ctypes.POINTER(LayerDesc), ctypes.POINTER(State), _vp, _vp],
    "rs_get_status": [ctypes.POINTER(State), ctypes.POINTER(ctypes.c_uint32), ctypes.c_int, _vp],
    "rs_decode_mamba2": [ctypes.POINTER(LayerDesc), ctypes.POINTER(State)] + [_vp] * 8,
    "rs_decode_gdn": [ctypes.POINTER(LayerDesc), ctypes.POINTER(State)] + [_vp] * 7,
    "rs_decode_kda": [ctypes.POINTER(LayerDesc), ctypes.POINTER(State)] + [_vp] * 7,
    "rs_verify": [ctypes.POINTER(LayerDesc), ctypes.POINTER(State), ctypes.c_int,
                  ctypes.POINTER(Inputs), _vp, _vp],
    "rs_commit": [ctypes.POINTER(LayerDesc), ctypes.POINTER(State), _vp, _vp],
    "rs_rollback": [ctypes.POINTER(LayerDesc), ctypes.POINTER(State), _vp],
    "rs_append": [ctypes.POINTER(LayerDesc), ctypes.POINTER(State), ctypes.c_int,
                  ctypes.POINTER(Inputs), _vp],
    "rs_flush": [ctypes.POINTER(LayerDesc), ctypes.POINTER(State), _vp],
    "rs_materialize": [ctypes.POINTER(LayerDesc), ctypes.POINTER(State), _vp, _vp],
    "rs_eager_step_mamba2": [ctypes.POINTER(LayerDesc)] + [_vp] * 9,
    "rs_eager_step_gdn": [ctypes.POINTER(LayerDesc)] + [_vp] * 8,
    "rs_eager_step_kda": [ctypes.POINTER(LayerDesc)] + [_vp] * 8,
    "rs_eager_verify_snapshots": [ctypes.POINTER(LayerDesc), _vp, _vp, ctypes.c_int,
                                  ctypes.POINTER(Inputs), _vp, _vp],
    "rs_eager_select": [ctypes.POINTER(LayerDesc), _vp, _vp, _vp, _vp],
    "rs_ragged_bytes_for": [ctypes.POINTER(RaggedDesc), ctypes.POINTER(RaggedBytes)],
    "rs_ragged_plan": [ctypes.POINTER(RaggedDesc), _vp, _vp, _vp, ctypes.POINTER(RaggedArrays), _vp, _vp],
    "rs_qk_norm": [ctypes.POINTER(QkDesc)] + [_vp] * 9,
    "rs_prefill_bytes_for": [ctypes.POINTER(LayerDesc), ctypes.POINTER(RaggedDesc), _c_i32,
                             ctypes.POINTER(ctypes.c_size_t)],
    "rs_prefill_gdn": [ctypes.POINTER(LayerDesc), ctypes.POINTER(State), ctypes.POINTER(RaggedDesc),
                       ctypes.POINTER(RaggedArrays), ctypes.POINTER(Prefill), _vp, _vp, _vp],
    "rs_kv_bytes_for": [ctypes.POINTER(KvDesc), ctypes.POINTER(KvBytes)],
    "rs_kv_write": [ctypes.POINTER(KvDesc), ctypes.POINTER(Kv), ctypes.POINTER(RaggedDesc), ctypes.POINTER(RaggedArrays),
                    _vp, _vp, _vp, ctypes.c_int64, ctypes.c_int64, _vp, _vp],
    "rs_kv_read": [ctypes.POINTER(KvDesc), ctypes.POINTER(Kv), ctypes.POINTER(RaggedDesc), ctypes.POINTER(RaggedArrays)] +
                  [_vp] * 5,
    "rs_attn_bytes_for": [ctypes.POINTER(KvDesc), ctypes.POINTER(RaggedDesc), _c_i32, ctypes.POINTER(AttnBytes)],
    "rs_attn_plan": [ctypes.POINTER(KvDesc), ctypes.POINTER(RaggedDesc), ctypes.POINTER(RaggedArrays), _c_i32, _vp, _vp, _vp],
    "rs_attend": [ctypes.POINTER(KvDesc), ctypes.POINTER(Kv), ctypes.POINTER(RaggedDesc), ctypes.POINTER(RaggedArrays),
                  ctypes.POINTER(Attn)] + [_vp] * 5,
    "rs_decode_mamba2_noalloc": [ctypes.POINTER(LayerDesc), ctypes.POINTER(State)] + [_vp] * 8,
}
_RESTYPE = {"rs_status_string": ctypes.c_char_p, "rs_version": ctypes.c_char_p,
            "rs_last_cuda_error": ctypes.c_char_p}

_lib = None


class RsError(RuntimeError):
    def __init__(self, fn: str, status: int, bits: int | None = None):
        self.status = status
        self.bits = bits
        extra = f" (device bits 0x{bits:x})" if bits is not None else ""
        super().__init__(f"{fn} returned {STATUS.get(status, status)}{extra}")


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load librs.so (no GPU needed).  Raises if the library was not built."""
    global _lib
    if _lib is None or path != LIB_PATH:
        if not os.path.exists(path):
            raise RuntimeError(f"librs.so not found at {path}: run rs_decode_gb300.build.build() "
                               "(or __graft_entry__.build()) first")
        lib = ctypes.CDLL(path)
        for name, args in _SIGS.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = _RESTYPE.get(name, ctypes.c_int)
        if path != LIB_PATH:
            return lib
        _lib = lib
    return _lib


# The current stream's handle without a Stream object around it: a decode step's
# calls are short enough for that to count.
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)
if _current_stream is None or _current_device is None:
    _current_device = torch.cuda.current_device

    def _current_stream(device: int) -> int:
        return torch.cuda.current_stream(device).cuda_stream


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensors passed to librs must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return _current_stream(_current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _check(fn: str, status: int) -> None:
    if status != 0:
        err = RsError(fn, status)
        if status == 4:  # RS_ERR_CUDA: say which CUDA error
            err.args = (f"{err.args[0]}: {load().rs_last_cuda_error().decode()}",)
        raise err


def make_desc(kind: int, B: int, H: int, G: int, P: int, N: int, L: int, T_max: int = 0,
              capacity: int | None = None, precision: int = PREC_FP32) -> LayerDesc:
    return LayerDesc(kind, B, H, G, P, N, L, T_max, capacity if capacity else max(L, T_max) + T_max, precision)


# Precision names of the synthetic workloads: the checkpoint's, and "+u16"
# for GDN records that keep u in bf16.
PRECISIONS = {"fp32": PREC_FP32, "two": PREC_TWO, "shared_bf16": PREC_SHARED_BF16,
              "fp32+u16": PREC_FP32 | U_BF16, "two+u16": PREC_TWO | U_BF16}


def make_inputs(**tensors) -> Inputs:
    return Inputs(**{k: _ptr(v) for k, v in tensors.items() if v is not None})


# ----------------------------------------------------------------------------- entry points
def rs_version() -> str:
    return load().rs_version().decode()


def rs_status_string(status: int) -> str:
    return load().rs_status_string(status).decode()


def rs_state_bytes_for(desc: LayerDesc) -> StateBytes:
    out = StateBytes()
    _check("rs_state_bytes_for", load().rs_state_bytes_for(ctypes.byref(desc), ctypes.byref(out)))
    return out


def rs_init(desc, state, init=None, stream=None):
    _check("rs_init", load().rs_init(ctypes.byref(desc), ctypes.byref(state), _ptr(init), _stream(stream)))


def rs_get_status(state, clear: bool = True, stream=None) -> int:
    bits = ctypes.c_uint32(0)
    st = load().rs_get_status(ctypes.byref(state), ctypes.byref(bits), int(clear), _stream(stream))
    if st not in (0, 5):
        raise RsError("rs_get_status", st)
    return bits.value


def rs_decode_mamba2(desc, state, x, dt, A, Bm, Cm, D, y, stream=None):
    _check("rs_decode_mamba2", load().rs_decode_mamba2(
        ctypes.byref(desc), ctypes.byref(state), _ptr(x), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm),
        _ptr(D), _ptr(y), _stream(stream)))


def rs_decode_gdn(desc, state, q, k, v, alpha, beta, y, stream=None):
    _check("rs_decode_gdn", load().rs_decode_gdn(
        ctypes.byref(desc), ctypes.byref(state), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
        _ptr(y), _stream(stream)))


def rs_decode_kda(desc, state, q, k, v, alpha, beta, y, stream=None):
    _check("rs_decode_kda", load().rs_decode_kda(
        ctypes.byref(desc), ctypes.byref(state), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
        _ptr(y), _stream(stream)))


def rs_verify(desc, state, T: int, inputs: Inputs, y, stream=None):
    _check("rs_verify", load().rs_verify(ctypes.byref(desc), ctypes.byref(state), T,
                                         ctypes.byref(inputs), _ptr(y), _stream(stream)))


def rs_commit(desc, state, accepted, stream=None):
    _check("rs_commit", load().rs_commit(ctypes.byref(desc), ctypes.byref(state), _ptr(accepted),
                                         _stream(stream)))


def rs_rollback(desc, state, stream=None):
    _check("rs_rollback", load().rs_rollback(ctypes.byref(desc), ctypes.byref(state), _stream(stream)))


def rs_append(desc, state, n: int, inputs: Inputs, stream=None):
    _check("rs_append", load().rs_append(ctypes.byref(desc), ctypes.byref(state), n,
                                         ctypes.byref(inputs), _stream(stream)))


def rs_flush(desc, state, stream=None):
    _check("rs_flush", load().rs_flush(ctypes.byref(desc), ctypes.byref(state), _stream(stream)))


def rs_materialize(desc, state, out, stream=None):
    _check("rs_materialize", load().rs_materialize(ctypes.byref(desc), ctypes.byref(state), _ptr(out),
                                                   _stream(stream)))


def rs_eager_step_mamba2(desc, S, x, dt, A, Bm, Cm, D, y, stream=None):
    _check("rs_eager_step_mamba2", load().rs_eager_step_mamba2(
        ctypes.byref(desc), _ptr(S), _ptr(x), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(D), _ptr(y),
        _stream(stream)))


def rs_eager_step_gdn(desc, S, q, k, v, alpha, beta, y, stream=None):
    _check("rs_eager_step_gdn", load().rs_eager_step_gdn(
        ctypes.byref(desc), _ptr(S), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(y),
        _stream(stream)))


def rs_eager_step_kda(desc, S, q, k, v, alpha, beta, y, stream=None):
    _check("rs_eager_step_kda", load().rs_eager_step_kda(
        ctypes.byref(desc), _ptr(S), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(y),
        _stream(stream)))


def rs_eager_verify_snapshots(desc, pool, cur, T: int, inputs: Inputs, y, stream=None):
    _check("rs_eager_verify_snapshots", load().rs_eager_verify_snapshots(
        ctypes.byref(desc), _ptr(pool), _ptr(cur), T, ctypes.byref(inputs), _ptr(y), _stream(stream)))


def rs_eager_select(desc, cur, accepted, status=None, stream=None):
    _check("rs_eager_select", load().rs_eager_select(ctypes.byref(desc), _ptr(cur), _ptr(accepted),
                                                     _ptr(status), _stream(stream)))


def rs_decode_mamba2_noalloc(desc, state, x, dt, A, Bm, Cm, D, y, stream=None):
    """rs_decode_mamba2 with the arrival counters in the library's static
    device array (state.arrive is ignored); for callers that cannot allocate."""
    _check("rs_decode_mamba2_noalloc", load().rs_decode_mamba2_noalloc(
        ctypes.byref(desc), ctypes.byref(state), _ptr(x), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm),
        _ptr(D), _ptr(y), _stream(stream)))


# ----------------------------------------------------------------------------- ragged prefill
def rs_ragged_bytes_for(rd: RaggedDesc) -> RaggedBytes:
    out = RaggedBytes()
    _check("rs_ragged_bytes_for", load().rs_ragged_bytes_for(ctypes.byref(rd), ctypes.byref(out)))
    return out


def rs_ragged_plan(rd, lengths, context, free_blocks, arrays, status, stream=None):
    st = load().rs_ragged_plan(rd, _ptr(lengths), _ptr(context), _ptr(free_blocks), arrays, _ptr(status), _stream(stream))
    if st:
        _check("rs_ragged_plan", st)


def rs_qk_norm(desc, q, k, wq, wk, inv_freq, positions, q_out, k_out, stream=None):
    """q, k, q_out, k_out are data pointers (their row strides are in desc)."""
    st = load().rs_qk_norm(desc, q, k, _ptr(wq), _ptr(wk), _ptr(inv_freq), _ptr(positions), q_out, k_out, _stream(stream))
    if st:
        _check("rs_qk_norm", st)


def rs_prefill_bytes_for(desc, rd, max_len: int) -> int:
    out = ctypes.c_size_t(0)
    _check("rs_prefill_bytes_for", load().rs_prefill_bytes_for(ctypes.byref(desc), ctypes.byref(rd), max_len,
                                                               ctypes.byref(out)))
    return out.value


def rs_prefill_gdn(desc, state, rd, arrays, prefill, y, work, stream=None):
    st = load().rs_prefill_gdn(desc, state, rd, arrays, prefill, _ptr(y), _ptr(work), _stream(stream))
    if st:
        _check("rs_prefill_gdn", st)


# ----------------------------------------------------------------------------- attention over a paged cache
def rs_kv_bytes_for(desc: KvDesc) -> KvBytes:
    out = KvBytes()
    _check("rs_kv_bytes_for", load().rs_kv_bytes_for(ctypes.byref(desc), ctypes.byref(out)))
    return out


def rs_kv_write(desc, kv, rd, rg, pages, k, v, ld_k, ld_v, status, stream=None):
    """k, v are data pointers (their row strides are ld_k, ld_v)."""
    st = load().rs_kv_write(desc, kv, rd, rg, _ptr(pages), k, v, ld_k, ld_v, _ptr(status), _stream(stream))
    if st:
        _check("rs_kv_write", st)


def rs_kv_read(desc, kv, rd, rg, pages, k, v, status, stream=None):
    st = load().rs_kv_read(desc, kv, rd, rg, _ptr(pages), _ptr(k), _ptr(v), _ptr(status), _stream(stream))
    if st:
        _check("rs_kv_read", st)


def rs_attn_bytes_for(desc, rd, max_len: int) -> AttnBytes:
    out = AttnBytes()
    _check("rs_attn_bytes_for", load().rs_attn_bytes_for(ctypes.byref(desc), ctypes.byref(rd), max_len, ctypes.byref(out)))
    return out


def rs_attn_plan(desc, rd, rg, max_len: int, plan, status, stream=None):
    st = load().rs_attn_plan(desc, rd, rg, max_len, _ptr(plan), _ptr(status), _stream(stream))
    if st:
        _check("rs_attn_plan", st)


def rs_attend(desc, kv, rd, rg, attn, plan, y, work, status, stream=None):
    st = load().rs_attend(desc, kv, rd, rg, attn, _ptr(plan), _ptr(y), _ptr(work), _ptr(status), _stream(stream))
    if st:
        _check("rs_attend", st)
