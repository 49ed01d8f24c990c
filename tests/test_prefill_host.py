"""CPU checks of the ragged prefill's entry points: sizes, and refusals of bad
arguments before anything is enqueued."""
from __future__ import annotations

import ctypes

import pytest
import torch

from rs_decode_gb300 import binding as rb

INVALID, UNSUPPORTED, CAPACITY = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from rs_decode_gb300 import build
    build.build()
    return rb.load()


def ragged(**kw):
    d = dict(R=4, tokens_cap=1000, block=128, max_blocks=8, n_free=10)
    d.update(kw)
    return rb.RaggedDesc(**d)


def addresses(cls, **kw):
    a = cls(*[0x100000 * (i + 1) for i in range(len(cls._fields_))])
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status", [
    ({}, 0), (dict(R=0), INVALID), (dict(R=65536), INVALID), (dict(R=65535), 0), (dict(tokens_cap=0), INVALID),
    (dict(tokens_cap=(1 << 30) + 1), INVALID), (dict(block=100), INVALID), (dict(block=-64), INVALID),
    (dict(max_blocks=0), INVALID), (dict(max_blocks=1 << 29), INVALID), (dict(block=0, max_blocks=0), 0),
    (dict(n_free=-1), INVALID), (dict(n_free=0), 0), (dict(block=1 << 29), 0), (dict(block=(1 << 29) + 64), INVALID)])
def test_ragged_descriptor(lib, kw, status):
    out = rb.RaggedBytes()
    assert lib.rs_ragged_bytes_for(ctypes.byref(ragged(**kw)), ctypes.byref(out)) == status


def test_ragged_sizes(lib):
    s = rb.rs_ragged_bytes_for(ragged())
    assert s.cu_tokens == s.cu_chunks == s.cu_blocks == 5 * 4 and s.counts == 16
    assert s.token_req == s.token_pos == 4000 and s.chunks == (1000 // 64 + 8) * 16 and s.block_table == 4 * 8 * 4
    assert rb.rs_ragged_bytes_for(ragged(block=0)).block_table == 0
    assert lib.rs_ragged_bytes_for(ctypes.byref(ragged()), None) == INVALID
    assert lib.rs_ragged_bytes_for(None, None) == INVALID


def test_plan_refusals(lib):
    rd, ok = ragged(), addresses(rb.RaggedArrays)
    call = lambda rd, lengths, ctx, free, rg, st: lib.rs_ragged_plan(
        ctypes.byref(rd), lengths, ctx, free, ctypes.byref(rg) if rg else None, st, None)
    assert call(rd, None, None, 0x40, ok, 0x80) == INVALID           # no lengths
    assert call(rd, 0x41, None, 0x40, ok, 0x80) == INVALID           # misaligned
    assert call(rd, 0x40, 0x42, 0x40, ok, 0x80) == INVALID
    assert call(rd, 0x40, None, None, ok, 0x80) == INVALID           # blocks, but no free list
    assert call(rd, 0x40, None, 0x40, ok, None) == INVALID           # no status word
    assert call(rd, 0x40, None, 0x40, None, 0x80) == INVALID
    for name in rb._RAGGED:
        assert call(rd, 0x40, None, 0x40, addresses(rb.RaggedArrays, **{name: None}), 0x80) == INVALID, name
    assert call(rd, 0x40, None, 0x40, addresses(rb.RaggedArrays, token_pos=0x100004), 0x80) == INVALID


def qk(**kw):
    d = rb.QkDesc(8, 4, 2, 128, rb.NORM_L2, 0, 0, 1e-6, 0.0, 1.0, 1.0, 512, 256, 512, 256)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("kw,status", [
    (dict(D=96), UNSUPPORTED), (dict(rot=24), UNSUPPORTED), (dict(rot=-16), INVALID), (dict(rot=144), INVALID),
    (dict(T=-1), INVALID), (dict(Hq=0, Hk=0), INVALID), (dict(Hq=-1), INVALID), (dict(norm=3), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(ld_q=511), INVALID), (dict(ld_q=516), INVALID), (dict(ld_k=248), INVALID), (dict(ld_qo=504), INVALID),
    (dict(ld_ko=8), INVALID), (dict(rot=64), INVALID)])
def test_qk_refusals(lib, kw, status):
    p = [0x1000 * (i + 1) for i in range(8)]
    inv, pos = (None, None)
    assert lib.rs_qk_norm(ctypes.byref(qk(**kw)), p[0], p[1], p[2], p[3], inv, pos, p[6], p[7], None) == status


def test_qk_pointer_refusals(lib):
    p = [0x1000 * (i + 1) for i in range(8)]
    for i in (0, 1, 6, 7):
        for bad in (None, p[i] + 2):
            a = list(p)
            a[i] = bad
            assert lib.rs_qk_norm(ctypes.byref(qk()), a[0], a[1], a[2], a[3], None, None, a[6], a[7], None) == INVALID
    assert lib.rs_qk_norm(None, *([None] * 9)) == INVALID
    assert lib.rs_qk_norm(ctypes.byref(qk(T=0)), p[0], p[1], None, None, None, None, p[6], p[7], None) == 0  # nothing to do


def layer_desc(**kw):
    d = dict(kind=rb.GDN, B=8, H=4, G=2, P=128, N=128, L=16, T_max=0, capacity=16, precision=rb.PREC_FP32)
    d.update(kw)
    return rb.LayerDesc(**d)


def state():
    return addresses(rb.State, ckpt_lp=None, buf_s=None)


def prefill(**kw):
    a = rb.Prefill(0x1000, 0x2000, 0x3000, 0x4000, 0x5000, 256, 256, 512, 0x6000, 0x7000, 0x8000, 4, 100)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def call_prefill(lib, desc=None, st=None, rd=None, rg=None, args=None, y=0x9000, work=0x10000):
    return lib.rs_prefill_gdn(ctypes.byref(desc or layer_desc()), ctypes.byref(st or state()), ctypes.byref(rd or ragged()),
                              ctypes.byref(rg or addresses(rb.RaggedArrays)), ctypes.byref(args or prefill()), y, work, None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(k=0x1008), dict(v=None), dict(alpha=None), dict(beta=0x5002), dict(ld_q=255), dict(ld_k=260),
    dict(ld_v=504), dict(rows=0x6002), dict(start=0x7001), dict(n_pool=-1), dict(n_pool=0), dict(pool=None),
    dict(pool=0x8008), dict(max_len=-1), dict(ld_v=(1 << 31) + 8)])
def test_prefill_argument_refusals(lib, kw):
    assert call_prefill(lib, args=prefill(**kw)) == INVALID


def test_prefill_other_refusals(lib):
    assert call_prefill(lib, desc=layer_desc(kind=rb.KDA)) == UNSUPPORTED
    assert call_prefill(lib, desc=layer_desc(kind=rb.MAMBA2, P=64)) == UNSUPPORTED
    assert call_prefill(lib, desc=layer_desc(P=96)) == UNSUPPORTED
    assert call_prefill(lib, desc=layer_desc(capacity=8)) == CAPACITY
    assert call_prefill(lib, rd=ragged(block=1)) == INVALID
    assert call_prefill(lib, rg=addresses(rb.RaggedArrays, chunks=None)) == INVALID
    assert call_prefill(lib, y=None) == INVALID
    assert call_prefill(lib, y=0x9002) == INVALID
    assert call_prefill(lib, work=None) == INVALID
    assert call_prefill(lib, work=0x10010) == INVALID
    assert call_prefill(lib, rd=ragged(R=9), args=prefill(rows=None)) == INVALID  # more requests than rows
    st = state()
    st.h = None
    assert call_prefill(lib, st=st) == INVALID
    assert lib.rs_prefill_gdn(*([None] * 8)) == INVALID
    n = ctypes.c_size_t(0)
    big = ragged(tokens_cap=1 << 30, R=65535, block=0)
    assert lib.rs_prefill_bytes_for(ctypes.byref(layer_desc(H=1024, G=1024)), ctypes.byref(big), 10, ctypes.byref(n)) == INVALID
    assert lib.rs_prefill_bytes_for(ctypes.byref(layer_desc()), ctypes.byref(ragged()), 10, None) == INVALID


def test_python_layer_refuses_bad_tensors():
    from rs_decode_gb300.layer import packed_stride
    x = torch.zeros(10, 4, 128, dtype=torch.bfloat16)
    assert packed_stride(x, 10, 4, 128, "x") == 512
    row = torch.zeros(10, 1024, dtype=torch.bfloat16)
    assert packed_stride(row[:, :512].unflatten(1, (4, 128)), 10, 4, 128, "x") == 1024
    for bad in (x.float(), x[:5], x[:, :3], x.transpose(0, 1), x.flip(2)[..., ::2], x[:, ::2]):
        with pytest.raises(ValueError):
            packed_stride(bad, 10, 4, 128, "x")


def test_qk_norm_refuses_bad_calls():
    from rs_decode_gb300.prefill import qk_norm
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    for kw in (dict(norm="l3"), dict(positions=torch.zeros(4, dtype=torch.int32)),
               dict(positions=torch.zeros(3, dtype=torch.int32), inv_freq=torch.ones(8)),
               dict(positions=torch.zeros(4, dtype=torch.int64), inv_freq=torch.ones(8)),
               dict(wq=torch.ones(63, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            qk_norm(x, None, **kw)
    with pytest.raises(ValueError):
        qk_norm(None, None)


def test_host_tensors_are_refused():
    """A pointer to host memory would be read on the device."""
    from rs_decode_gb300.prefill import qk_norm
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        qk_norm(x, x)
    with pytest.raises(ValueError, match="CUDA"):
        qk_norm(None, x)
