"""CPU checks of the paged cache and its attention: sizes, and refusals of bad
arguments before anything is enqueued, by the C entry points and by the Python
calls (whose tensors are fakes that say they are on a GPU)."""
from __future__ import annotations

import ctypes

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from rs_decode_gb300 import binding as rb
from rs_decode_gb300.attention import KVCache
from rs_decode_gb300.prefill import Ragged

pytestmark = pytest.mark.filterwarnings("ignore:Accessing the data pointer of FakeTensor")

INVALID, UNSUPPORTED = 1, 2
BF16, F16, F32, I16, I32, U8 = torch.bfloat16, torch.float16, torch.float32, torch.int16, torch.int32, torch.uint8


@pytest.fixture(scope="module")
def lib():
    from rs_decode_gb300 import build
    build.build()
    return rb.load()


# ----------------------------------------------------------------------------- the C entry points
def desc(**kw):
    d = dict(Hq=8, Hk=2, D=128, type=rb.KV_BF16, page=64, n_pages=20, max_pages=4)
    d.update(kw)
    return rb.KvDesc(**d)


def ragged(**kw):
    d = dict(R=3, tokens_cap=100, block=0, max_blocks=0, n_free=0)
    d.update(kw)
    return rb.RaggedDesc(**d)


def addresses(cls, **kw):
    a = cls(*[0x100000 * (i + 1) for i in range(len(cls._fields_))])
    for k, v in kw.items():
        setattr(a, k, v)
    return a


DESCRIPTORS = [
    ({}, 0), (dict(D=64), 0), (dict(D=96), UNSUPPORTED), (dict(D=256), UNSUPPORTED), (dict(page=16), 0), (dict(page=256), 0),
    (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(page=512), UNSUPPORTED), (dict(page=0), INVALID),
    (dict(Hq=9), INVALID), (dict(Hq=0), INVALID), (dict(Hk=0), INVALID), (dict(Hk=-2), INVALID), (dict(Hq=256, Hk=2), 0),
    (dict(Hq=258, Hk=2), UNSUPPORTED), (dict(Hq=65536), INVALID), (dict(type=2), INVALID), (dict(type=-1), INVALID),
    (dict(n_pages=0), INVALID), (dict(n_pages=1 << 30), INVALID), (dict(n_pages=(1 << 30) - 1), 0), (dict(max_pages=0), INVALID),
    (dict(max_pages=1 << 24), 0), (dict(max_pages=(1 << 24) + 1), INVALID)]


@pytest.mark.parametrize("kw,status", DESCRIPTORS)
def test_cache_descriptor(lib, kw, status):
    out = rb.KvBytes()
    assert lib.rs_kv_bytes_for(ctypes.byref(desc(**kw)), ctypes.byref(out)) == status


def test_cache_sizes(lib):
    s = rb.rs_kv_bytes_for(desc())
    assert s.k == s.v == 20 * 2 * 64 * 128 * 2 and s.ks == s.vs == 0
    s = rb.rs_kv_bytes_for(desc(type=rb.KV_E4M3, D=64, page=16))
    assert s.k == s.v == 20 * 2 * 16 * 64 and s.ks == s.vs == 20 * 2 * 16
    big = rb.rs_kv_bytes_for(desc(n_pages=1 << 29, page=256, max_pages=1 << 22))
    assert big.k == (1 << 29) * 2 * 256 * 128 * 2  # past 32 bits
    assert lib.rs_kv_bytes_for(ctypes.byref(desc()), None) == INVALID
    assert lib.rs_kv_bytes_for(None, None) == INVALID


def test_plan_and_workspace_sizes(lib):
    one = rb.rs_attn_bytes_for(desc(), ragged(), 1)
    many = rb.rs_attn_bytes_for(desc(), ragged(R=1000), 1)
    assert many.plan - one.plan == 997 * 48 and many.work == one.work
    # two parts a CTA of 16 rows, of 32, or of 256: sums, largest score, sum of weights
    assert one.work == 152 * 2 * 16 * 130 * 4
    assert rb.rs_attn_bytes_for(desc(), ragged(), 8).work == 152 * 2 * 32 * 130 * 4
    assert rb.rs_attn_bytes_for(desc(), ragged(), 9).work == 152 * 2 * 256 * 130 * 4
    assert rb.rs_attn_bytes_for(desc(type=rb.KV_E4M3), ragged(), 9).work == 152 * 2 * (256 + 16) * 130 * 4
    assert rb.rs_attn_bytes_for(desc(D=64), ragged(), 9).work == 152 * 2 * 256 * 66 * 4
    out = rb.AttnBytes()
    call = lambda d, rd, n, o=out: lib.rs_attn_bytes_for(ctypes.byref(d), ctypes.byref(rd), n, ctypes.byref(o) if o else None)
    assert call(desc(), ragged(), 0) == INVALID
    assert call(desc(), ragged(), 1, None) == INVALID
    assert call(desc(), ragged(R=0), 1) == INVALID
    assert call(desc(), ragged(tokens_cap=0), 1) == INVALID
    assert call(desc(max_pages=1 << 24), ragged(R=129), 1) == INVALID
    assert call(desc(D=32), ragged(), 1) == UNSUPPORTED


def kv(e4m3=False):
    return addresses(rb.Kv) if e4m3 else addresses(rb.Kv, ks=None, vs=None)


def call_write(lib, fn="rs_kv_write", d=None, cache=None, rd=None, rg=None, pages=0x40, k=0x1000, v=0x2000, ld_k=256, ld_v=256, status=0x80):
    a = [ctypes.byref(d or desc()), ctypes.byref(cache or kv()), ctypes.byref(rd or ragged()), ctypes.byref(rg or addresses(rb.RaggedArrays)),
         pages, k, v]
    return getattr(lib, fn)(*a, *([ld_k, ld_v] if fn == "rs_kv_write" else []), status, None)


@pytest.mark.parametrize("fn", ["rs_kv_write", "rs_kv_read"])
def test_write_and_read_refusals(lib, fn):
    e = desc(type=rb.KV_E4M3)
    for kw in (dict(pages=None), dict(pages=0x42), dict(k=None), dict(k=0x1008), dict(v=None), dict(v=0x2002), dict(status=None),
               dict(status=0x81), dict(cache=addresses(rb.Kv)), dict(cache=addresses(rb.Kv, ks=None, vs=None, k=None)),
               dict(cache=addresses(rb.Kv, ks=None, vs=None, v=0x200008)), dict(d=e, cache=kv()),
               dict(d=e, cache=addresses(rb.Kv, ks=0x300008)), dict(rg=addresses(rb.RaggedArrays, token_req=None)),
               dict(rg=addresses(rb.RaggedArrays, token_pos=0x500008)), dict(rd=ragged(R=0))):
        assert call_write(lib, fn, **kw) == INVALID, kw
    assert call_write(lib, fn, d=desc(D=32)) == UNSUPPORTED
    if fn == "rs_kv_write":
        for kw in (dict(ld_k=248), dict(ld_k=260), dict(ld_v=255), dict(ld_v=(1 << 31) + 8)):
            assert call_write(lib, **kw) == INVALID, kw


def test_attention_plan_refusals(lib):
    call = lambda d=None, rd=None, rg=None, n=4, plan=0x1000, st=0x80: lib.rs_attn_plan(
        ctypes.byref(d or desc()), ctypes.byref(rd or ragged()), ctypes.byref(rg or addresses(rb.RaggedArrays)), n, plan, st, None)
    assert call(n=0) == call(plan=None) == call(plan=0x1040) == call(st=None) == call(st=0x82) == INVALID
    assert call(rg=addresses(rb.RaggedArrays, cu_tokens=None)) == INVALID
    assert call(d=desc(page=4)) == UNSUPPORTED


def test_attend_refusals(lib):
    def call(a=(), d=None, cache=None, rd=None, rg=None, plan=0x4000, y=0x5000, work=0x6000, st=0x80, none=False):
        x = rb.Attn(0x1000, 1024, 0x2000, 0.1, 5)
        for n, v in dict(a).items():
            setattr(x, n, v)
        return lib.rs_attend(ctypes.byref(d or desc()), ctypes.byref(cache or kv()), ctypes.byref(rd or ragged()),
                             ctypes.byref(rg or addresses(rb.RaggedArrays)), None if none else ctypes.byref(x), plan, y, work, st, None)
    for a in (dict(q=None), dict(q=0x1008), dict(ld_q=1016), dict(ld_q=1028), dict(pages=None), dict(pages=0x2002), dict(scale=-1.0), dict(scale=0.0),
              dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3e38), dict(max_len=0), dict(max_len=-3), dict(ld_q=(1 << 31) + 8)):
        assert call(a) == INVALID, a
    for kw in (dict(none=True), dict(plan=None), dict(plan=0x4040), dict(y=None), dict(y=0x5008), dict(work=None), dict(work=0x6010),
               dict(st=None), dict(cache=addresses(rb.Kv)), dict(rd=ragged(tokens_cap=0)), dict(rg=addresses(rb.RaggedArrays, cu_tokens=0x100002)),
               dict(d=desc(Hq=7))):
        assert call(**kw) == INVALID, kw
    assert call(d=desc(D=256)) == UNSUPPORTED


# ----------------------------------------------------------------------------- the Python calls
T, R, HQ, HK, D = 10, 3, 8, 2, 128


@pytest.fixture
def calls(monkeypatch, lib):
    """Names of the entry points that were reached."""
    seen = []
    for name in ("rs_kv_write", "rs_kv_read", "rs_attn_plan", "rs_attend"):
        monkeypatch.setattr(rb, name, lambda *a, _n=name, **k: seen.append(_n))
    monkeypatch.setattr(rb, "_current_device", lambda: 0)
    with FakeTensorMode():
        yield seen


def fake(*shape, dtype=BF16, device="cuda"):
    return torch.empty(shape, dtype=dtype, device=device)


def plan_of(device="cuda"):
    r = object.__new__(Ragged)
    r.desc, r.counts, r.arrays = rb.RaggedDesc(R, T, 0, 0, 0), fake(4, dtype=I32, device=device), None
    return r


def cache(type="bf16"):
    return KVCache(HQ, HK, D, 20, 4, page=64, type=type, device="cuda")


def pages(*shape, **kw):
    return fake(*(shape or (R, 4)), **{"dtype": I32, **kw})


def test_the_calls_reach_the_library(calls):
    for type in ("bf16", "e4m3"):
        c = cache(type)
        rows = fake(T, (HQ + 2 * HK) * D)
        q, k, v = rows[:, :HQ * D].unflatten(1, (HQ, D)), rows[:, HQ * D:(HQ + HK) * D].unflatten(1, (HK, D)), fake(T + 2, HK, D, dtype=I16)
        p = c.plan(plan_of(), T)
        c.plan(plan_of(), T, out=p)
        c.write(plan_of(), k, v, pages())
        a, b = c.read(plan_of(), pages())
        assert a.shape == b.shape == (T, HK, D) and a.dtype is BF16
        y = c.attend(plan_of(), q, pages(), p, max_len=T)
        assert y.shape == (T, HQ, D) and y.dtype is BF16
        c.attend(plan_of(), q, pages(), p, max_len=T, y=y, work=c.workspace(plan_of(), T), scale=0.5)
    assert calls == ["rs_attn_plan", "rs_attn_plan", "rs_kv_write", "rs_kv_read", "rs_attend", "rs_attend"] * 2


def test_write_and_read_tensors(calls):
    c = cache()
    k = fake(T, HK, D)
    for bad in (fake(T, HK, D, dtype=F16), fake(T, HK, D, device="cpu"), fake(T, HK, D, device="cuda:1"), fake(T - 1, HK, D), fake(T, HQ, D),
                fake(T, HK, 2 * D)[:, :, ::2], fake(T, 2 * HK, D)[:, ::2], fake(T, HK * D)):
        for a in ((bad, k), (k, bad)):
            with pytest.raises(ValueError):
                c.write(plan_of(), *a, pages())
    for bad in (pages(R, 5), pages(R + 1, 4), pages(dtype=torch.int64), pages(device="cpu"), pages(R * 4)):
        with pytest.raises(ValueError):
            c.write(plan_of(), k, k, bad)
        with pytest.raises(ValueError):
            c.read(plan_of(), bad)
    for bad in (fake(T, HK, D, dtype=F16), fake(T, HK, D, device="cpu"), fake(T - 1, HK, D), fake(T, HK, 64)):
        with pytest.raises(ValueError):
            c.read(plan_of(), pages(), out=(bad, k))
    with pytest.raises(ValueError):
        c.write(plan_of("cuda:1"), k, k, pages())
    assert calls == []


def test_attend_tensors(calls):
    c = cache()
    p, w = c.plan(plan_of(), T), c.workspace(plan_of(), T)
    calls.clear()
    ok = dict(q=fake(T, HQ, D), pages=pages(), plan=p, y=fake(T, HQ, D), work=w)
    wrong = {
        "q": [fake(T, HQ, D, dtype=F32), fake(T, HQ, D, device="cpu"), fake(T - 1, HQ, D), fake(T, HK, D)],
        "pages": [pages(R, 8)[:, ::2], pages(R, 3), pages(device="cpu"), pages(dtype=torch.int64)],
        "plan": [fake(p.numel() - 1, dtype=U8), fake(p.numel(), dtype=U8, device="cpu"), fake(p.numel(), dtype=U8, device="cuda:1")],
        "y": [fake(T, HQ, D, dtype=F16), fake(T - 1, HQ, D), fake(T, HQ, D, device="cpu"), fake(T, HK, D)],
        "work": [fake(w.numel() - 1, dtype=U8), fake(w.numel(), dtype=U8, device="cpu")],
    }
    for name, bads in wrong.items():
        for bad in bads:
            a = {**ok, name: bad}
            with pytest.raises(ValueError):
                c.attend(plan_of(), a.pop("q"), a.pop("pages"), a.pop("plan"), max_len=T, **a)
    with pytest.raises(ValueError):
        c.plan(plan_of(), T, out=fake(p.numel() - 1, dtype=U8))
    with pytest.raises(ValueError):
        c.plan(plan_of("cuda:1"), T)
    with pytest.raises(rb.RsError):
        c.plan(plan_of(), 0)
    assert calls == []


def test_another_current_device_is_refused(calls, monkeypatch):
    c = cache()
    k = fake(T, HK, D)
    monkeypatch.setattr(rb, "_current_device", lambda: 1)
    for call in (lambda: c.write(plan_of(), k, k, pages()), lambda: c.read(plan_of(), pages()), lambda: c.plan(plan_of(), T),
                 lambda: c.attend(plan_of(), fake(T, HQ, D), pages(), fake(100_000, dtype=U8), max_len=T)):
        with pytest.raises(ValueError, match="current"):
            call()
    assert calls == []


def test_cache_on_the_host_is_refused(lib):
    c = KVCache(HQ, HK, D, 5, 4, device="cpu")
    k = torch.zeros(T, HK, D, dtype=BF16)
    r = object.__new__(Ragged)
    r.desc, r.counts, r.arrays = rb.RaggedDesc(R, T, 0, 0, 0), torch.zeros(4, dtype=I32), None
    table = torch.zeros(R, 4, dtype=I32)
    for call in (lambda: c.write(r, k, k, table), lambda: c.read(r, table), lambda: c.plan(r, T)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_cache_construction(lib):
    with pytest.raises(ValueError):
        KVCache(8, 2, 128, 5, 4, type="fp8", device="cpu")
    for kw in (dict(Hq=7), dict(D=96), dict(page=24), dict(n_pages=0)):
        a = {**dict(Hq=8, Hk=2, D=128, n_pages=5, max_pages=4, page=64, device="cpu"), **kw}
        with pytest.raises(rb.RsError):
            KVCache(**a)
    c = KVCache(8, 2, 64, 5, 4, page=16, type="e4m3", device="cpu")
    assert c.k.shape == (5, 2, 16, 64) and c.k.dtype is U8 and c.k_exp.shape == (5, 2, 16)


def test_a_cache_keeps_no_size_for_every_length(lib):
    c = KVCache(8, 2, 64, 5, 4, device="cpu")
    rd = rb.RaggedDesc(R, T, 0, 0, 0)
    for n in [1, 9, *range(10, 600), 1]:
        assert c._bytes(rd, n).work == rb.rs_attn_bytes_for(c.desc, rd, n).work
    assert sum(len(v) for v in vars(c).values() if isinstance(v, (dict, list, set, tuple))) < 10
