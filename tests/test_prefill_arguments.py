"""CPU checks that the Python calls of the ragged prefill refuse tensors that the
kernels would misread or could not reach, before anything is enqueued.

The tensors are fakes that say they are on a GPU; the binding's functions are
replaced by recorders, so no call reaches the library."""
from __future__ import annotations

import types

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from rs_decode_gb300 import binding as rb
from rs_decode_gb300.layer import Layer
from rs_decode_gb300.prefill import Ragged, qk_norm

pytestmark = pytest.mark.filterwarnings("ignore:Accessing the data pointer of FakeTensor")

T, R, H, G, D = 10, 3, 4, 2, 128
BF16, F16, F32, I16, I32 = torch.bfloat16, torch.float16, torch.float32, torch.int16, torch.int32


@pytest.fixture
def calls(monkeypatch):
    """Names of the entry points that were reached."""
    seen = []
    for name in ("rs_qk_norm", "rs_prefill_gdn", "rs_ragged_plan"):
        monkeypatch.setattr(rb, name, lambda *a, _n=name, **k: seen.append(_n))
    with FakeTensorMode():
        yield seen


def fake(*shape, dtype=BF16, device="cuda"):
    return torch.empty(shape, dtype=dtype, device=device)




# ----------------------------------------------------------------------------- norms
def norm_args(**kw):
    a = dict(q=fake(T, H, D), k=fake(T, G, D), wq=fake(D), wk=fake(D), positions=fake(T, dtype=I32), inv_freq=fake(32, dtype=F32),
             out=(fake(T, H, D), fake(T, G, D)))
    a.update(kw)
    return a.pop("q"), a.pop("k"), a


NORM_WRONG = {
    "q": lambda: [fake(T, H, D, dtype=F16), fake(T, H, D, device="cpu"), fake(T, H, D, dtype=torch.uint16)],
    "k": lambda: [fake(T, G, D, dtype=F16), fake(T, G, D, device="cpu")],
    "wq": lambda: [fake(D, dtype=F16), fake(D, device="cpu")],
    "wk": lambda: [fake(D, dtype=F16), fake(D, device="cpu")],
    "positions": lambda: [fake(T, dtype=torch.int64), fake(T, dtype=I32, device="cpu")],
    "inv_freq": lambda: [fake(32, dtype=F16), fake(32, dtype=F32, device="cpu")],
    "out": lambda: [(fake(T, H, D, device="cpu"), None), (None, fake(T, G, D, device="cpu")), (fake(T, H, D, dtype=F16), None),
                    (None, fake(T, G, D, dtype=F16)), (fake(T, H, D, device="cuda:1"), None)],
}


def test_norm_reaches_the_library(calls):
    q, k, kw = norm_args()
    qk_norm(q, k, **kw)
    qk_norm(q.view(I16), None)
    qk_norm(None, k)
    assert calls == ["rs_qk_norm"] * 3


@pytest.mark.parametrize("name", NORM_WRONG)
def test_norm_refusals(calls, name):
    for bad in NORM_WRONG[name]():
        q, k, kw = norm_args(**{name: bad})
        with pytest.raises(ValueError):
            qk_norm(q, k, **kw)
    assert calls == []


# ----------------------------------------------------------------------------- plan
def ragged(**kw):
    r = object.__new__(Ragged)
    r.desc = rb.RaggedDesc(R, T, 64, 4, 5)
    r.counts, r.arrays, r.status_word = fake(4, dtype=I32), None, fake(1, dtype=I32)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def test_plan_refusals(calls):
    i = lambda n, **kw: fake(n, **{"dtype": I32, **kw})
    ragged().plan(i(R), i(R), i(5))
    assert calls == ["rs_ragged_plan"]
    for a in ((i(R, device="cpu"), i(R), i(5)), (i(R), i(R, device="cpu"), i(5)), (i(R), i(R), i(5, device="cpu")),
              (i(R, dtype=torch.int64), i(R), i(5)), (i(R, device="cuda:1"), i(R), i(5)), (i(R), i(R), i(4)), (i(R), i(R), None)):
        with pytest.raises(ValueError):
            ragged().plan(*a)
    with pytest.raises(ValueError):
        ragged(counts=fake(4, dtype=I32, device="cpu")).plan(i(R, device="cpu"), None, i(5, device="cpu"))
    assert calls == ["rs_ragged_plan"]


# ----------------------------------------------------------------------------- prefill
def layer(precision=rb.PREC_FP32, device="cuda"):
    x = object.__new__(Layer)
    x.desc = rb.LayerDesc(rb.GDN, 8, H, G, D, D, 16, 0, 16, precision)
    x.H, x.G, x.N, x.P, x.base, x.state = H, G, D, D, fake(8, dtype=I32, device=device), None
    x._prefill_bytes = types.MethodType(lambda self, rd, max_len: 1024, x)
    return x


def prefill_args(**kw):
    a = dict(ragged=ragged(), q=fake(T, G, D), k=fake(T, G, D), v=fake(T, H, D), alpha=fake(T, H, dtype=F32), beta=fake(T, H, dtype=F32),
             max_len=T, rows=fake(R, dtype=I32), start=fake(R, dtype=I32), pool=fake(5, H, D, D, dtype=F32), y=fake(T, H, D),
             work=fake(1024, dtype=torch.uint8))
    a.update(kw)
    return a


PREFILL_WRONG = {
    "ragged": lambda: [ragged(counts=fake(4, dtype=I32, device="cuda:1"))],
    "q": lambda: [fake(T, G, D, dtype=F16), fake(T, G, D, device="cpu"), fake(T, G, D, device="cuda:1")],
    "k": lambda: [fake(T, G, D, dtype=F16), fake(T, G, D, device="cpu")],
    "v": lambda: [fake(T, H, D, dtype=F16), fake(T, H, D, device="cpu")],
    "alpha": lambda: [fake(T, H), fake(T, H, dtype=F32, device="cpu")],
    "beta": lambda: [fake(T, H, dtype=I32), fake(T, H, dtype=F32, device="cpu")],
    "rows": lambda: [fake(R, dtype=torch.int64), fake(R, dtype=I32, device="cpu")],
    "start": lambda: [fake(R + 1, dtype=I32), fake(R, dtype=I32, device="cpu")],
    "pool": lambda: [fake(5, H, D, D, dtype=I32), fake(5, H, D, D), fake(5, H, D, D, dtype=F32, device="cpu")],
    "y": lambda: [fake(T, H, D, dtype=F16), fake(T, H, D, device="cpu"), fake(T, H, D, device="cuda:1"), fake(T - 1, H, D)],
    "work": lambda: [fake(1024, dtype=torch.uint8, device="cpu"), fake(1023, dtype=torch.uint8)],
}


def test_prefill_reaches_the_library(calls):
    layer().prefill(**prefill_args())
    layer().prefill(**prefill_args(y=None, work=None, pool=None, rows=None, start=None))
    layer(rb.PREC_SHARED_BF16).prefill(**prefill_args(pool=fake(5, H, D, D), y=fake(T, H, D, dtype=I16)))
    assert calls == ["rs_prefill_gdn"] * 3


@pytest.mark.parametrize("name", PREFILL_WRONG)
def test_prefill_refusals(calls, name):
    for bad in PREFILL_WRONG[name]():
        with pytest.raises(ValueError):
            layer().prefill(**prefill_args(**{name: bad}))
    assert calls == []


def test_prefill_pool_of_a_bf16_layer(calls):
    for bad in (fake(5, H, D, D, dtype=F16), fake(5, H, D, D, dtype=F32)):
        with pytest.raises(ValueError):
            layer(rb.PREC_SHARED_BF16).prefill(**prefill_args(pool=bad))
    assert calls == []


def test_layer_on_the_host_is_refused(calls):
    cpu = {k: v.cpu() if isinstance(v, torch.Tensor) else v for k, v in prefill_args().items()}
    with pytest.raises(ValueError, match="CUDA"):
        layer(device="cpu").prefill(**{**cpu, "ragged": ragged(counts=fake(4, dtype=I32, device="cpu"))})
    assert calls == []


# ----------------------------------------------------------------------------- nothing to do
def test_norm_of_no_rows():
    """An empty tensor has no address; the descriptor is still checked."""
    import ctypes

    from rs_decode_gb300 import build
    build.build()
    d = rb.QkDesc(0, 4, 2, 128, rb.NORM_L2, 64, 0, 1e-6, 0.0, 1.0, 1.0, 512, 256, 512, 256)
    assert rb.load().rs_qk_norm(ctypes.byref(d), *[None] * 9) == 0
    d.D = 96
    assert rb.load().rs_qk_norm(ctypes.byref(d), *[None] * 9) == 2
    with FakeTensorMode():
        q, k = qk_norm(fake(0, H, D), fake(0, G, D), positions=fake(0, dtype=I32), inv_freq=fake(32, dtype=F32), stream=0)
        assert q.shape == (0, H, D) and k.shape == (0, G, D)


# ----------------------------------------------------------------------------- what a layer keeps
def test_a_layer_keeps_no_size_for_every_length():
    """Servers meet any longest length; the sizes stay right, and nothing grows with their number."""
    from rs_decode_gb300 import build
    build.build()
    x = Layer("gdn", 2, H, G, D, D, 16, device="cpu")
    rd = rb.RaggedDesc(R, 5000, 0, 0, 0)
    for n in [1, 12, 13, *range(100, 1100), 1, 13, 100]:
        assert x._prefill_bytes(rd, n) == rb.rs_prefill_bytes_for(x.desc, rd, n)
    kept = sum(len(v) for v in vars(x).values() if isinstance(v, (dict, list, set, tuple)))
    assert kept < 20
