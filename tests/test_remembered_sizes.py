"""The workspace sizes that a cache or a layer remembers from call to call, while another thread
asks the same object about another shape: each call gets its own shape's sizes."""
from __future__ import annotations

import threading

import pytest

from rs_decode_gb300 import binding as rb
from rs_decode_gb300.attention import KVCache
from rs_decode_gb300.layer import Layer


@pytest.fixture(scope="module", autouse=True)
def lib():
    from rs_decode_gb300 import build
    build.build()
    return rb.load()


def interrupted(cls, name):
    """cls whose attribute ``name`` lets another thread run ``meanwhile`` after each of its reads and writes."""
    def after(self):
        do = self.__dict__.pop("meanwhile", None)
        if do:
            t = threading.Thread(target=do)
            t.start()
            t.join()
            self.meanwhile = do

    def get(self):
        value = self.__dict__["_kept"]
        after(self)
        return value

    def put(self, value):
        self.__dict__["_kept"] = value
        after(self)

    return type(cls.__name__, (cls,), {name: property(get, put)})


@pytest.mark.parametrize("type", ["bf16", "e4m3"])
@pytest.mark.parametrize("first", [False, True])
def test_attention_sizes(type, first):
    small, large = rb.RaggedDesc(4, 4, 0, 0, 0), rb.RaggedDesc(4, 2000, 0, 0, 0)
    c = interrupted(KVCache, "_sizes")(8, 2, 128, 5, 4, type=type, device="cpu")
    want = rb.rs_attn_bytes_for(c.desc, large, 1000)
    assert want.work > rb.rs_attn_bytes_for(c.desc, small, 1).work
    if not first:
        c._bytes(large, 1000)  # remembered before the other thread asks
    c.meanwhile = lambda: c._bytes(small, 1)
    got = c._bytes(large, 1000)
    assert (got.plan, got.work) == (want.plan, want.work)


@pytest.mark.parametrize("first", [False, True])
def test_prefill_size(first):
    small, large = rb.RaggedDesc(2, 64, 0, 0, 0), rb.RaggedDesc(2, 4000, 0, 0, 0)
    x = interrupted(Layer, "_prefill_size")("gdn", 2, 4, 2, 128, 128, 16, device="cpu")
    want = rb.rs_prefill_bytes_for(x.desc, large, 4000)
    assert want > rb.rs_prefill_bytes_for(x.desc, small, 1)
    if not first:
        x._prefill_bytes(large, 4000)
    x.meanwhile = lambda: x._prefill_bytes(small, 1)
    assert x._prefill_bytes(large, 4000) == want
