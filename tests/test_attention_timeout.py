"""The bounded waits of the attention kernels: where a part of a CTA does not do its work, the
others' waits run out, raise RS_DEV_TIMEOUT, wait for the copies in flight, free the tensor memory and return.

tests/csrc/attn_stall_*.cu run the kernels' own roles with some of them left out and a limit of 5 ms.  The CPU
test only builds them; the GPU tests run them, and an ordinary call after each, whose result has to be right."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OUT = os.path.join(ROOT, "tests", "_build", "libattn_stall.so")
LIMIT_NS = 5_000_000


def _build() -> str:
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    os.makedirs(os.path.dirname(OUT), exist_ok=True)
    tmp = OUT + f".tmp{os.getpid()}"
    csrc = os.path.join(ROOT, "tests", "csrc")
    cmd = [nvcc, "-std=c++17", "-O2", "-gencode", "arch=compute_103a,code=sm_103a", "-shared", "-Xcompiler", "-fPIC", "--threads", "2",
           f"-DRS_WAIT_LIMIT_NS={LIMIT_NS}ull", "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "rs_decode_gb300", "csrc"),
           "-I", csrc, os.path.join(csrc, "attn_stall_short.cu"), os.path.join(csrc, "attn_stall_long.cu"), "-o", tmp, "--cudart=shared"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    os.replace(tmp, OUT)
    return OUT


@pytest.fixture(scope="module")
def lib():
    return ctypes.CDLL(_build())


def test_stalled_kernels_build(lib):
    assert lib.rs_test_short_stall and lib.rs_test_long_stall


def _stall(lib, b, q, max_len, fn, idle):
    import torch
    from rs_decode_gb300 import binding as rb
    c = b.cache
    plan, work = c.plan(b.ragged, max_len), c.workspace(b.ragged, max_len)
    y = torch.full((b.cap, b.Hq, b.D), 4.0, dtype=torch.bfloat16, device="cuda")
    seen = torch.zeros(2, dtype=torch.int32, device="cuda")
    attn = rb.Attn(q.data_ptr(), b.Hq * b.D, b.pages.data_ptr(), b.D ** -0.5, max_len)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    begin.record()
    st = getattr(lib, fn)(ctypes.byref(c.desc), ctypes.byref(c.kv), ctypes.byref(b.ragged.desc), ctypes.byref(attn),
                          *(ctypes.c_void_p(t.data_ptr()) for t in (plan, y, work, c.status_word)), idle, ctypes.c_void_p(seen.data_ptr()),
                          ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    end.record()
    assert st == 0
    torch.cuda.synchronize()
    return begin.elapsed_time(end), seen.tolist(), c.status()


@pytest.mark.gpu
@pytest.mark.parametrize("type", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 4])
@pytest.mark.parametrize("idle", [1, 2])
def test_few_rows(lib, type, n, idle):
    import torch
    from rs_decode_gb300 import binding as rb
    from test_gpu_attention import Batch
    b = Batch([n] * 20, [9000] * 20, 16, 2, 128, type, 32)
    q = b.randn(b.cap, 16, 128).to(torch.bfloat16)
    assert _stall(lib, b, q, n, "rs_test_short_stall", 0)[1:] == ([0, 0], 0)  # nothing left out
    ms, (ctas, begun), status = _stall(lib, b, q, n, "rs_test_short_stall", idle)
    assert status == rb.DEV_TIMEOUT and 140 <= ctas <= 152  # the last few may have no share
    assert (begun == 0) == (idle == 1)
    assert LIMIT_NS * 1e-6 * 0.9 <= ms < 2000
    b.check(q, b.attend(q))


@pytest.mark.gpu
@pytest.mark.parametrize("type,idle", [("bf16", 1), ("bf16", 2), ("bf16", 4), ("e4m3", 1), ("e4m3", 2), ("e4m3", 4), ("e4m3", 8)])
@pytest.mark.parametrize("n", [10, 70])
def test_many_rows(lib, type, n, idle):
    import torch
    from rs_decode_gb300 import binding as rb
    from test_gpu_attention import Batch
    b = Batch([n] * 20, [9000] * 20, 16, 2, 128, type, 32)
    q = b.randn(b.cap, 16, 128).to(torch.bfloat16)
    assert _stall(lib, b, q, n, "rs_test_long_stall", 0)[1:] == ([0, 0], 0)
    ms, (ctas, begun), status = _stall(lib, b, q, n, "rs_test_long_stall", idle)
    assert status == rb.DEV_TIMEOUT and 140 <= ctas <= 152  # the last few may have no share
    assert (begun == 0) == (idle == 1)
    assert LIMIT_NS * 1e-6 * 0.9 <= ms < 2000
    b.check(q, b.attend(q))
