"""What the library keeps per process against what the CUDA context keeps: the
calls work, with the same bits, in the context that follows a cudaDeviceReset.
Each test runs in a child process, whose context is its own."""
import os
import subprocess
import sys

import pytest

from sparse_attention_video_tra_b200 import build as trabuild

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    trabuild.build()
    yield


def child(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]


# device memory from the CUDA runtime that torch has loaded; torch itself holds none here
RESET = """
import ctypes
import numpy as np
import torch
import sparse_attention_video_tra_b200 as tra

rt = ctypes.CDLL("libcudart.so.12")
def ok(status): assert status == 0, status
def alloc(nbytes, data=None):
    p = ctypes.c_void_p()
    ok(rt.cudaMalloc(ctypes.byref(p), ctypes.c_size_t(nbytes)))
    ok(rt.cudaMemset(p, 0, ctypes.c_size_t(nbytes)))
    if data is not None:
        ok(rt.cudaMemcpy(p, data.ctypes.data_as(ctypes.c_void_p), ctypes.c_size_t(nbytes), 1))
    return p.value

def everything():
    p = tra.Plan(5, 17, 23, 2, 128, 1.0, 0.5, 0.8, 3, 1)
    i = p.info
    n, rows = i.heads * i.N_pad * i.d, i.heads * i.N_pad
    rng = np.random.default_rng(1)
    q, k, v = (alloc(2 * n, (rng.standard_normal(n).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)) for _ in range(3))
    out, lse, frames, flse = alloc(4 * n), alloc(4 * rows), alloc(4 * n), alloc(4 * rows)
    grads = [alloc(4 * n) for _ in range(3)]
    ent, mask, cache = alloc(4 * rows), alloc(i.mask_bytes), alloc(p.cache_info.cache_bytes)
    nws, ncw = tra.tra_attention_backward_bytes(p.handle), tra.tra_cache_attention_bytes(p.handle, 5)
    ws, cw = alloc(nws), alloc(ncw)
    token, radius = alloc(4 * 60, np.arange(60, dtype=np.int32)), alloc(4 * 120, np.full(120, 4, np.int32))
    tout, tlse = alloc(4 * 120 * i.d), alloc(4 * 120)
    tra.tra_entropy(p.handle, q, k, ent)
    tra.tra_radius_and_mask(p.handle, ent, mask, i.mask_bytes)
    tra.tra_attention(p.handle, q, k, v, mask, out)
    tra.tra_attention_lse(p.handle, q, k, v, mask, out, lse)
    tra.tra_attention_backward(p.handle, q, k, v, mask, out, lse, out, *grads, ws, nws)
    tra.tra_cache_store(p.handle, k, v, 0, 5, cache, p.cache_info.cache_bytes)
    tra.tra_cache_attention(p.handle, q, 0, 5, cache, p.cache_info.cache_bytes, 5, mask, frames, flse, cw, ncw)
    tra.tra_cache_attention_tokens(p.handle, q, token, radius, 1, cache, p.cache_info.cache_bytes, 5, tout, tlse)
    tra.tra_cache_attention_tokens(p.handle, q, token, radius, 60, cache, p.cache_info.cache_bytes, 5, tout, tlse)
    ok(rt.cudaDeviceSynchronize())
    assert tra.tra_plan_status(p.handle) == 0
    got = []
    for ptr, nbytes in [(grads[2], 4 * n), (lse, 4 * rows), (flse, 4 * rows), (tout, 4 * 120 * i.d)]:
        host = np.empty(nbytes, np.uint8)
        ok(rt.cudaMemcpy(host.ctypes.data_as(ctypes.c_void_p), ctypes.c_void_p(ptr), ctypes.c_size_t(nbytes), 2))
        got.append(host)
    assert got[0].any() and got[3].any()
    return got

first = everything()
for _ in range(2):
    ok(rt.cudaDeviceReset())
    for a, b in zip(first, everything()):
        assert np.array_equal(a, b)
"""


def test_calls_after_a_device_reset():
    child(RESET)
