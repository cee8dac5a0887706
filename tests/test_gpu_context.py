"""What the library keeps per process against what the CUDA context keeps: the
calls work, with the same bits, in the context that follows a cudaDeviceReset,
and a call that fails leaves no error behind for the next one.  Each test runs
in a child process, whose context is its own."""
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


# a launch on the legacy default stream is refused while another stream that
# synchronises with it is being captured: an error on the host, nothing runs
FAILED_LAUNCH = """
import ctypes
import torch
import sparse_attention_video_tra_b200 as tra

rt = ctypes.CDLL("libcudart.so.12")
p = tra.Plan(5, 17, 23, 2, 128, 1.0, 0.5, 0.8, 3, 1, tra.TRA_FLAG_NATURAL)
big = tra.Plan(5, 17, 23, 8, 128, 1.0, 0.5, 0.8, 3, 1, tra.TRA_FLAG_NATURAL)
q, k, v = (torch.randn(2, p.info.N, 128, device="cuda").bfloat16() for _ in range(3))
Q, K, V = (torch.randn(8, p.info.N, 128, device="cuda").bfloat16() for _ in range(3))
ent, mask = p.new_entropy(), p.new_mask()
ent2, mask2 = big.new_entropy(), big.new_mask()
p.radius_and_mask(p.entropy(q, k, ent), mask)
big.radius_and_mask(big.entropy(Q, K, ent2), mask2)
out, lse, Out, Lse = p.new_out(), p.new_lse(), big.new_out(), big.new_lse()
tiles = p.new_tile_major()
cache, cw = p.new_cache(), p.new_cache_workspace(5)
ws, grads = p.new_backward_workspace(), [p.new_out() for _ in range(3)]
p.cache_store(k, v, 0, cache)
token = torch.arange(60, device="cuda", dtype=torch.int32)
radius = torch.full((2, 60), 4, device="cuda", dtype=torch.int32)
tq, tout, tlse = q[:, :60].contiguous(), torch.empty(2, 60, 128, device="cuda"), torch.empty(2, 60, device="cuda")
d = lambda *xs: [x.data_ptr() for x in xs]
tokens = lambda n: tra.tra_cache_attention_tokens(p.handle, *d(tq, token, radius), n, cache.data_ptr(), cache.numel(), 5,
                                                  *d(tout, tlse))
calls = {
    "lse, clusters": lambda: tra.tra_attention_lse(p.handle, *d(q, k, v, mask, out, lse)),
    "lse, pairs": lambda: tra.tra_attention_lse(big.handle, *d(Q, K, V, mask2, Out, Lse)),
    "backward": lambda: tra.tra_attention_backward(p.handle, *d(q, k, v, mask, out, lse, out, *grads, ws), ws.numel()),
    "store": lambda: tra.tra_cache_store(p.handle, *d(k, v), 0, 5, cache.data_ptr(), cache.numel()),
    "frames": lambda: tra.tra_cache_attention(p.handle, q.data_ptr(), 0, 5, cache.data_ptr(), cache.numel(), 5,
                                              *d(mask, out, lse, cw), cw.numel()),
    "one token": lambda: tokens(1), "a few": lambda: tokens(30), "groups": lambda: tokens(60),
    "attention": lambda: tra.tra_attention(p.handle, *d(q, k, v, mask, out)),
    "mask": lambda: tra.tra_radius_and_mask(p.handle, *d(ent, mask), mask.numel()),
}
for f in calls.values():
    f()
torch.cuda.synchronize()
assert p.status() == 0
stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
assert rt.cudaStreamCreate(ctypes.byref(stream)) == 0
for name, f in calls.items():
    assert rt.cudaStreamBeginCapture(stream, 0) == 0
    try:
        f()
        status = 0
    except tra.TraError as e:
        status = e.status
    rt.cudaStreamEndCapture(stream, ctypes.byref(graph))
    rt.cudaGetLastError()
    assert status == 4, (name, status)
    tra.tra_permute(p.handle, *d(q, tiles), 1, 2)
torch.cuda.synchronize()
assert p.status() == 0
"""


def test_a_failed_launch_leaves_no_error_for_the_next_call():
    child(FAILED_LAUNCH)
