"""CPU checks of the training and cache calls of the C ABI: sizes, layouts and
every refusal that is decided before a CUDA call (pointers are numbers here,
never followed)."""
import ctypes

import pytest

import sparse_attention_video_tra_b200 as tra
from sparse_attention_video_tra_b200 import build as trabuild

P = 4096                                                 # an aligned address that no call gets to read


@pytest.fixture(scope="module", autouse=True)
def built():
    trabuild.build()
    yield


def plan(flags=0, T=5, H=17, W=23, heads=2, d=128, Rt=3):
    return tra.Plan(T, H, W, heads, d, 1.0, 0.0, 0.8, Rt, 1, flags)


@pytest.mark.parametrize("flags,copies", [
    (0, 1), (tra.TRA_FLAG_NATURAL, 4), (tra.TRA_FLAG_NATURAL | tra.TRA_FLAG_OUT_BF16, 4), (tra.TRA_FLAG_OUT_BF16, 1),
    (tra.TRA_FLAG_QSORT | tra.tra_flag_tile_w(8), 2),
    (tra.TRA_FLAG_QSORT | tra.tra_flag_tile_w(8) | tra.TRA_FLAG_NATURAL | tra.TRA_FLAG_OUT_BF16, 4)])
def test_backward_workspace_holds_its_parts(flags, copies):
    p = plan(flags)
    i = p.info
    words = (i.list_cap + 31) // 32
    parts = 16 * i.heads * i.N_pad + 4 * i.heads * i.n_tiles * words + copies * i.heads * i.N_pad * i.d * 2
    got = tra.tra_attention_backward_bytes(p.handle)
    assert parts <= got <= parts + 6 * 256 and got % 256 == 0


@pytest.mark.parametrize("shape", [dict(), dict(T=1, H=1, W=1, heads=1, d=64, Rt=0), dict(T=21, H=45, W=80, heads=40, Rt=6)])
def test_cache_layout(shape):
    p = plan(**shape)
    i, c = p.info, tra.tra_cache_query(p.handle)
    codes, scales = i.heads * i.N_pad * i.d, 4 * i.heads * i.n_tiles
    offs = [c.off_k, c.off_v, c.off_k_scale, c.off_v_scale, c.cache_bytes]
    assert all(o % 256 == 0 for o in offs)
    for k, size in enumerate((codes, codes, scales, scales)):
        assert offs[k] + size <= offs[k + 1] < offs[k] + size + 256
    # half of K and V in bf16, but for the scales
    assert c.cache_bytes < 2 * codes * 1.001 + 2 * scales + 1024


def test_cache_workspace_is_the_largest_window():
    p = plan(T=21, H=45, W=80, heads=3, Rt=6)
    i = p.info
    tpf = i.n_tiles_h * i.n_tiles_w
    for n, window in ((1, 13), (4, 16), (9, 21), (21, 21)):
        assert tra.tra_cache_attention_bytes(p.handle, n) == 2 * i.heads * window * tpf * 128 * i.d * 2
    for n in (0, -1, 22):
        with pytest.raises(tra.TraError) as e:
            tra.tra_cache_attention_bytes(p.handle, n)
        assert e.value.status == 1


def refused(func, args, status, **change):
    """func(*args) with one argument changed returns the status."""
    names = list(args)
    vals = dict(args)
    vals.update(change)
    with pytest.raises(tra.TraError) as e:
        func(*[vals[n] for n in names])
    assert e.value.status == status, change


def test_lse_and_backward_refusals():
    p = plan()
    big = 1 << 40
    fwd = dict(plan=p.handle, q=P, k=P, v=P, mask=P, out=P, lse=P)
    for n in ("plan", "q", "k", "v", "mask", "out", "lse"):
        refused(tra.tra_attention_lse, fwd, 1, **{n: None})
    for n, off in (("q", 8), ("k", 2), ("v", 4), ("mask", 128), ("out", 8), ("lse", 2)):
        refused(tra.tra_attention_lse, fwd, 1, **{n: P + off})
    bwd = dict(plan=p.handle, q=P, k=P, v=P, mask=P, out=P, lse=P, dout=P, dq=P, dk=P, dv=P, ws=P, bytes=big)
    for n in ("plan", "q", "k", "v", "mask", "out", "lse", "dout", "dq", "dk", "dv", "ws"):
        refused(tra.tra_attention_backward, bwd, 1, **{n: None})
    for n, off in (("q", 8), ("k", 2), ("v", 4), ("mask", 128), ("out", 8), ("lse", 2), ("dout", 8), ("dq", 4), ("dk", 8),
                   ("dv", 12), ("ws", 128)):
        refused(tra.tra_attention_backward, bwd, 1, **{n: P + off})
    refused(tra.tra_attention_backward, bwd, 3, bytes=tra.tra_attention_backward_bytes(p.handle) - 1)
    lib = tra.load_library()
    assert lib.tra_attention_backward_bytes(None, ctypes.byref(ctypes.c_size_t())) == 1
    assert lib.tra_attention_backward_bytes(p.handle, None) == 1


def test_cache_refusals():
    p = plan()
    need, work = tra.tra_cache_query(p.handle).cache_bytes, tra.tra_cache_attention_bytes(p.handle, 2)
    store = dict(plan=p.handle, k=P, v=P, frame=0, n=1, cache=P, bytes=need)
    for n in ("plan", "k", "v", "cache"):
        refused(tra.tra_cache_store, store, 1, **{n: None})
    for change in (dict(k=P + 8), dict(v=P + 2), dict(cache=P + 64), dict(frame=-1), dict(frame=5), dict(n=0), dict(n=6),
                   dict(frame=4, n=2), dict(frame=2 ** 31 - 1), dict(frame=1, n=2 ** 31 - 1), dict(n=-3)):
        refused(tra.tra_cache_store, store, 1, **change)
    refused(tra.tra_cache_store, store, 3, bytes=need - 1)

    att = dict(plan=p.handle, q=P, frame=1, n=2, cache=P, bytes=need, cached=5, mask=P, out=P, lse=P, ws=P, ws_bytes=work)
    for n in ("plan", "q", "cache", "mask", "out", "lse", "ws"):
        refused(tra.tra_cache_attention, att, 1, **{n: None})
    for change in (dict(q=P + 8), dict(cache=P + 128), dict(mask=P + 16), dict(out=P + 4), dict(lse=P + 1), dict(ws=P + 128),
                   dict(frame=4), dict(frame=-1), dict(n=0), dict(cached=-1), dict(cached=6)):
        refused(tra.tra_cache_attention, att, 1, **change)
    refused(tra.tra_cache_attention, att, 3, bytes=need - 1)
    refused(tra.tra_cache_attention, att, 3, ws_bytes=work - 256)

    tok = dict(plan=p.handle, q=P, token=P, radius=P, n=3, cache=P, bytes=need, cached=5, out=P, lse=P)
    for n in ("plan", "q", "token", "radius", "cache", "out", "lse"):
        refused(tra.tra_cache_attention_tokens, tok, 1, **{n: None})
    for change in (dict(q=P + 8), dict(token=P + 2), dict(radius=P + 1), dict(cache=P + 128), dict(out=P + 8), dict(lse=P + 2),
                   dict(n=-1), dict(cached=-1), dict(cached=6)):
        refused(tra.tra_cache_attention_tokens, tok, 1, **change)
    refused(tra.tra_cache_attention_tokens, tok, 3, bytes=need - 1)
    refused(tra.tra_cache_attention_tokens, tok, 2, n=2 ** 31 - 1)
    # no tokens: nothing to do, nothing needed
    tra.tra_cache_attention_tokens(p.handle, None, None, None, 0, None, 0, 5, None, None)
    lib = tra.load_library()
    assert lib.tra_cache_query(None, None) == 1 and lib.tra_cache_query(p.handle, None) == 1
