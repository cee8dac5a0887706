"""The 8-bit cache of keys and values and the attention over it, against plain
64-bit computations: stored codes and scales bit for bit, whole frames of
queries and single tokens over any number of cached frames, both layouts and
spatial tests, empty rows, unused places, graphs, and the calls together."""
import math

import numpy as np
import pytest
import torch

import masked_reference as ref
import sparse_attention_video_tra_b200 as tra
from sparse_attention_video_tra_b200 import build as trabuild
from sparse_attention_video_tra_b200 import synth
import gpu_helpers as gh

pytestmark = pytest.mark.gpu
N_, B_, D_, Q_ = tra.TRA_FLAG_NATURAL, tra.TRA_FLAG_OUT_BF16, tra.TRA_FLAG_DISK, tra.TRA_FLAG_QSORT


@pytest.fixture(scope="module", autouse=True)
def built():
    trabuild.build()
    yield


def quantised(tile_rows):
    """[.., 128, d] -> (values of the codes, scales) in numpy float64, from the definition."""
    x = tile_rows.double().cpu().numpy()
    most = np.abs(x).max((-2, -1))
    e = np.zeros(most.shape, np.int64)
    for at in np.ndindex(most.shape):
        if most[at] > 0:
            m, k = math.frexp(most[at] / 448.0)            # 448 = 7 * 2^6: exact up to the division's rounding
            e[at] = k - 1 if m == 0.5 else k
            while most[at] > math.ldexp(448.0, int(e[at])):
                e[at] += 1
            e[at] = max(e[at], -126)
    y = np.ldexp(x, -e[..., None, None])
    # e4m3: 3 fraction bits down to 2^-6, multiples of 2^-9 below, ties to even
    with np.errstate(divide="ignore"):
        step = np.exp2(np.maximum(np.floor(np.log2(np.abs(y))), -6) - 3)
    y = np.where(y == 0, 0.0, np.round(y / np.where(y == 0, 1.0, step)) * step)
    return y, np.ldexp(1.0, e)


class Setup:
    def __init__(self, T, H, W, heads, d, gamma, Rt, flags=0, seed=5, b=0.5):
        self.grid, self.gamma, self.Rt, self.flags = (T, H, W), gamma, Rt, flags
        self.plan = tra.Plan(T, H, W, heads, d, 1.0, b, gamma, Rt, 1, flags)
        self.i = self.plan.info
        self.tpf = self.i.n_tiles_h * self.i.n_tiles_w
        self.q, self.k, self.v = synth.make_qkv(T, H, W, heads, d, seed, device="cuda", dtype=torch.bfloat16)
        self.cache = self.plan.new_cache()

    def rows(self, x, frame, n):
        """Natural [heads, N, ...] -> the call's layout for the frames [frame, frame + n)."""
        T, H, W = self.grid
        if self.plan.natural:
            return x[:, frame * H * W:(frame + n) * H * W].contiguous()
        tm = gh.to_tile_major(x, self.i)
        return tm[:, frame * self.tpf * 128:(frame + n) * self.tpf * 128].contiguous()

    def natural(self, x, frame, n):
        T, H, W = self.grid
        if self.plan.natural:
            return x
        full = torch.zeros((x.shape[0], self.i.N_pad) + tuple(x.shape[2:]), dtype=x.dtype, device=x.device)
        full[:, frame * self.tpf * 128:(frame + n) * self.tpf * 128] = x
        return gh.to_natural(full, self.i)[:, frame * H * W:(frame + n) * H * W]

    def store(self, frame=0, n=None):
        n = self.grid[0] - frame if n is None else n
        self.plan.cache_store(self.rows(self.k, frame, n), self.rows(self.v, frame, n), frame, self.cache)

    def held(self):
        """The stored K and V values in natural order, fp64."""
        out = []
        k8, v8, ks, vs = self.plan.cache_views(self.cache)
        for c, s in ((k8, ks), (v8, vs)):
            out.append(gh.to_natural((c.double() * s.double()[..., None, None]).flatten(1, 2), self.i))
        return out

    def make_mask(self):
        mask, h = self.plan.new_mask(), self.plan.new_entropy()
        tm = [x if self.plan.natural else gh.to_tile_major(x, self.i) for x in (self.q, self.k)]
        self.plan.entropy(*tm, h)
        self.plan.radius_and_mask(h, mask)
        return mask, gh.to_natural(self.plan.mask_views(mask)[0], self.i)

    def frames(self, frame, n, cached, mask, fill=7.0):
        q = self.rows(self.q, frame, n)
        out = torch.full(q.shape, fill, dtype=self.plan.out_dtype, device="cuda")
        lse = torch.full(q.shape[:2], fill, device="cuda")
        self.plan.cache_attention(q, frame, self.cache, cached, mask, out, lse, self.plan.new_cache_workspace(n))
        return self.natural(out, frame, n), self.natural(lse, frame, n)

    def tokens(self, token, radius, cached, q=None, fill=7.0):
        q = self.q[:, token.long().clamp(0, self.i.N - 1)].contiguous() if q is None else q
        out = torch.full(q.shape, fill, dtype=self.plan.out_dtype, device="cuda")
        lse = torch.full(q.shape[:2], fill, device="cuda")
        self.plan.cache_attention_tokens(q, token, radius, self.cache, cached, out, lse)
        return out, lse

    def ok(self):
        torch.cuda.synchronize()
        assert self.plan.status() == 0


GRIDS = [(1, 1, 1, 1, 64, 0.7, 0), (4, 8, 8, 2, 64, 0.7, 2), (5, 17, 23, 2, 128, 0.8, 3), (3, 33, 9, 3, 64, 0.9, 1),
         (2, 9, 50, 1, 128, 1.0, 1)]


@pytest.mark.parametrize("grid", GRIDS)
@pytest.mark.parametrize("flags", [0, N_])
def test_stored_codes_and_scales(grid, flags):
    s = Setup(*grid, flags)
    s.k[0, 0] = 0
    s.store()
    k8, v8, ks, vs = s.plan.cache_views(s.cache)
    s.ok()
    for x, c, sc in ((s.k, k8, ks), (s.v, v8, vs)):
        want, scale = quantised(gh.to_tile_major(x, s.i).view(s.i.heads, s.i.n_tiles, 128, s.i.d))
        np.testing.assert_array_equal(sc.double().cpu().numpy(), scale)
        np.testing.assert_array_equal(c.double().cpu().numpy(), want)


@pytest.mark.parametrize("most", [0.0, 448.0, 449.0, 450.0, 447.0, 1.75, 1.7578125, 2.0 ** -133, 2.0 ** -126, 1e-30, 3.38e38,
                                  57344.0, 57600.0])
def test_scales_at_their_borders(most):
    """Tiles whose largest magnitude lies at the ends of the type and on both sides of 448 * 2^e."""
    s = Setup(2, 16, 8, 1, 64, 0.7, 1, N_)
    g = torch.Generator(device="cuda").manual_seed(1)
    for x in (s.k, s.v):
        x.copy_(torch.rand(x.shape, generator=g, device="cuda") * 2 - 1)
        x.mul_(most / 2)
        x[0, 5, 3] = -most
        x[0, 130, 60] = most
    s.store()
    k8, v8, ks, vs = s.plan.cache_views(s.cache)
    s.ok()
    for x, c, sc in ((s.k, k8, ks), (s.v, v8, vs)):
        want, scale = quantised(x.view(1, 2, 128, 64))
        np.testing.assert_array_equal(sc.double().cpu().numpy(), scale)
        np.testing.assert_array_equal(c.double().cpu().numpy(), want)


@pytest.mark.parametrize("flags", [0, N_])
def test_storing_frames_leaves_the_others_and_replaces_its_own(flags):
    s = Setup(5, 17, 23, 2, 128, 0.8, 3, flags)
    s.cache.fill_(0xA5)
    before = [x.clone() for x in s.plan.cache_views(s.cache)]
    s.store(2, 2)
    after = s.plan.cache_views(s.cache)
    s.ok()
    inside = torch.zeros(s.i.n_tiles, dtype=torch.bool)
    inside[2 * s.tpf:4 * s.tpf] = True
    for x, y in zip(before, after):
        same = (x.view(torch.uint8) == y.view(torch.uint8)).flatten(2).all(2) if x.dim() > 2 else x.view(torch.int32) == y.view(torch.int32)
        assert same[:, ~inside].all() and not same[:, inside].all(1).any()
    whole = Setup(5, 17, 23, 2, 128, 0.8, 3, flags)
    whole.store()
    for f in range(5):                                   # frame by frame, one of them twice
        s.store(f, 1)
    s.store(1, 3)
    s.ok()
    for x, y in zip(s.plan.cache_views(s.cache), whole.plan.cache_views(whole.cache)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


FRAME_CASES = [
    # grid..., flags, frame, frames, cached
    ((1, 1, 1, 1, 64, 0.7, 0), 0, 0, 1, 1),
    ((4, 8, 8, 2, 64, 0.7, 2), 0, 3, 1, 4),
    ((4, 8, 8, 2, 64, 0.7, 2), N_ | B_, 0, 4, 4),
    ((5, 17, 23, 2, 128, 0.8, 3), 0, 2, 2, 3),
    ((5, 17, 23, 2, 128, 0.8, 3), N_ | B_, 4, 1, 5),
    ((5, 17, 23, 2, 128, 0.8, 3), N_ | D_, 1, 3, 2),
    ((5, 17, 23, 2, 128, 0.8, 3), D_ | B_, 0, 5, 5),
    ((5, 17, 23, 2, 64, 0.8, 1), Q_ | tra.tra_flag_tile_w(8), 1, 3, 4),
    ((5, 17, 23, 2, 128, 0.8, 1), Q_ | N_ | B_ | tra.tra_flag_tile_w(8), 2, 3, 5),
    ((5, 17, 23, 2, 128, 0.8, 1), Q_ | N_ | D_ | tra.tra_flag_tile_w(8), 3, 2, 3),
    ((3, 33, 9, 1, 64, 0.9, 1), N_ | tra.tra_flag_tile_w(4), 1, 2, 2),
    ((2, 9, 50, 1, 128, 1.0, 1), tra.tra_flag_tile_w(32), 1, 1, 2),
    ((7, 12, 11, 3, 64, 0.8, 2), N_, 5, 2, 3),           # the last query frame reaches no cached frame
    ((7, 12, 11, 3, 64, 0.8, 2), 0, 5, 2, 4),            # likewise, with pad rows
    ((7, 12, 11, 3, 64, 0.8, 2), N_ | B_, 1, 2, 0),      # nothing is cached
    ((7, 12, 11, 3, 64, 0.8, 2), 0, 6, 1, 2),            # nothing in reach
    # more query tiles than SMs
    ((5, 17, 23, 12, 128, 0.8, 2), N_ | B_, 2, 3, 4),
    ((5, 17, 23, 12, 64, 0.8, 2), 0, 1, 3, 3),
    ((5, 17, 23, 12, 128, 0.8, 2), Q_ | N_ | D_ | tra.tra_flag_tile_w(8), 1, 3, 5),
    ((6, 17, 23, 12, 64, 0.8, 1), Q_ | B_ | tra.tra_flag_tile_w(8), 3, 3, 4),
    ((7, 12, 11, 60, 64, 0.8, 2), N_, 5, 2, 3),          # and the last query frame reaches no cached frame
]


@pytest.mark.parametrize("grid,flags,frame,n,cached", FRAME_CASES)
def test_frames_over_the_cache(grid, flags, frame, n, cached):
    s = Setup(*grid, flags)
    mask, radius = s.make_mask()
    s.cache.fill_(0x7F)                                  # NaN codes and scales in the frames that are not cached
    if cached:
        s.store(0, cached)
    out, lse = s.frames(frame, n, cached, mask)
    s.ok()
    T, H, W = s.grid
    rows = slice(frame * H * W, (frame + n) * H * W)
    k, v = (x[:, :cached * H * W] for x in s.held())
    keep = ref.token_mask(T, H, W, s.gamma, s.Rt, radius[:, rows], bool(flags & D_), frame, cached)
    o, l, oe, le = ref.attention(s.q[:, rows], k, v, keep)
    ref.check(out, o, oe, "out")
    ref.check(lse, l, le, "lse")
    empty = ~keep.any(-1)
    assert not out[empty].any() and torch.isneginf(lse[empty]).all()


@pytest.mark.parametrize("flags", [0, N_, N_ | B_, D_, N_ | D_ | B_])
@pytest.mark.parametrize("grid", GRIDS + [(9, 24, 40, 2, 128, 0.8, 8)])
def test_tokens_over_the_cache(grid, flags):
    s = Setup(*grid, flags)
    T, H, W = s.grid
    g = torch.Generator(device="cuda").manual_seed(2)
    for n, cached in ((1, T), (3, max(0, T - 1)), (17, T), (2, 0), (97, T), (83, max(0, T - 1)), (70, 0)):
        s.cache.fill_(0x7F)
        if cached:
            s.store(0, cached)
        token = torch.randint(0, s.i.N, (n,), generator=g, device="cuda", dtype=torch.int32)     # any order, repeats
        radius = torch.randint(-1, max(H, W) + 2, (s.i.heads, n), generator=g, device="cuda", dtype=torch.int32)
        if n > 3:
            radius[:, 0], radius[:, 1], radius[:, 2] = 2 ** 31 - 1, 0, -5
        out, lse = s.tokens(token, radius, cached)
        s.ok()
        k, v = (x[:, :cached * H * W] for x in s.held())
        keep = ref.pairs_kept(T, H, W, s.gamma, s.Rt, token.long(), torch.arange(cached * H * W, device="cuda"), radius,
                              bool(flags & D_))
        o, l, oe, le = ref.attention(s.q[:, token.long()], k, v, keep, 0.0)
        ref.check(out, o, oe + 2.0 ** -18 * oe.new_tensor(1.0) * o.abs(), "out")
        ref.check(lse, l, le, "lse")
        empty = ~keep.any(-1)
        assert not out[empty].any() and torch.isneginf(lse[empty]).all()


@pytest.mark.parametrize("n", [5, 100])
@pytest.mark.parametrize("d", [64, 128])
def test_tokens_over_tiles_of_very_different_scales(n, d):
    """Values of frames that differ by up to 2^40, keys that reach scores of +-100, query rows from 2^-30 to 2^7."""
    s = Setup(6, 12, 11, 2, d, 0.9, 2, N_)
    g = torch.Generator(device="cuda").manual_seed(8)
    frame = torch.arange(s.i.N, device="cuda") // (12 * 11)
    s.v.mul_(torch.exp2(torch.tensor([0.0, 20.0, -20.0, 3.0, -20.0, 20.0], device="cuda"))[frame][None, :, None].bfloat16())
    s.q.mul_(torch.exp2(torch.randint(-30, 8, (2, s.i.N, 1), generator=g, device="cuda").float()).bfloat16())
    s.store()
    token = torch.randint(0, s.i.N, (n,), generator=g, device="cuda", dtype=torch.int32)
    radius = torch.randint(0, 8, (2, n), generator=g, device="cuda", dtype=torch.int32)
    out, lse = s.tokens(token, radius, 6)
    s.ok()
    keep = ref.pairs_kept(6, 12, 11, 0.9, 2, token.long(), torch.arange(s.i.N, device="cuda"), radius)
    o, l, oe, le = ref.attention(s.q[:, token.long()], *s.held(), keep, 2.0 ** -20)
    ref.check(out, o, oe, "out")
    ref.check(lse, l, le, "lse")


def test_many_tokens_and_unused_places():
    s = Setup(5, 17, 23, 2, 128, 0.8, 3, N_)
    s.store()
    n = 700
    g = torch.Generator(device="cuda").manual_seed(4)
    token = torch.randint(0, s.i.N, (n,), generator=g, device="cuda", dtype=torch.int32)
    radius = torch.randint(0, 12, (s.i.heads, n), generator=g, device="cuda", dtype=torch.int32)
    whole, whole_lse = s.tokens(token, radius, 5)
    some = token.clone()
    some[::3] = -1
    out, lse = s.tokens(some, radius, 5, s.q[:, token.long()].contiguous())
    s.ok()
    used = some >= 0
    assert torch.equal(out[:, used], whole[:, used]) and torch.equal(lse[:, used], whole_lse[:, used])
    assert (out[:, ~used] == 7).all() and (lse[:, ~used] == 7).all()
    # few tokens at a time take more CTAs each: the same up to the order of the sums
    few, few_lse = s.tokens(token[:5], radius[:, :5].contiguous(), 5)
    T, H, W = s.grid
    keep = ref.pairs_kept(T, H, W, s.gamma, s.Rt, token[:5].long(), torch.arange(s.i.N, device="cuda"), radius[:, :5])
    o, l, oe, le = ref.attention(s.q[:, token[:5].long()], *s.held(), keep, 0.0)
    ref.check(few, o, oe, "few")
    ref.check(whole[:, :5], o, oe, "whole")
    none, _ = s.tokens(token[:0], radius[:, :0].contiguous(), 5)
    assert none.numel() == 0


def test_token_outside_the_grid_is_reported_and_its_rows_left():
    s = Setup(4, 8, 8, 2, 64, 0.7, 2, N_)
    s.store()
    token = torch.tensor([3, s.i.N, 2 ** 31 - 1, 5], dtype=torch.int32, device="cuda")
    radius = torch.full((2, 4), 3, dtype=torch.int32, device="cuda")
    out, lse = s.tokens(token, radius, 4)
    torch.cuda.synchronize()
    assert s.plan.status() == 6                          # TRA_ERR_DEVICE_CHECK
    assert (out[:, 1:3] == 7).all() and (lse[:, 1:3] == 7).all()
    assert torch.isfinite(out).all() and (out[:, 0] != 7).all()
    s.tokens(token[:1], radius[:, :1].contiguous(), 4)
    s.ok()


@pytest.mark.parametrize("n", [1, 4, 5, 6, 7, 15, 16, 33])
@pytest.mark.parametrize("d,flags", [(64, N_ | D_), (128, N_)])
def test_few_tokens_of_many_heads(n, d, flags):
    """Around the number of tokens from which they are taken in groups; the last row's token is the grid's last."""
    s = Setup(4, 11, 19, 13, d, 0.85, 2, flags)
    s.store()
    g = torch.Generator(device="cuda").manual_seed(n)
    token = torch.randint(0, s.i.N, (n,), generator=g, device="cuda", dtype=torch.int32)
    token[-1] = s.i.N - 1
    radius = torch.randint(0, 20, (13, n), generator=g, device="cuda", dtype=torch.int32)
    out, lse = s.tokens(token, radius, 4)
    s.ok()
    keep = ref.pairs_kept(4, 11, 19, 0.85, 2, token.long(), torch.arange(s.i.N, device="cuda"), radius, bool(flags & D_))
    o, l, oe, le = ref.attention(s.q[:, token.long()], *s.held(), keep, 0.0)
    ref.check(out, o, oe + 2.0 ** -18 * o.abs(), "out")
    ref.check(lse, l, le, "lse")


def test_tokens_outside_the_grid_among_many_are_reported_and_their_rows_left():
    s = Setup(4, 8, 8, 2, 64, 0.7, 2, N_)
    s.store()
    g = torch.Generator(device="cuda").manual_seed(6)
    token = torch.randint(0, s.i.N, (50,), generator=g, device="cuda", dtype=torch.int32)
    radius = torch.full((2, 50), 3, dtype=torch.int32, device="cuda")
    whole, whole_lse = s.tokens(token, radius, 4)
    s.ok()
    bad = token.clone()
    bad[0], bad[17], bad[49] = s.i.N, 2 ** 31 - 1, -2 ** 31
    out, lse = s.tokens(bad, radius, 4, s.q[:, token.long()].contiguous())
    torch.cuda.synchronize()
    assert s.plan.status() == 6                          # TRA_ERR_DEVICE_CHECK
    left = torch.zeros(50, dtype=torch.bool, device="cuda")
    left[[0, 17, 49]] = True
    assert (out[:, left] == 7).all() and (lse[:, left] == 7).all()
    assert torch.equal(out[:, ~left], whole[:, ~left]) and torch.equal(lse[:, ~left], whole_lse[:, ~left])
    s.ok()


@pytest.mark.parametrize("flags", [0, N_ | B_, N_ | D_])
def test_generating_a_clip_frame_by_frame(flags):
    """Store, then attend, one frame after the other; single tokens agree with the frame's rows, and the parts of a
    row over two sets of frames, merged by their log-sum-exps, with the row over both."""
    s = Setup(6, 13, 21, 2, 64, 0.8, 2, flags)
    mask, radius = s.make_mask()
    T, H, W = s.grid
    for t in range(T):
        s.store(t, 1)
        out, lse = s.frames(t, 1, t + 1, mask)
        token = torch.arange(t * H * W, t * H * W + W, device="cuda", dtype=torch.int32)
        tout, tlse = s.tokens(token, radius[:, token.long()].contiguous(), t + 1)
        s.ok()
        rows = slice(t * H * W, (t + 1) * H * W)
        k, v = (x[:, :(t + 1) * H * W] for x in s.held())
        keep = ref.token_mask(T, H, W, s.gamma, s.Rt, radius[:, rows], bool(flags & D_), t, t + 1)
        o, l, oe, le = ref.attention(s.q[:, rows], k, v, keep)
        ref.check(out, o, oe, "frame")
        ref.check(lse, l, le, "frame lse")
        ref.check(tout, o[:, :W], oe[:, :W], "tokens")
        ref.check(tlse, l[:, :W], le[:, :W], "tokens lse")
        # the frame's own keys apart from the earlier ones
        earlier, elarge = s.frames(t, 1, t, mask)
        own = keep.clone()
        own[..., :t * H * W] = False
        oo, ol, ooe, ole = ref.attention(s.q[:, rows], k, v, own)
        both = torch.logaddexp(elarge.double(), ol)
        merged = earlier.double() * torch.exp(elarge.double() - both)[..., None] + oo * torch.exp(ol - both)[..., None]
        step = ref.BF16 if out.dtype == torch.bfloat16 else ref.FP32
        ref.check(merged, o, oe + ooe + (step + 2 * (le + ole))[..., None] * (o.abs() + oo.abs() + earlier.double().abs()) if step == ref.FP32
                  else oe + ooe + step * (o.abs() + oo.abs() + earlier.double().abs()) + 2 * (le + ole)[..., None] * (oo.abs() + earlier.double().abs()), "merged")
        ref.check(both, l, le + ole, "merged lse")


def test_offsets_past_32_bits():
    """The last heads of a cache of 4.5 GB of keys and as much of values: frames, lone tokens and grouped ones."""
    T, H, W, heads, d = 21, 45, 80, 440, 128
    plan = tra.Plan(T, H, W, heads, d, 1.0, -30.0, 0.8, 0, 1, N_ | B_)          # a budget of one token, no temporal reach
    assert tra.tra_cache_query(plan.handle).off_v > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(6)
    k, v, q = (torch.randn(heads, H * W, d, generator=g, device="cuda").bfloat16() for _ in range(3))
    cache = plan.new_cache()
    plan.cache_store(k, v, 20, cache)
    k8, v8, ks, vs = plan.cache_views(cache)
    tpf = plan.info.n_tiles_h * plan.info.n_tiles_w
    held = []
    for c, s in ((k8, ks), (v8, vs)):
        one = tra.Plan(1, H, W, 1, d, 1.0, 0.0, 0.8, 0, 1, N_)
        held.append(gh.to_natural((c[-1:, 20 * tpf:].double() * s[-1:, 20 * tpf:].double()[..., None, None]).flatten(1, 2), one.info))
    for n in (1, 16):
        token = 20 * H * W + torch.randint(0, H * W, (n,), generator=g, device="cuda", dtype=torch.int32)
        radius = torch.full((heads, n), 3, dtype=torch.int32, device="cuda")
        qt = q[:, (token - 20 * H * W).long()].contiguous()
        out, lse = torch.empty_like(qt), torch.empty(heads, n, device="cuda")
        plan.cache_attention_tokens(qt, token, radius, cache, 21, out, lse)
        keep = ref.pairs_kept(1, H, W, 0.8, 0, (token - 20 * H * W).long(), torch.arange(H * W, device="cuda"), radius[-1:])
        o, l, oe, le = ref.attention(qt[-1:], *held, keep, 0.0)
        ref.check(out[-1:], o, oe, "out")
        ref.check(lse[-1:], l, le, "lse")
    mask = plan.new_mask()
    plan.radius_and_mask(torch.zeros(heads, T * H * W, device="cuda"), mask)
    out, lse = torch.empty_like(q), torch.empty(heads, H * W, device="cuda")
    plan.cache_attention(q, 20, cache, 21, mask, out, lse, plan.new_cache_workspace(1))
    torch.cuda.synchronize()
    assert plan.status() == 0
    # each query keeps itself alone
    ref.check(out[-1:], held[1], held[1].abs() * ref.BF16, "frame")


def test_two_calls_at_once_on_two_streams():
    """Frames and tokens of two clips on two streams, each with its own workspace, equal the calls one after the other."""
    a, b = (Setup(5, 17, 23, 2, 128, 0.8, 3, N_ | B_, seed=s) for s in (1, 2))
    masks = [x.make_mask()[0] for x in (a, b)]
    for x in (a, b):
        x.store()
    want = [x.frames(2, 3, 5, m) for x, m in zip((a, b), masks)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for x, m, st in zip((a, b), masks, streams):
        with torch.cuda.stream(st):
            got.append([x.frames(2, 3, 5, m) for _ in range(5)])
    a.ok()
    for w, g5 in zip(want, got):
        for o, l in g5:
            assert torch.equal(o, w[0]) and torch.equal(l, w[1])


def test_graphs_and_streams():
    s = Setup(5, 17, 23, 2, 128, 0.8, 3, N_ | B_)
    mask, radius = s.make_mask()
    token = torch.arange(4 * 17 * 23, 4 * 17 * 23 + 9, device="cuda", dtype=torch.int32)
    tr = radius[:, token.long()].contiguous()
    kn, vn, q = s.rows(s.k, 4, 1), s.rows(s.v, 4, 1), s.rows(s.q, 4, 1)
    qt = s.q[:, token.long()].contiguous()
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    tout, tlse = torch.empty_like(qt), torch.empty(qt.shape[:2], device="cuda")
    ws = s.plan.new_cache_workspace(1)
    s.store()

    def step(stream=None):
        s.plan.cache_store(kn, vn, 4, s.cache, stream)
        s.plan.cache_attention(q, 4, s.cache, 5, mask, out, lse, ws, stream)
        s.plan.cache_attention_tokens(qt, token, tr, s.cache, 5, tout, tlse, stream)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    step(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g = torch.Generator(device="cuda").manual_seed(9)
    for x in (kn, vn, q, qt):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
    token.add_(30)
    graph.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in (out, lse, tout, tlse)]
    step()
    s.ok()
    for x, y in zip(got, (out, lse, tout, tlse)):
        assert torch.equal(x, y)
    graph.reset()


def test_refusals():
    s = Setup(4, 8, 8, 2, 64, 0.7, 2, N_)
    mask, radius = s.make_mask()
    s.store()
    q = s.rows(s.q, 1, 1)
    out, lse = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:2], device="cuda")
    ws = s.plan.new_cache_workspace(1)

    def status(call):
        with pytest.raises(tra.TraError) as e:
            call()
        return e.value.status

    P = s.plan
    assert status(lambda: P.cache_store(q, q, 4, s.cache)) == 1                    # frame outside the grid
    assert status(lambda: P.cache_store(q, q, -1, s.cache)) == 1
    assert status(lambda: P.cache_store(q, q, 0, s.cache[:-256])) == 3
    assert status(lambda: P.cache_attention(q, 4, s.cache, 4, mask, out, lse, ws)) == 1
    assert status(lambda: P.cache_attention(q, 1, s.cache, 5, mask, out, lse, ws)) == 1
    assert status(lambda: P.cache_attention(q, 1, s.cache, 4, mask, out, lse, ws[:-256])) == 3
    assert status(lambda: P.cache_attention(q, 1, s.cache[:-256], 4, mask, out, lse, ws)) == 3
    token = torch.zeros(3, dtype=torch.int32, device="cuda")
    qt = s.q[:, :3].contiguous()
    ot, lt = torch.empty(qt.shape, device="cuda"), torch.empty(qt.shape[:2], device="cuda")
    rad = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    assert status(lambda: P.cache_attention_tokens(qt, token, rad, s.cache, -1, ot, lt)) == 1
    assert status(lambda: P.cache_attention_tokens(qt, token, rad, s.cache[:-256], 4, ot, lt)) == 3
    for call in (lambda: P.cache_store(q[:, :-1].contiguous(), q, 0, s.cache),
                 lambda: P.cache_store(q, q.float(), 0, s.cache),
                 lambda: P.cache_store(q, s.rows(s.q, 0, 2), 0, s.cache),
                 lambda: P.cache_attention(q, 1, s.cache, 4, mask, out.bfloat16(), lse, ws),
                 lambda: P.cache_attention(q, 1, s.cache, 4, mask[:-1], out, lse, ws),
                 lambda: P.cache_attention_tokens(qt, token.long(), rad, s.cache, 4, ot, lt),
                 lambda: P.cache_attention_tokens(qt, token, rad[:, :2].contiguous(), s.cache, 4, ot, lt),
                 lambda: P.cache_attention_tokens(qt.cpu(), token, rad, s.cache, 4, ot, lt)):
        with pytest.raises(ValueError):
            call()
    s.ok()


def wide_scale_tokens(change, n, d=128, heads=12, q=None):
    """n neighbouring tokens of frame 6 over 13 cached 30x52 frames, k and v as `change` makes them: (setup, tokens,
    their queries, the kept pairs, out, lse).  A warp of the grouped form walks dozens of granules there."""
    s = Setup(13, 30, 52, heads, d, 0.9, 6, N_)
    change(s)
    s.store()
    g = torch.Generator(device="cuda").manual_seed(n)
    token = 6 * 30 * 52 + 400 + torch.arange(n, device="cuda", dtype=torch.int32)
    radius = torch.randint(6, 20, (heads, n), generator=g, device="cuda", dtype=torch.int32)
    q = s.q[:, token.long()].contiguous() if q is None else q(s.q[:, token.long()].contiguous())
    out, lse = s.tokens(token, radius, 13, q)
    s.ok()
    keep = ref.pairs_kept(13, 30, 52, 0.9, 6, token.long(), torch.arange(s.i.N, device="cuda"), radius)
    return s, q, keep, out, lse


def frame_of(s):
    return torch.arange(s.i.N, device="cuda") // (30 * 52)


@pytest.mark.parametrize("n,d", [(5, 128), (6, 128), (8, 128), (52, 128), (16, 64)])
@pytest.mark.parametrize("bits", [-6, -10, -13, -17])
def test_tokens_over_a_frame_of_zero_values(n, d, bits):
    """Tiles of zeros have the scale 2^0: they must not cost the small values of the other frames their bits."""
    def change(s):
        s.v.mul_(2.0 ** bits)
        s.v[:, frame_of(s) == 0] = 0
    s, q, keep, out, lse = wide_scale_tokens(change, n, d)
    o, l, oe, le = ref.attention(q, *s.held(), keep, 2.0 ** -20)
    ref.check(out, o, oe, "out")
    ref.check(lse, l, le, "lse")


@pytest.mark.parametrize("n,d", [(5, 128), (6, 128), (8, 128), (52, 128), (16, 64)])
@pytest.mark.parametrize("bits", [16, 20])
def test_tokens_over_a_frame_of_large_values_at_low_scores(n, d, bits):
    """One frame's values are 2^bits larger and its scores 30 bits lower: its weights do not set the others' accuracy."""
    def change(s):
        at = frame_of(s) == 1
        s.k[..., 0] = 0
        s.k[:, at, 0] = -30 * math.log(2) * math.sqrt(d) / 8
        s.v[:, at] *= 2.0 ** bits

    def query(q):
        q[..., 0] = 8
        return q
    s, q, keep, out, lse = wide_scale_tokens(change, n, d, q=query)
    o, l, oe, le = ref.attention(q, *s.held(), keep, 2.0 ** -20)
    ref.check(out, o, oe, "out")
    ref.check(lse, l, le, "lse")


@pytest.mark.parametrize("n,d", [(5, 128), (6, 128), (8, 128), (52, 128), (16, 64)])
@pytest.mark.parametrize("large", [0, 12])
def test_tokens_over_an_outlier_channel_of_one_frame(n, d, large):
    """The large frame, first or last, fills one channel only: the other channels come from the small frames and carry
    a bound of their own size."""
    def change(s):
        at = frame_of(s) == large
        s.v[:, at, 1:] = 0
        s.v[:, at, 0] *= 2.0 ** 20
        s.v[:, ~at, 0] = 0
    s, q, keep, out, lse = wide_scale_tokens(change, n, d)
    o, l, oe, le = ref.attention(q, *s.held(), keep, 2.0 ** -20)
    ref.check(out, o, oe, "out")
    ref.check(lse, l, le, "lse")


@pytest.mark.parametrize("n,d", [(5, 128), (6, 128), (8, 128), (52, 128), (16, 64)])
@pytest.mark.parametrize("bits", [20, 34, 40, 90])
def test_tokens_whose_queries_have_an_outlier(n, d, bits):
    """One element of each query is 2^bits where the keys are zeros: the scores come from the others, in full."""
    def change(s):
        s.k[..., 0] = 0

    def query(q):
        q[..., 0] = 2.0 ** bits
        return q
    s, q, keep, out, lse = wide_scale_tokens(change, n, d, q=query)
    o, l, oe, le = ref.attention(q, *s.held(), keep, 2.0 ** -20)
    ref.check(out, o, oe, "out")
    ref.check(lse, l, le, "lse")


@pytest.mark.parametrize("n", [5, 40])
def test_tokens_with_large_queries_over_large_keys_that_do_not_meet(n):
    """Queries of 2^90 in one element, keys of 2^60 in another one: every score is zero, every output the mean value."""
    def change(s):
        s.k.zero_()
        s.k[..., 1] = 2.0 ** 60

    def query(q):
        q.zero_()
        q[..., 0] = 2.0 ** 90
        return q
    s, q, keep, out, lse = wide_scale_tokens(change, n, q=query)
    o, l, oe, le = ref.attention(q, *s.held(), keep, 2.0 ** -20)
    ref.check(out, o, oe, "out")
    ref.check(lse, l, le, "lse")


@pytest.mark.parametrize("heads,n", [(13, 8), (13, 7), (12, 8), (11, 8), (11, 9), (2, 47), (2, 48), (1, 95), (1, 96)])
@pytest.mark.parametrize("d,flags", [(64, N_), (128, N_ | D_ | B_)])
def test_tokens_on_both_sides_of_grouping(heads, n, d, flags):
    """8 tokens and 96 (token, head) pairs, one less of either, scattered over the clip."""
    s = Setup(4, 11, 19, heads, d, 0.85, 2, flags)
    s.store()
    g = torch.Generator(device="cuda").manual_seed(n)
    token = torch.randint(0, s.i.N, (n,), generator=g, device="cuda", dtype=torch.int32)
    radius = torch.randint(-1, 20, (heads, n), generator=g, device="cuda", dtype=torch.int32)
    out, lse = s.tokens(token, radius, 4)
    s.ok()
    keep = ref.pairs_kept(4, 11, 19, 0.85, 2, token.long(), torch.arange(s.i.N, device="cuda"), radius, bool(flags & D_))
    o, l, oe, le = ref.attention(s.q[:, token.long()], *s.held(), keep, 2.0 ** -20)
    ref.check(out, o, oe, "out")
    ref.check(lse, l, le, "lse")


@pytest.mark.parametrize("n,d", [(5, 128), (8, 128), (52, 128), (16, 64)])
@pytest.mark.parametrize("bits", [-100, -110, -116, 100, 116])
def test_tokens_over_the_smallest_and_largest_values(n, d, bits):
    """Values near the ends of the type's exponents keep as many bits as ordinary ones (compared after a power of two)."""
    def change(s):
        s.v.mul_(2.0 ** bits)
    s, q, keep, out, lse = wide_scale_tokens(change, n, d)
    k, v = s.held()
    o, l, oe, le = ref.attention(q, k, v * 2.0 ** -bits, keep, 2.0 ** -20)
    assert out.dtype == torch.float32
    ref.check(out * 2.0 ** -bits, o, oe, "out")
    ref.check(lse, l, le, "lse")
