"""The training and cache calls at the ends of what a plan allows: frames of
256 x 256 tokens (coordinates of 255, more than a thousand key tiles in a list),
32767 tiles of one token, and corrupted mask buffers in every form of the
forward kernel.  Rows and columns are sampled and compared with the 64-bit
formulas over all keys or queries."""
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


class Case:
    """A plan, natural inputs and a mask whose budgets spread evenly over the orders of magnitude."""

    def __init__(self, T, H, W, heads, d, gamma, Rt, flags=0, seed=3):
        self.grid, self.gamma, self.Rt, self.flags = (T, H, W), gamma, Rt, flags
        self.plan = tra.Plan(T, H, W, heads, d, 1.0, 0.0, gamma, Rt, 1, flags)
        self.i = self.plan.info
        self.nat = synth.make_qkv(T, H, W, heads, d, seed, device="cuda", dtype=torch.bfloat16)
        g = torch.Generator(device="cuda").manual_seed(seed)
        h = torch.rand(heads, T * H * W, generator=g, device="cuda") * 1.1 * float(torch.log(torch.tensor(float(T * H * W))))
        self.mask = self.plan.new_mask()
        self.plan.radius_and_mask(self.layout(h), self.mask)
        self.radius = gh.to_natural(self.plan.mask_views(self.mask)[0], self.i)

    def layout(self, x):
        return x.contiguous() if self.plan.natural else gh.to_tile_major(x, self.i)

    def natural(self, x):
        return x if self.plan.natural else gh.to_natural(x, self.i)

    def keep(self, n, m, radius=None):
        r = self.radius[:, n] if radius is None else radius
        return ref.pairs_kept(*self.grid, self.gamma, self.Rt, n, m, r, bool(self.flags & D_))

    def ok(self):
        torch.cuda.synchronize()
        assert self.plan.status() == 0


def check_step(c, rows):
    """lse, out and dq of the sampled rows, dk and dv of the same tokens as keys."""
    q, k, v = (c.layout(x) for x in c.nat)
    p = c.plan
    out, lse = p.new_out(), p.new_lse()
    p.attention_lse(q, k, v, c.mask, out, lse)
    g = torch.Generator(device="cuda").manual_seed(7)
    dout = torch.randn(c.nat[0].shape, generator=g, device="cuda").to(p.out_dtype)
    grads = [p.new_out() for _ in range(3)]
    p.attention_backward(q, k, v, c.mask, out, lse, c.layout(dout), *grads, p.new_backward_workspace())
    c.ok()
    every = torch.arange(c.i.N, device="cuda")
    out, lse, grads = c.natural(out), c.natural(lse), [c.natural(x) for x in grads]
    o, l, oe, le = ref.attention(c.nat[0][:, rows], *c.nat[1:], c.keep(rows, every))
    ref.check(out[:, rows], o, oe, "out")
    ref.check(lse[:, rows], l, le, "lse")
    do = dout.bfloat16()
    (dq, _, _), (bq, _, _) = ref.gradients(c.nat[0][:, rows], *c.nat[1:], out[:, rows], lse[:, rows], do[:, rows],
                                           c.keep(rows, every))
    ref.check(grads[0][:, rows], dq, bq, "dq")
    (_, dk, dv), (_, bk, bv) = ref.gradients(c.nat[0], c.nat[1][:, rows], c.nat[2][:, rows], out, lse, do, c.keep(every, rows))
    ref.check(grads[1][:, rows], dk, bk, "dk")
    ref.check(grads[2][:, rows], dv, bv, "dv")


def held(c, cache):
    k8, v8, ks, vs = c.plan.cache_views(cache)
    return [gh.to_natural((x.double() * s.double()[..., None, None]).flatten(1, 2), c.i) for x, s in ((k8, ks), (v8, vs))]


def corners(T, H, W, extra, seed=1):
    """Tokens at the corners of the first, a middle and the last frame, and some others."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    at = [(t * H + h) * W + w for t in sorted({0, T // 2, T - 1}) for h in sorted({0, H - 1}) for w in sorted({0, W - 1})]
    return torch.cat([torch.tensor(at, device="cuda"), torch.randint(0, T * H * W, (extra,), generator=g, device="cuda")])


@pytest.mark.parametrize("d,flags", [(64, N_ | B_), (128, D_), (128, N_ | D_ | B_ | tra.tra_flag_tile_w(32))])
def test_a_training_step_on_frames_of_256_by_256(d, flags):
    c = Case(3, 256, 256, 1, d, 1.0, 1, flags)
    assert c.i.list_cap == 1536 and int(c.plan.mask_views(c.mask)[1].max()) > 1024
    check_step(c, corners(3, 256, 256, 20))


@pytest.mark.parametrize("d,flags", [(64, N_), (128, D_ | B_)])
def test_the_cache_on_frames_of_256_by_256(d, flags):
    c = Case(3, 256, 256, 1, d, 1.0, 1, flags)
    cache = c.plan.new_cache()
    cache.fill_(0x7F)
    area = 256 * 256
    tpf = c.i.n_tiles // 3
    q, k, v = (c.layout(x) for x in c.nat)
    per = area if c.plan.natural else tpf * 128
    c.plan.cache_store(k[:, :2 * per].contiguous(), v[:, :2 * per].contiguous(), 0, cache)
    kv = [x[:, :2 * area] for x in held(c, cache)]
    keys = torch.arange(2 * area, device="cuda")
    # whole frames: the middle one and the one behind the cached ones
    qf = q[:, per:].contiguous()
    out, lse = torch.empty(qf.shape, dtype=c.plan.out_dtype, device="cuda"), torch.empty(qf.shape[:2], device="cuda")
    c.plan.cache_attention(qf, 1, cache, 2, c.mask, out, lse, c.plan.new_cache_workspace(2))
    c.ok()
    rows = corners(3, 256, 256, 20)
    rows = rows[rows >= area]
    at = rows - area
    if not c.plan.natural:
        tile_row = torch.empty(c.i.N, dtype=torch.int64, device="cuda")
        nat = torch.from_numpy(gh.tile_major_index(c.i)).cuda()
        tile_row[nat[nat >= 0]] = torch.arange(c.i.N_pad, device="cuda")[nat >= 0]
        at = tile_row[rows] - per
    o, l, oe, le = ref.attention(c.nat[0][:, rows], *kv, c.keep(rows, keys))
    ref.check(out[:, at], o, oe, "frames")
    ref.check(lse[:, at], l, le, "frames lse")
    # tokens, one at a time and grouped
    for n, token in ((4, corners(3, 256, 256, 0)[4:8]), (120, corners(3, 256, 256, 108))):
        token = token.int()
        radius = torch.randint(200, 260, (1, n), device="cuda", dtype=torch.int32, generator=torch.Generator(device="cuda").manual_seed(n))
        qt = c.nat[0][:, token.long()].contiguous()
        to, tl = torch.empty(qt.shape, dtype=c.plan.out_dtype, device="cuda"), torch.empty(qt.shape[:2], device="cuda")
        c.plan.cache_attention_tokens(qt, token, radius, cache, 2, to, tl)
        c.ok()
        o, l, oe, le = ref.attention(qt, *kv, c.keep(token.long(), keys, radius), 2.0 ** -20)
        ref.check(to, o, oe, f"{n} tokens")
        ref.check(tl, l, le, f"{n} tokens lse")


@pytest.mark.parametrize("flags", [N_ | B_, N_ | D_])
def test_the_largest_number_of_tiles(flags):
    """32767 frames of one token: tile numbers of 15 bits in every list, with the longest temporal reach."""
    c = Case(32767, 1, 1, 1, 64, 0.9, 31, flags)
    assert c.i.n_tiles == 32767 and c.i.list_cap == 63
    rows = corners(32767, 1, 1, 30)
    check_step(c, rows)
    cache = c.plan.new_cache()
    c.plan.cache_store(c.nat[1], c.nat[2], 0, cache)
    kv = held(c, cache)
    every = torch.arange(32767, device="cuda")
    last = every[-40:]
    qf = c.nat[0][:, last].contiguous()
    out, lse = torch.empty(qf.shape, dtype=c.plan.out_dtype, device="cuda"), torch.empty(qf.shape[:2], device="cuda")
    c.plan.cache_attention(qf, 32767 - 40, cache, 32767, c.mask, out, lse, c.plan.new_cache_workspace(40))
    for n in (3, 120):
        token = corners(32767, 1, 1, n - 3).int()
        radius = torch.randint(-1, 3, (1, n), device="cuda", dtype=torch.int32, generator=torch.Generator(device="cuda").manual_seed(n))
        qt = c.nat[0][:, token.long()].contiguous()
        to, tl = torch.empty(qt.shape, dtype=c.plan.out_dtype, device="cuda"), torch.empty(qt.shape[:2], device="cuda")
        c.plan.cache_attention_tokens(qt, token, radius, cache, 32767, to, tl)
        c.ok()
        o, l, oe, le = ref.attention(qt, *kv, c.keep(token.long(), every, radius), 2.0 ** -20)
        ref.check(to, o, oe, f"{n} tokens")
        ref.check(tl, l, le, f"{n} tokens lse")
    o, l, oe, le = ref.attention(qf, *kv, c.keep(last, every))
    ref.check(out, o, oe, "frames")
    ref.check(lse, l, le, "frames lse")


SPOILT = ["count", "list", "reach", "group"]


def spoil(c, mask, what):
    """Mistakes in the first and the last list of the last head, and in a group."""
    _, count, _, lists = c.plan.mask_views(mask)
    if what == "count":
        count[-1, 0], count[-1, -1] = c.i.list_cap + 5, -1
    elif what == "list":
        lists[-1, 0, 0], lists[-1, -1, 0] = 0x7FFE, 0x7FFF
    elif what == "reach":                                # a tile of the grid, too many frames away
        lists[-1, 0, 0], lists[-1, -1, 0] = c.i.n_tiles - 1, 0
    else:
        c.plan.group_view(mask)[-1, 0, 5] = 128 * c.i.n_tiles_h
        c.plan.group_view(mask)[-1, -1, 127] = 0x7FFF


@pytest.mark.parametrize("grid", [(5, 8, 8, 2, 64, 0.7, 1), (9, 24, 10, 1, 64, 0.9, 6), (5, 17, 23, 2, 128, 0.8, 3),
                                  (5, 17, 23, 8, 128, 0.8, 3)])
@pytest.mark.parametrize("flags", [N_ | B_, Q_ | tra.tra_flag_tile_w(8), N_ | D_ | Q_ | tra.tra_flag_tile_w(8)])
def test_corrupted_masks_in_every_form_of_the_forward(grid, flags):
    """One chain, clusters of CTAs per tile and pairs of tiles: a mistake in the mask is reported and not followed, heads
    without one keep their results, nothing is written past the outputs, and the next call is whole again."""
    c = Case(*grid, flags)
    q, k, v = (c.layout(x) for x in c.nat)
    T, heads, d = grid[0], grid[3], grid[4]
    n = c.plan.io_rows
    store = torch.empty(heads + 1, n, d, dtype=c.plan.out_dtype, device="cuda")
    lstore = torch.empty(heads + 1, n, device="cuda")
    cache, ws = c.plan.new_cache(), c.plan.new_cache_workspace(T)
    c.plan.cache_store(k, v, 0, cache)

    def run(call, mask):
        store.fill_(7)
        lstore.fill_(7)
        call(mask, store[:heads], lstore[:heads])
        torch.cuda.synchronize()
        assert (store[heads] == 7).all() and (lstore[heads] == 7).all()
        return store[:heads].clone(), lstore[:heads].clone()

    def lse_call(mask, out, lse):
        c.plan.attention_lse(q, k, v, mask, out, lse)

    def frames_call(mask, out, lse):
        c.plan.cache_attention(q, 0, cache, T, mask, out, lse, ws)

    for call in (lse_call, frames_call):
        want = run(call, c.mask)
        assert c.plan.status() == 0
        for what in SPOILT[:4 if flags & Q_ else 3]:
            bad = c.mask.clone()
            spoil(c, bad, what)
            got = run(call, bad)
            assert c.plan.status() == 6, what            # TRA_ERR_DEVICE_CHECK
            for x, y in zip(want, got):
                assert torch.equal(x[:-1], y[:-1])
            again = run(call, c.mask)
            assert c.plan.status() == 0
            for x, y in zip(want, again):
                assert torch.equal(x, y)


def same_but_nan(got, want, bad):
    """NaN in the rows of `bad`, the bits of want elsewhere."""
    assert torch.isnan(got[bad]).all()
    assert torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("grid", [(5, 8, 8, 2, 64, 0.7, 1), (5, 17, 23, 2, 128, 0.8, 3), (5, 17, 23, 8, 128, 0.8, 3)])
def test_a_nan_query_gives_nan_rows_not_empty_ones(grid):
    """In every form of the forward, over the cache too: out and lse of that row are NaN, the other rows as they were."""
    c = Case(*grid, N_)
    q, k, v = c.nat
    cache = c.plan.new_cache()
    c.plan.cache_store(k, v, 0, cache)
    ws = c.plan.new_cache_workspace(grid[0])
    bad = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    bad[0, 3] = bad[-1, -1] = True
    spoilt = q.clone()
    spoilt[bad] = float("nan")

    def lse_call(q, out, lse):
        c.plan.attention_lse(q, k, v, c.mask, out, lse)

    def frames_call(q, out, lse):
        c.plan.cache_attention(q, 0, cache, grid[0], c.mask, out, lse, ws)

    for call in (lse_call, frames_call):
        res = []
        for x in (q, spoilt):
            out, lse = c.plan.new_out(), c.plan.new_lse()
            call(x, out, lse)
            res.append((out, lse))
        c.ok()
        same_but_nan(res[1][0], res[0][0], bad)
        same_but_nan(res[1][1], res[0][1], bad)


@pytest.mark.parametrize("n", [3, 7, 40])
def test_a_nan_query_of_a_token_gives_nan_not_an_empty_row(n):
    c = Case(5, 17, 23, 3, 128, 0.8, 3, N_)
    cache = c.plan.new_cache()
    c.plan.cache_store(c.nat[1], c.nat[2], 0, cache)
    token = torch.arange(800, 800 + n, device="cuda", dtype=torch.int32)
    radius = torch.full((3, n), 4, device="cuda", dtype=torch.int32)
    bad = torch.zeros(3, n, dtype=torch.bool, device="cuda")
    bad[1, n // 2] = bad[2, 0] = True
    radius[2, 1] = -1                                    # an empty row stays one
    q = c.nat[0][:, token.long()].contiguous()
    res = []
    for x in (q, q.masked_fill(bad[..., None], float("nan"))):
        out, lse = torch.empty(3, n, 128, device="cuda"), torch.empty(3, n, device="cuda")
        c.plan.cache_attention_tokens(x, token, radius, cache, 5, out, lse)
        res.append((out, lse))
    c.ok()
    same_but_nan(res[1][0], res[0][0], bad)
    same_but_nan(res[1][1], res[0][1], bad)
    assert torch.isneginf(res[1][1][2, 1]) and not res[1][0][2, 1].any()
