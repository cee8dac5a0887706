"""tra_attention_lse and tra_attention_backward against plain 64-bit formulas and
differences: layouts, output types, spatial tests, query groups, tile widths,
head dims, one-token and ragged grids, masks that keep one key, and the calls
that are refused."""
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


class Setup:
    """A plan with inputs and mask on the GPU; q, k, v, radius in natural order besides."""

    def __init__(self, T, H, W, heads, d, gamma, Rt, flags=0, b=0.5, seed=3, Bmin=1, a=1.0):
        self.grid, self.gamma, self.Rt, self.flags = (T, H, W), gamma, Rt, flags
        self.plan = tra.Plan(T, H, W, heads, d, a, b, gamma, Rt, Bmin, flags)
        self.i = self.plan.info
        self.nat = synth.make_qkv(T, H, W, heads, d, seed, device="cuda", dtype=torch.bfloat16)
        self.q, self.k, self.v = (self.layout(x) for x in self.nat)
        self.mask = self.plan.new_mask()
        h = self.plan.new_entropy()
        self.plan.entropy(self.q, self.k, h)
        self.plan.radius_and_mask(h, self.mask)
        self.radius = gh.to_natural(self.plan.mask_views(self.mask)[0], self.i)
        self.keep = ref.token_mask(T, H, W, gamma, Rt, self.radius, bool(flags & D_))

    def layout(self, x):
        return x.contiguous() if self.plan.natural else gh.to_tile_major(x, self.i)

    def natural(self, x):
        return x if self.plan.natural else gh.to_natural(x, self.i)

    def forward(self):
        out, lse = self.plan.new_out(), self.plan.new_lse()
        self.plan.attention_lse(self.q, self.k, self.v, self.mask, out, lse)
        return out, lse

    def dout(self, seed=11):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x = torch.randn(self.nat[0].shape, generator=g, device="cuda").to(self.plan.out_dtype)
        return x, self.layout(x)

    def backward(self, out, lse, dout, workspace=None):
        grads = tuple(self.plan.new_out() for _ in range(3))
        self.plan.attention_backward(self.q, self.k, self.v, self.mask, out, lse, dout, *grads,
                                     self.plan.new_backward_workspace() if workspace is None else workspace)
        return grads


CASES = [
    # T, H, W, heads, d, gamma, Rt, flags
    (1, 1, 1, 1, 64, 0.7, 0, 0),
    (1, 1, 1, 2, 128, 0.7, 3, N_ | B_),
    (4, 8, 8, 2, 64, 0.7, 2, 0),
    (4, 8, 8, 2, 64, 0.7, 2, N_ | B_),
    (3, 16, 8, 1, 128, 0.8, 1, N_),                     # exactly one tile per frame
    (2, 16, 40, 1, 128, 1.0, 1, B_),
    (5, 17, 23, 2, 128, 0.8, 3, 0),
    (5, 17, 23, 2, 128, 0.8, 3, N_ | B_),
    (5, 17, 23, 2, 128, 0.8, 3, N_ | D_),
    (5, 17, 23, 2, 128, 0.8, 3, D_ | B_),
    (5, 17, 23, 2, 64, 0.8, 3, Q_ | tra.tra_flag_tile_w(8)),
    (5, 17, 23, 2, 128, 0.8, 3, Q_ | N_ | B_ | tra.tra_flag_tile_w(8)),
    (5, 17, 23, 2, 128, 0.8, 3, Q_ | D_ | N_ | tra.tra_flag_tile_w(8)),
    (3, 33, 9, 1, 64, 0.9, 2, N_ | B_ | tra.tra_flag_tile_w(4)),
    (3, 33, 9, 1, 128, 0.9, 2, D_ | tra.tra_flag_tile_w(4)),
    (2, 9, 50, 1, 64, 0.6, 1, N_ | tra.tra_flag_tile_w(32)),
    (2, 9, 50, 2, 128, 0.6, 1, D_ | B_ | tra.tra_flag_tile_w(32)),
    (2, 9, 50, 1, 64, 0.6, 1, D_ | tra.tra_flag_tile_w(16)),
    (7, 1, 5, 3, 64, 0.8, 2, N_),
    (9, 24, 10, 2, 128, 0.8, 0, N_ | B_),               # no temporal reach
    (9, 24, 10, 1, 128, 1.0, 8, N_ | B_),               # every frame reaches every frame
    # more query tiles than SMs: two tiles per CTA
    (5, 17, 23, 8, 64, 0.8, 3, N_ | B_),
    (5, 17, 23, 8, 128, 0.8, 3, 0),
    (5, 17, 23, 8, 128, 0.8, 3, Q_ | N_ | tra.tra_flag_tile_w(8)),
    (5, 17, 23, 8, 64, 0.8, 3, Q_ | D_ | B_ | tra.tra_flag_tile_w(8)),
]


@pytest.mark.parametrize("case", CASES)
def test_lse_and_out(case):
    s = Setup(*case)
    out, lse = s.forward()
    torch.cuda.synchronize()
    assert s.plan.status() == 0
    o_ref, l_ref, o_err, l_err = ref.attention(*s.nat, s.keep)
    ref.check(s.natural(out), o_ref, o_err, "out")
    ref.check(s.natural(lse), l_ref, l_err, "lse")
    # the same attention as the call without the log-sum-exp, up to the rounding of P in the normaliser
    plain = s.plan.new_out()
    s.plan.attention(s.q, s.k, s.v, s.mask, plain)
    ref.check(s.natural(plain), o_ref, 2 * o_err, "out without lse")


@pytest.mark.parametrize("case", CASES)
def test_gradients(case):
    s = Setup(*case)
    out, lse = s.forward()
    dout_nat, dout = s.dout()
    grads = s.backward(out, lse, dout)
    torch.cuda.synchronize()
    assert s.plan.status() == 0
    want, bounds = ref.gradients(*s.nat, s.natural(out), s.natural(lse), dout_nat.bfloat16(), s.keep)
    for name, g, w, e in zip(("dq", "dk", "dv"), grads, want, bounds):
        ref.check(s.natural(g), w, e, name)
        if not s.plan.natural:
            pad = torch.from_numpy(gh.tile_major_index(s.i) < 0).cuda()
            assert not g[:, pad].any(), f"{name}: pad rows are zeros"


@pytest.mark.parametrize("b,Bmin", [(-20.0, 1), (20.0, 1), (-3.0, 2)])
@pytest.mark.parametrize("flags", [0, N_ | B_, N_ | Q_ | tra.tra_flag_tile_w(8), D_])
def test_gradients_of_the_narrowest_and_widest_masks(b, Bmin, flags):
    """One key kept per query (a budget of one token), every key, and a handful."""
    s = Setup(3, 20, 11, 2, 64, 0.7, 1, flags, b=b, Bmin=Bmin)
    out, lse = s.forward()
    dout_nat, dout = s.dout()
    grads = s.backward(out, lse, dout)
    torch.cuda.synchronize()
    assert s.plan.status() == 0
    if b == -20.0:
        assert int(s.keep.sum(-1).min()) >= 1 and (s.radius == 0).all()
    want, bounds = ref.gradients(*s.nat, s.natural(out), s.natural(lse), dout_nat.bfloat16(), s.keep)
    for name, g, w, e in zip(("dq", "dk", "dv"), grads, want, bounds):
        ref.check(s.natural(g), w, e, name)


def test_gradients_against_differences():
    """Along random directions, central differences of the 64-bit loss sum(out * dout) match the kernels' gradients."""
    s = Setup(4, 9, 13, 2, 64, 0.8, 2, N_, b=-1.0)
    out, lse = s.forward()
    dout_nat, dout = s.dout()
    grads = [g.double() for g in s.backward(out, lse, dout)]
    w = dout_nat.bfloat16().double()
    q, k, v = (x.double() for x in s.nat)
    bounds = ref.gradients(*s.nat, out, lse, dout_nat.bfloat16(), s.keep)[1]

    def loss(q, k, v):
        return float((ref.attention(q, k, v, s.keep)[0] * w).sum())

    g = torch.Generator(device="cuda").manual_seed(5)
    for n in range(3):
        u = torch.randn(q.shape, generator=g, device="cuda", dtype=torch.float64)
        step = [torch.zeros_like(u) for _ in range(3)]
        step[n] = u * 1e-5
        diff = (loss(q + step[0], k + step[1], v + step[2]) - loss(q - step[0], k - step[1], v - step[2])) / 2e-5
        # the bounds hold for the gradient given the kernel's out and lse; those are themselves off by P's rounding
        tol = 2 * float((bounds[n] * u.abs()).sum()) + 1e-6 * abs(diff)
        assert abs(float((grads[n] * u).sum()) - diff) <= tol


def test_gradients_are_bit_identical_across_runs_and_workspaces():
    s = Setup(5, 17, 23, 2, 128, 0.8, 3, N_ | B_ | Q_ | tra.tra_flag_tile_w(8))
    out, lse = s.forward()
    _, dout = s.dout()
    ws = s.plan.new_backward_workspace()
    a = s.backward(out, lse, dout, ws)
    ws.fill_(255)                                       # the workspace carries nothing over
    b = s.backward(out, lse, dout, ws)
    torch.cuda.synchronize()
    assert s.plan.status() == 0
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_a_training_step_in_a_graph_and_on_another_stream():
    """Forward and backward captured together, replayed on new inputs, equal the eager calls."""
    s = Setup(4, 18, 10, 2, 64, 0.8, 2, N_ | B_)
    _, dout = s.dout()
    out, lse = s.plan.new_out(), s.plan.new_lse()
    grads = tuple(s.plan.new_out() for _ in range(3))
    ws = s.plan.new_backward_workspace()

    def step():
        s.plan.attention_lse(s.q, s.k, s.v, s.mask, out, lse)
        s.plan.attention_backward(s.q, s.k, s.v, s.mask, out, lse, dout, *grads, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g = torch.Generator(device="cuda").manual_seed(9)
    for x in (s.q, s.k, s.v, dout):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in (out, lse, *grads)]
    step()
    torch.cuda.synchronize()
    assert s.plan.status() == 0
    for x, y in zip(got, (out, lse, *grads)):
        assert torch.equal(x, y)
    graph.reset()


def test_two_backward_passes_at_once_on_two_streams():
    """Each with its own workspace: the same bits as one after the other."""
    sets = [Setup(5, 17, 23, 2, 128, 0.8, 3, N_ | B_, seed=x) for x in (1, 2)]
    fwd = [s.forward() for s in sets]
    douts = [s.dout()[1] for s in sets]
    want = [s.backward(*f, d) for s, f, d in zip(sets, fwd, douts)]
    torch.cuda.synchronize()
    got = []
    for s, f, d in zip(sets, fwd, douts):
        with torch.cuda.stream(torch.cuda.Stream()):
            ws = s.plan.new_backward_workspace()
            got.append([s.backward(*f, d, ws) for _ in range(5)])
    torch.cuda.synchronize()
    assert sets[0].plan.status() == 0
    for w, g5 in zip(want, got):
        for g in g5:
            assert all(torch.equal(x, y) for x, y in zip(g, w))


def test_gradients_at_a_720p_frame_grid():
    """A grid whose key tiles are listed by hundreds of slots, against the formulas on the rows of two frames' reach."""
    s = Setup(3, 45, 80, 1, 128, 0.8, 2, N_ | B_ | Q_, b=1.5)
    out, lse = s.forward()
    dout_nat, dout = s.dout()
    grads = s.backward(out, lse, dout)
    torch.cuda.synchronize()
    assert s.plan.status() == 0
    assert int(s.plan.mask_views(s.mask)[1].max()) > 60
    want, bounds = ref.gradients(*s.nat, out, lse, dout_nat, s.keep)
    for name, g, w, e in zip(("dq", "dk", "dv"), grads, want, bounds):
        ref.check(g, w, e, name)


def test_autograd_use():
    """The calls inside a torch.autograd.Function: leaf gradients are the kernels'."""
    s = Setup(3, 10, 12, 2, 64, 0.8, 1, N_)

    class Attention(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v):
            out, lse = s.plan.new_out(), s.plan.new_lse()
            s.plan.attention_lse(q, k, v, s.mask, out, lse)
            ctx.save_for_backward(q, k, v, out, lse)
            return out

        @staticmethod
        def backward(ctx, dout):
            q, k, v, out, lse = ctx.saved_tensors
            grads = tuple(s.plan.new_out() for _ in range(3))
            s.plan.attention_backward(q, k, v, s.mask, out, lse, dout.contiguous(), *grads, s.plan.new_backward_workspace())
            return tuple(g.to(q.dtype) for g in grads)

    leaves = [x.clone().requires_grad_() for x in (s.q, s.k, s.v)]
    out = Attention.apply(*leaves)
    w = torch.randn_like(out)
    (out * w).sum().backward()
    eager_out, lse = s.forward()
    want = s.backward(eager_out, lse, w)
    for x, y in zip(leaves, want):
        assert torch.equal(x.grad, y.bfloat16())


def test_corrupted_mask_is_reported_by_the_backward_and_not_followed():
    s = Setup(5, 17, 23, 2, 128, 0.8, 3, N_ | B_ | Q_ | tra.tra_flag_tile_w(8))
    out, lse = s.forward()
    _, dout = s.dout()
    torch.cuda.synchronize()
    good = s.mask.clone()
    for spoil in ("count", "list", "group"):
        s.mask.copy_(good)
        if spoil == "count":
            s.plan.mask_views(s.mask)[1][0, 0] = s.i.list_cap + 5
            s.plan.mask_views(s.mask)[1][1, 2] = -1
        elif spoil == "list":
            s.plan.mask_views(s.mask)[3][0, 0, 0] = 0x7FFE
            s.plan.mask_views(s.mask)[3][1, 0, 0] = s.i.n_tiles - 1
        else:
            s.plan.group_view(s.mask)[1, 2, 5] = 0x7FFF
        s.backward(out, lse, dout)
        torch.cuda.synchronize()
        assert s.plan.status() == 6, spoil
    s.mask.copy_(good)
    grads = s.backward(out, lse, dout)
    torch.cuda.synchronize()
    assert s.plan.status() == 0
    assert all(torch.isfinite(g).all() for g in grads)


def test_bounded_waits_of_the_training_kernels_give_up():
    s = Setup(4, 8, 8, 2, 64, 0.7, 2)
    out, lse = s.forward()
    _, dout = s.dout()
    torch.cuda.synchronize()
    p = tra.Plan(4, 8, 8, 2, 64, 1.0, 0.5, 0.7, 2, 1, tra.TRA_FLAG_DEBUG_NO_WAIT)
    p.attention_backward(s.q, s.k, s.v, s.mask, out, lse, dout, p.new_out(), p.new_out(), p.new_out(),
                         p.new_backward_workspace())
    torch.cuda.synchronize()
    assert p.status() == 5                              # TRA_ERR_TIMEOUT
    s.backward(out, lse, dout)
    torch.cuda.synchronize()
    assert s.plan.status() == 0


@pytest.mark.parametrize("grid", [(4, 8, 8, 2), (9, 24, 10, 1), (5, 17, 23, 2), (5, 17, 23, 8)])
def test_bounded_waits_of_the_forward_variants_give_up(grid):
    """One chain, clusters of four and two CTAs per tile, and pairs of tiles: each ends and reports the timeout."""
    T, H, W, heads = grid
    s = Setup(T, H, W, heads, 64, 0.9, 8, N_)
    want = [x.clone() for x in s.forward()]
    torch.cuda.synchronize()
    assert s.plan.status() == 0
    p = tra.Plan(T, H, W, heads, 64, 1.0, 0.5, 0.9, 8, 1, N_ | tra.TRA_FLAG_DEBUG_NO_WAIT)
    p.attention_lse(s.q, s.k, s.v, s.mask, p.new_out(), p.new_lse())
    torch.cuda.synchronize()
    assert p.status() == 5                              # TRA_ERR_TIMEOUT
    got = s.forward()
    torch.cuda.synchronize()
    assert s.plan.status() == 0
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_refusals():
    s = Setup(4, 8, 8, 2, 64, 0.7, 2, N_)
    out, lse = s.forward()
    _, dout = s.dout()
    ws = s.plan.new_backward_workspace()
    grads = [s.plan.new_out() for _ in range(3)]
    with pytest.raises(tra.TraError) as e:
        s.plan.attention_backward(s.q, s.k, s.v, s.mask, out, lse, dout, *grads, ws[:-256])
    assert e.value.status == 3                          # TRA_ERR_WORKSPACE
    with pytest.raises(ValueError):
        s.plan.attention_backward(s.q, s.k, s.v, s.mask, out, lse, dout.bfloat16(), *grads, ws)
    with pytest.raises(ValueError):
        s.plan.attention_backward(s.q, s.k, s.v, s.mask, out, lse[:, :-1].contiguous(), dout, *grads, ws)
    with pytest.raises(ValueError):
        s.plan.attention_lse(s.q, s.k, s.v, s.mask[:-1], out, lse)
    with pytest.raises(ValueError):
        s.plan.attention_lse(s.q.mT.contiguous().mT, s.k, s.v, s.mask, out, lse)
    with pytest.raises(ValueError):
        s.plan.attention_lse(s.q.cpu(), s.k, s.v, s.mask, out, lse)
    torch.cuda.synchronize()
    assert s.plan.status() == 0
