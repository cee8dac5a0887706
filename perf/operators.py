"""What is measured of the attention operators that train under a radius mask and
that read keys and values from an 8-bit cache.

Every operator works on a T x H x W grid of video tokens in natural frame-major
order, n = (t*H + h)*W + w.  A query of radius r keeps the keys of the frames
|dt| <= min(Rt, T-1) whose spatial distance (Chebyshev, or Euclidean for the
disk) is at most floor(r * gamma^|dt| + 1e-9).

  forward   attention under the mask with the log-sum-exp of each row
  backward  the gradients of q, k and v, probabilities recomputed
  store     frames of keys and values into the cache: e4m3 codes with one
            power-of-two scale for each (1, 128/tw, tw) box of tokens and head
  frames    whole frames of queries over the cached frames
  tokens    single tokens over the cached frames

`run` computes the plain form in elementary torch operations, or, where `own`
is true, makes the calls that a user of the framework makes.
"""
import math

import torch

own = False

E4M3_MAX = 448.0


# ------------------------------------------------------------------ the cases
def _case(name, op, T, H, W, heads, d, gamma, Rt, **more):
    c = {"op": op, "T": T, "H": H, "W": W, "heads": heads, "d": d, "gamma": gamma, "Rt": Rt, "disk": False,
         "qsort": False, "tile_w": _tile_w(H, W)}
    c.update(more)
    if name is not None:
        c["name"] = name
    return c


def _tile_w(H, W):
    """The tile width with the least padding (ties: the tile's long side along the frame's short side)."""
    best = None
    for tw in (4, 8, 16, 32):
        if -(-W // tw) > 32:
            continue
        key = (-(-H // (128 // tw)) * -(-W // tw), tw if H <= W else -tw)
        if best is None or key < best[0]:
            best = (key, tw)
    return best[1]


def listed():
    return [
        # the smallest grid of the tests: latency of a training step's two calls
        _case("forward-4x8x8", "forward", 4, 8, 8, 2, 64, 0.7, 2),
        # Wan-1.3B at 480p, some of its heads: an ordinary training forward
        _case("forward-21x30x52", "forward", 21, 30, 52, 4, 128, 0.8, 6),
        _case("backward-4x8x8", "backward", 4, 8, 8, 2, 64, 0.7, 2),
        # a ragged grid (tiles padded on both sides), the Euclidean disk
        _case("backward-5x17x23-disk", "backward", 5, 17, 23, 3, 128, 0.8, 3, disk=True),
        _case("backward-21x30x52", "backward", 21, 30, 52, 4, 128, 0.8, 6),
        # Wan-14B at 720p, some of its heads, radius-sorted query groups: the largest
        _case("backward-21x45x80-sorted", "backward", 21, 45, 80, 4, 128, 0.8, 6, qsort=True),
        # a newly generated latent frame goes into the cache, every head of Wan-14B
        _case("store-1x45x80", "store", 21, 45, 80, 40, 128, 0.8, 6, frame=20, frames=1),
        # a whole clip of Wan-1.3B goes into the cache at once (a conditioning video)
        _case("store-21x30x52", "store", 21, 30, 52, 12, 128, 0.8, 6, frame=0, frames=21),
        # one denoising call of the newest frame of a 720p clip over the cache
        _case("frames-1of21x45x80", "frames", 21, 45, 80, 8, 128, 0.8, 6, frame=20, frames=1),
        # a chunk of three frames inside a ragged clip, half of it cached
        _case("frames-3of9x17x23", "frames", 9, 17, 23, 4, 64, 0.8, 3, frame=3, frames=3),
        # one token at a time, every head of Wan-14B
        _case("tokens-1of21x45x80", "tokens", 21, 45, 80, 40, 128, 0.8, 6, frame=20, tokens=1),
        # one row of a frame of Wan-1.3B
        _case("tokens-52of21x30x52", "tokens", 21, 30, 52, 12, 128, 0.8, 6, frame=20, tokens=52),
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["forward", "backward", "backward", "store", "frames", "tokens"])
    d = rng.choice([64, 128])
    T, H, W = log(1, 33), log(3, 45), log(3, 80)
    Rt = rng.randint(0, 6)
    heads = log(1, 40)
    most = 12_000_000_000 if op in ("forward", "backward", "frames") else 2 ** 62
    while heads > 1 and heads * T * H * W * min(T, 2 * Rt + 1) * H * W > most:
        heads -= 1
    more = {}
    if op in ("forward", "backward"):
        tw = _tile_w(H, W)
        more["qsort"] = -(-H // (128 // tw)) <= 4 and rng.random() < 0.5
    else:
        more["frame"] = rng.randrange(T)
        more["frames"] = rng.randint(1, max(1, min(4, T - more["frame"])))
    if op == "tokens":
        more["tokens"] = min(log(1, 52), H * W)
    return _case(None, op, T, H, W, heads, d, rng.choice([0.6, 0.7, 0.8, 0.9, 1.0]), Rt,
                 disk=op != "store" and rng.random() < 0.3, **more)


# ------------------------------------------------------------------ the inputs
def _generator(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(7_000_003 * (int(seed) + 1))
    return g


def _radii(case, g, device, heads, rows):
    """Radii with the spread that lognormal entropies give, about 15 % of the pairs at 21 frames."""
    r0 = 0.42 * math.sqrt(case["H"] * case["W"])
    z = torch.randn(heads, rows, generator=g, device=device)
    return (r0 * torch.exp(0.4 * z)).round().clamp(0, 200).to(torch.int32)


def _activations(case, g, device, rows):
    """q, k, v of one attention layer: keys with a smooth field over the grid, query rows of lognormal temperature."""
    heads, d = case["heads"], case["d"]
    q, k, v = (torch.randn(heads, rows, d, generator=g, device=device) for _ in range(3))
    q *= torch.exp(0.5 * torch.randn(heads, rows, 1, generator=g, device=device))
    n = torch.arange(rows, device=device)
    at = torch.stack([n // (case["H"] * case["W"]) / max(1, case["T"]), n // case["W"] % case["H"] / case["H"],
                      n % case["W"] / case["W"]], 1).float()
    wave = torch.randint(1, 4, (heads, 3, d), generator=g, device=device).float()
    phase = torch.rand(heads, 1, d, generator=g, device=device)
    k += torch.sin(2 * math.pi * (at @ wave + phase))
    return q.bfloat16(), k.bfloat16(), v.bfloat16()


def _tiles(case, device):
    """The natural token of each row of each (1, th, tw) tile of one frame (H*W past the grid's edge): [tiles, 128]."""
    H, W, tw = case["H"], case["W"], case["tile_w"]
    th = 128 // tw
    nh, nw = -(-H // th), -(-W // tw)
    a = torch.arange(nh * nw, device=device)[:, None]
    i = torch.arange(128, device=device)[None]
    h, w = (a // nw) * th + i // tw, (a % nw) * tw + i % tw
    return torch.where((h < H) & (w < W), h * W + w, H * W)


def _reach(case, delta):
    return case["gamma"] ** abs(delta)


def _entropies(case, radius):
    """Entropies whose budget exp(H) is reached exactly at the given radii: ln(count - 1/2)."""
    T, H, W = case["T"], case["H"], case["W"]
    n = torch.arange(T * H * W, device=radius.device)
    t, h, w = n // (H * W), n // W % H, n % W
    rt = min(case["Rt"], T - 1)
    count = torch.zeros(radius.shape, dtype=torch.float64, device=radius.device)
    for dt in range(-rt, rt + 1):
        s = torch.floor(radius.double() * _reach(case, dt) + 1e-9)
        if case["disk"]:
            inside = torch.zeros_like(count)
            for dh in range(-H + 1, H):
                half = torch.floor(torch.sqrt((s * s - dh * dh).clamp(min=0)))
                wide = torch.minimum(w + half, torch.tensor(W - 1.0, device=s.device)) - (w - half).clamp(min=0) + 1
                inside += torch.where((s >= abs(dh)) & (h + dh >= 0) & (h + dh < H), wide, 0.0)
        else:
            tall = (h + s).clamp(max=H - 1) - (h - s).clamp(min=0) + 1
            inside = tall * ((w + s).clamp(max=W - 1) - (w - s).clamp(min=0) + 1)
        count += torch.where((t + dt >= 0) & (t + dt < T), inside, 0.0)
    return torch.log(count - 0.5).float()


def prepare(case, seed):
    device = "cuda"
    g = _generator(seed, device)
    T, H, W, heads, d, op = (case[n] for n in ("T", "H", "W", "heads", "d", "op"))
    N = T * H * W
    s = {"case": case}
    if op in ("forward", "backward"):
        s["q"], s["k"], s["v"] = _activations(case, g, device, N)
        s["radius"] = _radii(case, g, device, heads, N)
        if op == "backward":
            s["dout"] = torch.randn(heads, N, d, generator=g, device=device).bfloat16()
            s["out"], s["lse"] = _attention(case, s["q"], s["k"], s["v"], s["radius"], 0)
    else:
        cached = case["frame"] + case["frames"] if op != "tokens" else case["frame"] + 1
        q, k, v = _activations(case, g, device, N)
        rows = slice(case["frame"] * H * W, (case["frame"] + case.get("frames", 1)) * H * W)
        if op == "store":
            s["k"], s["v"] = k[:, rows].contiguous(), v[:, rows].contiguous()
        else:
            s["tiles"] = _tiles(case, device)
            s["cached"] = cached
            s["k8"], s["k_scale"] = _quantise(case, k)
            s["v8"], s["v_scale"] = _quantise(case, v)
            s["radius"] = _radii(case, g, device, heads, N)
            if op == "frames":
                s["q"] = q[:, rows].contiguous()
            else:
                first = rows.start + int(torch.randint(0, H * W - case["tokens"] + 1, (1,), generator=g, device=device))
                s["token"] = torch.arange(first, first + case["tokens"], device=device, dtype=torch.int32)
                s["q"] = q[:, s["token"].long()].contiguous()
                s["token_radius"] = s["radius"][:, s["token"].long()].contiguous()
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """The plan, the mask and the buffers that a user's program keeps."""
    import sparse_attention_video_tra_b200 as tra

    c = s["case"]
    flags = tra.TRA_FLAG_NATURAL | tra.TRA_FLAG_OUT_BF16 | tra.tra_flag_tile_w(c["tile_w"])
    flags |= tra.TRA_FLAG_DISK if c["disk"] else 0
    flags |= tra.TRA_FLAG_QSORT if c["qsort"] else 0
    plan = s["plan"] = tra.Plan(c["T"], c["H"], c["W"], c["heads"], c["d"], 1.0, 0.0, c["gamma"], c["Rt"], 1, flags)
    if c["op"] in ("forward", "backward", "frames"):
        s["mask"] = plan.radius_and_mask(_entropies(c, s["radius"]), plan.new_mask())
    if c["op"] == "forward":
        s["out"], s["lse"] = plan.new_out(), plan.new_lse()
    elif c["op"] == "backward":
        s["dq"], s["dk"], s["dv"] = plan.new_out(), plan.new_out(), plan.new_out()
        s["workspace"] = plan.new_backward_workspace()
    elif c["op"] == "store":
        s["cache"] = plan.new_cache()
    else:
        s["cache"] = plan.new_cache()
        for view, held in zip(plan.cache_views(s["cache"]), (s["k8"], s["v8"], s["k_scale"], s["v_scale"])):
            view.view(torch.uint8).copy_(held.view(view.shape).view(torch.uint8))
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:2], device="cuda")
        if c["op"] == "frames":
            s["workspace"] = plan.new_cache_workspace(c["frames"])


# ------------------------------------------------------------------ one pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    c, plan = s["case"], s["plan"]
    if c["op"] == "forward":
        plan.attention_lse(s["q"], s["k"], s["v"], s["mask"], s["out"], s["lse"])
        return s["out"], s["lse"]
    if c["op"] == "backward":
        plan.attention_backward(s["q"], s["k"], s["v"], s["mask"], s["out"], s["lse"], s["dout"], s["dq"], s["dk"],
                                s["dv"], s["workspace"])
        return s["dq"], s["dk"], s["dv"]
    if c["op"] == "store":
        plan.cache_store(s["k"], s["v"], c["frame"], s["cache"])
        f = slice(c["frame"], c["frame"] + c["frames"])
        return tuple(x.unflatten(1, (c["T"], -1))[:, f] for x in plan.cache_views(s["cache"]))
    if c["op"] == "frames":
        plan.cache_attention(s["q"], c["frame"], s["cache"], s["cached"], s["mask"], s["out"], s["lse"], s["workspace"])
    else:
        plan.cache_attention_tokens(s["q"], s["token"], s["token_radius"], s["cache"], s["cached"], s["out"], s["lse"])
    return s["out"], s["lse"]


def _run_plain(s):
    c = s["case"]
    if c["op"] == "forward":
        return _attention(c, s["q"], s["k"], s["v"], s["radius"], 0)
    if c["op"] == "backward":
        return _gradients(c, s)
    if c["op"] == "store":
        (k8, ks), (v8, vs) = _quantise(c, s["k"]), _quantise(c, s["v"])
        return k8, v8, ks, vs
    k = _values(c, s["k8"], s["k_scale"], s["tiles"], s["cached"])
    v = _values(c, s["v8"], s["v_scale"], s["tiles"], s["cached"])
    if c["op"] == "frames":
        first = c["frame"] * c["H"] * c["W"]
        return _attention(c, s["q"], k, v, s["radius"][:, first:first + s["q"].shape[1]], c["frame"])
    keep = _keep(c, s["token"].long(), torch.arange(k.shape[1], device=k.device), s["token_radius"])
    x = torch.where(keep, (s["q"].float() / math.sqrt(c["d"])) @ k.mT, -math.inf)
    top = x.amax(2, keepdim=True)
    p = torch.exp(x - top)
    total = p.sum(2, keepdim=True)
    return (p @ v / total).bfloat16(), (top + torch.log(total))[..., 0]


# ------------------------------------------------------------------ plain forms
def _keep(c, n, m, radius):
    """Which keys m the queries n of the given radii keep: [heads, len(n), len(m)]."""
    H, W = c["H"], c["W"]
    dt = (n[:, None] // (H * W) - m[None] // (H * W)).abs()
    dh = (n[:, None] // W % H - m[None] // W % H).abs()
    dw = (n[:, None] % W - m[None] % W).abs()
    rt = min(c["Rt"], c["T"] - 1)
    decay = torch.tensor([_reach(c, i) for i in range(max(rt, c["T"]) + 1)], dtype=torch.float64, device=n.device)
    far = dh * dh + dw * dw if c["disk"] else torch.maximum(dh, dw)
    steps = torch.arange(decay.numel(), device=n.device)
    half = torch.floor(radius[..., None].double() * decay + 1e-9).to(torch.int32)          # [heads, n, |dt|]
    half = torch.where(steps <= rt, half * half if c["disk"] else half, -1)
    return half.gather(2, dt.expand(radius.shape[0], -1, -1)) >= far


def _spans(c, frame, frames, cached):
    """Blocks of query frames with the frames their keys lie in, small enough for the score matrices."""
    area, rt = c["H"] * c["W"], min(c["Rt"], c["T"] - 1)
    step = max(1, frames)
    while step > 1 and c["heads"] * step * area * min(cached, step + 2 * rt) * area > 400_000_000:
        step = -(-step // 2)
    return [(a, min(a + step, frame + frames), max(0, a - rt), min(cached, a + step + rt))
            for a in range(frame, frame + frames, step)]


def _attention(c, q, k, v, radius, frame):
    """softmax of the kept scores times v, and the rows' log-sum-exp; q and radius begin at the given frame."""
    area = c["H"] * c["W"]
    out, lse = [], []
    for a, b, lo, hi in _spans(c, frame, q.shape[1] // area, k.shape[1] // area):
        rows, keys = slice((a - frame) * area, (b - frame) * area), slice(lo * area, hi * area)
        n = torch.arange(a * area, b * area, device=q.device)
        m = torch.arange(lo * area, hi * area, device=q.device)
        x = (q[:, rows].float() / math.sqrt(c["d"])) @ k[:, keys].float().mT
        x = torch.where(_keep(c, n, m, radius[:, rows]), x, -math.inf)
        top = x.amax(2, keepdim=True)
        p = torch.exp(x - top)
        total = p.sum(2, keepdim=True)
        out.append(p @ v[:, keys].float() / total)
        lse.append((top + torch.log(total))[..., 0])
    return torch.cat(out, 1).bfloat16(), torch.cat(lse, 1)


def _gradients(c, s):
    """P = exp(x - lse), dP = dO V^T, dS = P (dP - rowsum(dO O)); dQ = dS K, dK = dS^T Q, dV = P^T dO."""
    area, root = c["H"] * c["W"], 1 / math.sqrt(c["d"])
    dq = []
    dk = torch.zeros(s["k"].shape, device=s["k"].device)
    dv = torch.zeros_like(dk)
    for a, b, lo, hi in _spans(c, 0, c["T"], c["T"]):
        rows, keys = slice(a * area, b * area), slice(lo * area, hi * area)
        n = torch.arange(a * area, b * area, device=dk.device)
        m = torch.arange(lo * area, hi * area, device=dk.device)
        q, k, v, do = s["q"][:, rows].float(), s["k"][:, keys].float(), s["v"][:, keys].float(), s["dout"][:, rows].float()
        p = torch.exp((q * root) @ k.mT - s["lse"][:, rows, None])
        p = torch.where(_keep(c, n, m, s["radius"][:, rows]), p, 0.0)
        dv[:, keys] += p.mT @ do
        ds = p * (do @ v.mT - (do * s["out"][:, rows].float()).sum(2, keepdim=True)) * root
        dq.append(ds @ k)
        dk[:, keys] += ds.mT @ q
    return torch.cat(dq, 1).bfloat16(), dk.bfloat16(), dv.bfloat16()


def _quantise(c, x):
    """Frames of rows [heads, frames*H*W, d] as e4m3 codes [heads, frames, tiles, 128, d] (zeros past the grid's edge) with
    one scale per tile: the smallest power of two, at least 2^-126, that brings the largest magnitude to at most 448."""
    area = c["H"] * c["W"]
    x = torch.nn.functional.pad(x.float().unflatten(1, (-1, area)), (0, 0, 0, 1))[:, :, _tiles(c, x.device)]
    mantissa, exponent = torch.frexp(x.abs().amax((3, 4)))
    exponent = torch.where(mantissa == 0, 0, (exponent - 9 + (mantissa > E4M3_MAX / 512)).clamp(min=-126))
    scale = torch.ldexp(torch.ones_like(mantissa), exponent)
    return (x / scale[..., None, None]).to(torch.float8_e4m3fn), scale


def _values(c, codes, scale, tiles, cached):
    """The rows [heads, cached*H*W, d] in natural order that the cache holds for its first frames."""
    x = codes[:, :cached].float() * scale[:, :cached, :, None, None]
    at = torch.empty(c["H"] * c["W"] + 1, dtype=torch.int64, device=x.device)
    at[tiles.flatten()] = torch.arange(tiles.numel(), device=x.device)
    return x.flatten(2, 3)[:, :, at[:-1]].flatten(1, 2)


# ------------------------------------------------------------------ the work
def work(case):
    c = case
    T, H, W, heads, d = c["T"], c["H"], c["W"], c["heads"], c["d"]
    N, area = T * H * W, H * W
    tiles = -(-H // (128 // c["tile_w"])) * -(-W // c["tile_w"])
    if c["op"] == "store":
        rows = heads * c["frames"]
        return {"bytes": rows * (2 * area * d * 2 + 2 * tiles * (128 * d + 4)), "flops": rows * area * d * 4}
    # pairs kept by the queries, counted on one head of fixed radii
    probe = {**c, "heads": 1}
    radius = _radii(probe, _generator(0, "cpu"), "cpu", 1, N)
    counts = torch.exp(_entropies({**probe}, radius).double()) + 0.5
    if c["op"] in ("forward", "backward"):
        pairs = float(counts.sum()) * heads
        rows = heads * N
        if c["op"] == "forward":
            return {"bytes": rows * (4 * d * 2 + 4), "flops": 4 * d * pairs}
        return {"bytes": rows * (8 * d * 2 + 4), "flops": 10 * d * pairs}
    first, cached = c["frame"], c["frame"] + c.get("frames", 1)
    window = cached - max(0, first - min(c["Rt"], T - 1))
    queries = c["tokens"] if c["op"] == "tokens" else c["frames"] * area
    # the queries lie in the newest frames: no key lies behind them
    ahead = {**probe, "T": cached}
    counts = torch.exp(_entropies(ahead, radius[:, :cached * area]).double()) + 0.5
    mean = float(counts[:, first * area:].mean())
    pairs = heads * queries * mean
    keys = heads * min(window * area, queries * mean) if c["op"] == "tokens" else heads * window * area
    return {"bytes": 2 * keys * d + heads * queries * (2 * d * 2 + 4), "flops": 4 * d * pairs}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    T, H, W, heads, d, op = (case[n] for n in ("T", "H", "W", "heads", "d", "op"))
    area, rt, device = H * W, min(case["Rt"], case["T"] - 1), "cuda"
    y, x = torch.meshgrid(torch.arange(H, device=device), torch.arange(W, device=device), indexing="ij")
    place = torch.stack([y.flatten(), x.flatten()], 1).double()
    far = torch.cdist(place, place, p=2.0, compute_mode="donot_use_mm_for_euclid_dist") if case["disk"] else \
        torch.cdist(place, place, p=math.inf)

    def kept(t, u, radius):
        """Of the queries of frame t, all of them, the keys of frame u: [heads, H*W, H*W]."""
        half = torch.floor(radius.double() * case["gamma"] ** abs(t - u) + 1e-9)[..., None]
        return far * far <= half * half + 0.25 if case["disk"] else far <= half + 0.25

    if op == "store":
        def codes(rows):
            a = torch.zeros(heads, case["frames"], area + 1, d, dtype=torch.float64, device=device)
            a[:, :, :area] = rows.double().view(heads, case["frames"], area, d)
            boxes = torch.stack([a[:, :, at] for at in _tiles(case, device)], 2)
            most = boxes.abs().amax((3, 4))
            scale = torch.where(most > 0, torch.exp2(torch.ceil(torch.log2(most / 448))), 1.0)
            return boxes / scale[..., None, None], scale

        (k8, ks), (v8, vs) = codes(s["k"]), codes(s["v"])
        return k8, v8, ks, vs
    if op in ("forward", "backward"):
        k, v, cached = s["k"].double(), s["v"].double(), T
        frames, first = range(T), 0
    else:
        def held(codes, scale):
            full = torch.empty(heads, T, area + 1, d, dtype=torch.float64, device=device)
            for i, at in enumerate(s["tiles"]):
                full[:, :, at] = codes[:, :, i].double() * scale[:, :, i, None, None].double()
            return full[:, :, :area].flatten(1, 2)

        k, v, cached = held(s["k8"], s["k_scale"]), held(s["v8"], s["v_scale"]), s["cached"]
        first = case["frame"]
        frames = range(first, first + case.get("frames", 1))
    if op == "tokens":
        outs, lses = [], []
        for i, n in enumerate(s["token"].tolist()):
            t, at = n // area, n % area
            score, value = [], []
            for u in range(max(0, t - rt), min(cached, t + rt + 1)):
                half = torch.floor(s["token_radius"][:, i].double() * case["gamma"] ** abs(t - u) + 1e-9)[:, None]
                ok = far[at] ** 2 <= half * half + 0.25 if case["disk"] else far[at] <= half + 0.25
                ku = k[:, u * area:(u + 1) * area]
                dot = (ku * s["q"][:, i, None].double()).sum(2) / math.sqrt(d)
                score.append(dot.masked_fill(~ok, -math.inf))
                value.append(v[:, u * area:(u + 1) * area])
            score, value = torch.cat(score, 1), torch.cat(value, 1)
            lses.append(torch.logsumexp(score, 1))
            outs.append((torch.softmax(score, 1)[..., None] * value).sum(1))
        return torch.stack(outs, 1), torch.stack(lses, 1)
    out, lse, dq = [], [], []
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    for t in frames:
        rows = slice((t - first) * area, (t - first + 1) * area)
        lo, hi = max(0, t - rt), min(cached, t + rt + 1)
        keys = slice(lo * area, hi * area)
        radius = s["radius"][:, t * area:(t + 1) * area]
        q = s["q"][:, rows].double()
        score = torch.einsum("gid,gjd->gij", q, k[:, keys]) / math.sqrt(d)
        ok = torch.cat([kept(t, u, radius) for u in range(lo, hi)], 2)
        score = score.masked_fill(~ok, -math.inf)
        if op != "backward":
            lse.append(torch.logsumexp(score, 2))
            out.append(torch.softmax(score, 2) @ v[:, keys])
            continue
        p = torch.exp(score - s["lse"][:, rows, None].double())
        do = s["dout"][:, rows].double()
        dv[:, keys] += torch.einsum("gij,gid->gjd", p, do)
        dp = torch.einsum("gid,gjd->gij", do, v[:, keys])
        dp -= torch.einsum("gid,gid->gi", do, s["out"][:, rows].double())[..., None]
        dp *= p
        dq.append(torch.einsum("gij,gjd->gid", dp, k[:, keys]) / math.sqrt(d))
        dk[:, keys] += torch.einsum("gij,gid->gjd", dp, q) / math.sqrt(d)
    if op == "backward":
        return torch.cat(dq, 1), dk, dv
    return torch.cat(out, 1), torch.cat(lse, 1)
