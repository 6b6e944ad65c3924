"""Cases that time the operators around the DiT's attention: rotary positions over (time, height, width),
layer norm with modulation forward and backward, and the linear layer with 4-bit weights and group scales.

``run`` computes a case in its plain form (elementary torch operations), or, with ``own`` set, by the calls
a user makes of this package.  ``exact`` is the operator's definition in 64 bits.

Definitions
  rope        pairs (x1, x2) of channels turn by a = p * theta^(-2 i / d) (i-th of an axis' d / 2 pairs, p the
              token's position on that axis): y1 = x1 cos a - x2 sin a, y2 = x1 sin a + x2 cos a; the adjoint
              (gradient) turns by -a; channels that no axis holds pass through
  ln_fwd      y = (x - mean) rstd (u + w) + b per row, u = 1 with unit_offset else 0, w and b per group of rows
  ln_bwd      g = dy (u + w): dx = rstd (g - mean(g) - xhat mean(g xhat)); dw = sum dy xhat, db = sum dy over
              the rows of each group
  w4          y = x W^T, W = bf16(code * scale), 4-bit codes -8..7 (stored + 8, two per byte, the even column in
              the low half), one bf16 scale per row of W and group of columns; fp32 sums
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# time, height and width channels of a head
AXES = {64: ((16, 24, 24), (22, 20, 22), (0, 32, 32)), 128: ((16, 56, 56), (44, 42, 42), (32, 48, 48), (64, 32, 0))}


def listed():
    return [
        # text tokens of one action tail, each with a position of its own: a call whose latency counts
        dict(name="rope_tail", op="rope", tokens=64, heads=16, dim=128, axes="16,56,56", dtype="bf16", halves=False,
             adjoint=False, fused=False, grid_h=0, grid_w=0),
        # q and k of one 30-frame segment at 1280x704 (22 x 40 tokens a frame), views of the QKV projection's output
        dict(name="rope_segment", op="rope", tokens=26400, heads=16, dim=128, axes="16,56,56", dtype="bf16", halves=False,
             adjoint=False, fused=True, grid_h=22, grid_w=40),
        # gradients in fp32 of an 8-frame segment at 480x832 (15 x 26 tokens a frame), channel halves paired
        dict(name="rope_grad", op="rope", tokens=3120, heads=16, dim=128, axes="44,42,42", dtype="f32", halves=True,
             adjoint=True, fused=False, grid_h=15, grid_w=26),
        # one conditioning vector
        dict(name="ln_vector", op="ln_fwd", rows=1, cols=2048, x="bf16", y="bf16", p="bf16", rpg=0, unit=False, stats=False),
        # the video tokens of a segment, modulated per latent frame
        dict(name="ln_segment", op="ln_fwd", rows=26400, cols=2048, x="bf16", y="bf16", p="bf16", rpg=880, unit=True,
             stats=False),
        # its backward pass: gradients of the tokens and of each frame's modulation
        dict(name="ln_segment_grad", op="ln_bwd", rows=26400, cols=2048, x="bf16", y="bf16", p="bf16", rpg=880, unit=True),
        # text features of an odd width from an fp32 stream, with learned weights: backward pass
        dict(name="ln_text_grad", op="ln_bwd", rows=1280, cols=3581, x="f32", y="bf16", p="f32", rpg=0, unit=False),
        # the six modulation vectors of a block from one timestep embedding
        dict(name="w4_modulation", op="w4", m=1, n=12288, k=2048, group=64, y="bf16"),
        # the same with one embedding per latent frame of a segment
        dict(name="w4_modulation_frames", op="w4", m=30, n=12288, k=2048, group=64, y="bf16"),
        # a down projection of a few tokens (8192 -> 2048), added to an fp32 stream
        dict(name="w4_down", op="w4", m=5, n=2048, k=8192, group=128, y="f32"),
        # a wide projection of a vector pair: the weights' bytes count, not the call
        dict(name="w4_wide", op="w4", m=2, n=28001, k=8192, group=32, y="bf16"),
        # the text tokens of a segment through an up projection
        dict(name="w4_text", op="w4", m=1280, n=8192, k=2048, group=64, y="bf16"),
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "ln_fwd", "ln_bwd", "w4", "w4"])
    if op == "rope":
        heads, dim = rng.choice([1, 2, 3, 8, 16, 24]), rng.choice([64, 128])
        tokens = _spread(rng, 1, min(60000, 26400 * 2048 // (heads * dim)))
        gh, gw = rng.choice([(0, 0), (22, 40), (15, 26), (rng.randint(1, 50), rng.randint(1, 50))])
        return dict(op=op, tokens=tokens, heads=heads, dim=dim, axes=",".join(map(str, rng.choice(AXES[dim]))),
                    dtype=rng.choice(["bf16", "bf16", "f32"]) if tokens * heads * dim < 26400 * 1024 else "bf16",
                    halves=rng.random() < 0.5, adjoint=rng.random() < 0.5, fused=rng.random() < 0.5, grid_h=gh, grid_w=gw)
    if op in ("ln_fwd", "ln_bwd"):
        cols = _spread(rng, 64, 8192)
        cols = cols if rng.random() < 0.3 else max(64, cols // 8 * 8)
        rows = _spread(rng, 1, min(60000, 26400 * 1024 // cols))
        case = dict(op=op, rows=rows, cols=cols, x=rng.choice(["bf16", "f32"]), y=rng.choice(["bf16", "bf16", "f32"]),
                    p=rng.choice(["bf16", "f32"]), rpg=rng.choice([0, _spread(rng, 1, rows)]), unit=rng.random() < 0.5)
        if op == "ln_fwd":
            case["stats"] = rng.random() < 0.5
        return case
    k, n = 32 * _spread(rng, 2, 256), _spread(rng, 16, 16384)
    m = _spread(rng, 1, 1280) if rng.random() < 0.4 else _spread(rng, 1, 64)
    return dict(op=op, m=max(1, min(m, 1280 * 8192 * 2048 // (n * k))), n=n, k=k, group=rng.choice([32, 64, 128]),
                y=rng.choice(["bf16", "bf16", "f32"]))


# ---- inputs -------------------------------------------------------------------------------------------------------

def _axes(case):
    return tuple(int(d) for d in case["axes"].split(","))


def _pairs(case):
    """Channel of each pair's first and second value, its axis, and its turn per unit of position."""
    first, second, axis, freq, at = [], [], [], [], 0
    for a, d in enumerate(_axes(case)):
        for i in range(d // 2):
            first.append(at + (i if case["halves"] else 2 * i))
            second.append(at + (i + d // 2 if case["halves"] else 2 * i + 1))
            axis.append(a)
            freq.append(10000.0 ** (-2.0 * i / d))
        at += d
    return first, second, axis, freq


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 13)

    def randn(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(dtype)

    s = {"case": case}
    if case["op"] == "rope":
        t, h, d, dt = case["tokens"], case["heads"], case["dim"], DTYPES[case["dtype"]]
        if case["fused"]:
            qkv = randn(t, 3, h, d, dtype=dt)
            s["q"], s["k"] = qkv[:, 0], qkv[:, 1]
        else:
            s["q"], s["k"] = randn(t, h, d, dtype=dt), randn(t, h, d, dtype=dt)
        if case["grid_h"]:
            s["positions"] = None
            s["frame0"] = float(seed % 180)             # frames of the rollout before this segment
        else:
            s["positions"] = (torch.rand(t, 3, generator=g, device=dev) * torch.tensor([240.0, 50.0, 50.0], device=dev)).round()
        first, second, axis, freq = _pairs(case)
        s["first"], s["second"] = (torch.tensor(v, device=dev) for v in (first, second))
        s["axis"] = torch.tensor(axis, device=dev)
        s["freq"] = torch.tensor(freq, dtype=torch.float64, device=dev)
        if own:
            from int8_kv_cache_action_b200.runtime import AxisRope, rope_grid
            s["rope"] = AxisRope(d, _axes(case), theta=10000.0, pairing="halves" if case["halves"] else "interleaved")
            s["grid"] = rope_grid(case["grid_h"], case["grid_w"], origin=(s["frame0"], 0.0, 0.0)) if case["grid_h"] else None
    elif case["op"] in ("ln_fwd", "ln_bwd"):
        r, c = case["rows"], case["cols"]
        groups = -(-r // case["rpg"]) if case["rpg"] else 1
        # a residual stream: rows of different size, an offset, a few loud channels
        x = randn(r, c) * torch.exp(randn(r, 1, scale=0.5)) + randn(r, 1)
        x[:, : max(1, c // 50)] *= 8.0
        s["x"] = x.to(DTYPES[case["x"]])
        s["w"] = randn(groups, c, scale=0.3, dtype=DTYPES[case["p"]])
        s["b"] = randn(groups, c, scale=0.3, dtype=DTYPES[case["p"]])
        if case["op"] == "ln_bwd":
            s["dy"] = randn(r, c, dtype=DTYPES[case["y"]])
            s["mean"], s["rstd"] = _stats(s["x"])
    else:
        n, k = case["n"], case["k"]
        s["x"] = randn(case["m"], k, dtype=torch.bfloat16)
        s["codes"] = torch.randint(0, 256, (n, k // 2), generator=g, device=dev, dtype=torch.uint8)
        s["scales"] = (torch.rand(n, -(-k // case["group"]), generator=g, device=dev) * 0.01 + 0.002).to(torch.bfloat16)
        if own:
            from int8_kv_cache_action_b200.runtime import Int4Linear
            s["linear"] = Int4Linear(s["codes"], s["scales"], case["group"])
    return s


# ---- plain forms --------------------------------------------------------------------------------------------------

EPS = 1e-6


def _positions(s):
    case = s["case"]
    if s["positions"] is not None:
        return s["positions"].double()
    n = torch.arange(case["tokens"], device=s["q"].device)
    gw, plane = case["grid_w"], case["grid_h"] * case["grid_w"]
    return torch.stack([s["frame0"] + (n // plane).double(), ((n // gw) % case["grid_h"]).double(), (n % gw).double()], 1)


def _turn(x, s, cos, sin):
    x1, x2 = x[..., s["first"]].float(), x[..., s["second"]].float()
    y = x.clone(memory_format=torch.contiguous_format)
    y[..., s["first"]] = (x1 * cos - x2 * sin).to(x.dtype)
    y[..., s["second"]] = (x1 * sin + x2 * cos).to(x.dtype)
    return y


def _rope_plain(s):
    angle = _positions(s)[:, s["axis"]] * s["freq"]
    if s["case"]["adjoint"]:
        angle = -angle
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    return [_turn(s["q"], s, cos, sin), _turn(s["k"], s, cos, sin)]


def _stats(x):
    x = x.float()
    mean = x.mean(1)
    return mean, torch.rsqrt((x - mean[:, None]).square().mean(1) + EPS)


def _by_row(p, case):
    """The parameter row of every row: [rows][cols], or [1][cols] for one group."""
    p = p.float()
    if not case["rpg"]:
        return p
    return p[torch.arange(case["rows"], device=p.device) // case["rpg"]]


def _ln_fwd_plain(s):
    case = s["case"]
    mean, rstd = _stats(s["x"])
    y = (s["x"].float() - mean[:, None]) * rstd[:, None] * (float(case["unit"]) + _by_row(s["w"], case)) + _by_row(s["b"], case)
    y = y.to(DTYPES[case["y"]])
    return [y, mean, rstd] if case["stats"] else y


def _group_sums(v, case):
    rows, rpg = case["rows"], case["rpg"] or case["rows"]
    groups = -(-rows // rpg)
    if groups * rpg != rows:
        v = torch.cat([v, v.new_zeros(groups * rpg - rows, v.shape[1])])
    return v.view(groups, rpg, -1).sum(1)


def _ln_bwd_plain(s):
    case = s["case"]
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xhat = (s["x"].float() - s["mean"][:, None]) * rstd
    g = dy * (float(case["unit"]) + _by_row(s["w"], case))
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    return [dx.to(DTYPES[case["x"]]), _group_sums(dy * xhat, case), _group_sums(dy, case)]


def _w4_plain(s):
    case = s["case"]
    c = s["codes"]
    codes = torch.stack([c & 15, c >> 4], 2).view(case["n"], case["k"]).float() - 8.0
    scale = s["scales"].float().repeat_interleave(case["group"], 1)[:, : case["k"]]
    w = (codes * scale).to(torch.bfloat16).float()
    return (s["x"].float() @ w.t()).to(DTYPES[case["y"]])


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"rope": _rope_plain, "ln_fwd": _ln_fwd_plain, "ln_bwd": _ln_bwd_plain, "w4": _w4_plain}[op](state)
    from int8_kv_cache_action_b200.runtime import layer_norm, layer_norm_backward
    if op == "rope":
        return list(state["rope"]((state["q"], state["k"]), grid=state["grid"], positions=state["positions"],
                                  inverse=case["adjoint"]))
    if op == "ln_fwd":
        out = layer_norm(state["x"], state["w"], state["b"], eps=EPS, rows_per_group=case["rpg"], unit_offset=case["unit"],
                         out_dtype=DTYPES[case["y"]], want_stats=case["stats"])
        return list(out) if case["stats"] else out
    if op == "ln_bwd":
        return list(layer_norm_backward(state["dy"], state["x"], state["mean"], state["rstd"], state["w"],
                                        rows_per_group=case["rpg"], unit_offset=case["unit"]))
    return state["linear"](state["x"], out_dtype=DTYPES[case["y"]])


# ---- what a pass cannot do without --------------------------------------------------------------------------------

def _size(name):
    return 2 if name == "bf16" else 4


def work(case):
    if case["op"] == "rope":
        values = 2 * case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": 2 * values * _size(case["dtype"]) + (0 if case["grid_h"] else 12 * case["tokens"]), "flops": 3 * values}
    if case["op"] in ("ln_fwd", "ln_bwd"):
        r, c = case["rows"], case["cols"]
        groups = -(-r // case["rpg"]) if case["rpg"] else 1
        moved = r * c * (_size(case["x"]) + _size(case["y"]))
        if case["op"] == "ln_fwd":
            return {"bytes": moved + 2 * groups * c * _size(case["p"]) + (8 * r if case["stats"] else 0), "flops": 8 * r * c}
        return {"bytes": moved + r * c * _size(case["x"]) + groups * c * (_size(case["p"]) + 8) + 8 * r, "flops": 14 * r * c}
    m, n, k = case["m"], case["n"], case["k"]
    return {"bytes": n * k // 2 + 2 * n * -(-k // case["group"]) + 2 * m * k + m * n * _size(case["y"]), "flops": 2 * m * n * k}


# ---- the definitions in 64 bits -----------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        dev = s["q"].device
        if s["positions"] is None:
            frames = -(-case["tokens"] // (case["grid_h"] * case["grid_w"]))
            at = torch.cartesian_prod(*(torch.arange(float(e), dtype=torch.float64, device=dev)
                                        for e in (frames, case["grid_h"], case["grid_w"])))[: case["tokens"]]
            at[:, 0] += s["frame0"]
        else:
            at = s["positions"].double()
        outs = []
        for x in (s["q"].double(), s["k"].double()):
            parts, c0 = [], 0
            for a, d in enumerate(_axes(case)):
                z = x[..., c0:c0 + d]
                z = torch.complex(z[..., : d // 2], z[..., d // 2:]) if case["halves"] else torch.complex(z[..., 0::2], z[..., 1::2])
                i = torch.arange(d // 2, dtype=torch.float64, device=dev)
                turn = at[:, a, None] * torch.exp(-(2.0 * i / max(d, 1)) * math.log(10000.0))
                z = z * torch.polar(torch.ones_like(turn), -turn if case["adjoint"] else turn)[:, None]
                parts.append(torch.cat([z.real, z.imag], -1) if case["halves"] else torch.view_as_real(z).flatten(-2))
                c0 += d
            outs.append(torch.cat(parts + [x[..., c0:]], -1))
        return outs
    if case["op"] in ("ln_fwd", "ln_bwd"):
        x = s["x"].double()
        rows, cols = x.shape
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        rstd = (var + EPS) ** -0.5
        xhat = (x - mean) * rstd
        rpg = case["rpg"] or rows
        sizes = [min(rpg, rows - r) for r in range(0, rows, rpg)]
        count = torch.tensor(sizes, device=x.device)
        weight = s["w"].double().repeat_interleave(count, 0) + (1.0 if case["unit"] else 0.0)
        if case["op"] == "ln_fwd":
            y = xhat * weight + s["b"].double().repeat_interleave(count, 0)
            return [y, mean[:, 0], rstd[:, 0]] if case["stats"] else y
        dy = s["dy"].double()
        g = dy * weight
        dx = (cols * g - g.sum(1, keepdim=True) - xhat * (g * xhat).sum(1, keepdim=True)) * (rstd / cols)
        if len(sizes) > 4000:
            owner = torch.arange(rows, device=x.device) // rpg
            zeros = torch.zeros(len(sizes), cols, dtype=torch.float64, device=x.device)
            return [dx, zeros.index_add(0, owner, dy * xhat), zeros.index_add(0, owner, dy)]
        return [dx, torch.stack([v.sum(0) for v in (dy * xhat).split(sizes)]), torch.stack([v.sum(0) for v in dy.split(sizes)])]
    c = s["codes"].to(torch.int16)
    codes = torch.empty(case["n"], case["k"], dtype=torch.float64, device=c.device)
    codes[:, 0::2], codes[:, 1::2] = (c % 16).double() - 8.0, torch.div(c, 16, rounding_mode="floor").double() - 8.0
    group = torch.arange(case["k"], device=c.device) // case["group"]
    w = (codes * s["scales"].double()[:, group]).to(torch.bfloat16).double()     # code * scale is exact before it
    return s["x"].double() @ w.T
