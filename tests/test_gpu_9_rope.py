"""Rotary positions through the C ABI against the oracle, element by element.  The bound counts, beside the
one rounding to the type (half a step, eps / 2 relative): the angle, held in fp32 turns after an fp64 reduction
(|angle| <= pi, relative 2^-24), sine and cosine (2 ulp of at most 2^-24 each), two products and a sum: under
2^-20 (|x1| + |x2|) in all."""
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

from int8_kv_cache_action_b200 import _nomas as N
from int8_kv_cache_action_b200.runtime import AxisRope, rope_grid
from oracle import rope as oracle

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _randn(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def _check(y, x, pos, axes, pairing, inverse=False, theta=10000.0):
    halves = pairing == "halves"
    xs = x.float().cpu().numpy()
    ref = oracle.rotate(xs, pos, axes, theta, halves, inverse)
    step = torch.finfo(y.dtype).eps / 2
    slack = 2.0 ** -20 * oracle.partner_abs(xs, axes, halves)
    err = np.abs(y.float().cpu().numpy() - ref)
    turned = slice(0, sum(axes))
    assert np.all((err <= step * (np.abs(ref) + slack) + slack)[..., turned])
    assert torch.equal(y[..., sum(axes):].cpu(), x[..., sum(axes):].cpu())


GRIDS = [(1, 4, 5), (37, 3, 5), (300, 15, 26), (901, 22, 40)]


@pytest.mark.parametrize("tokens,gh,gw", GRIDS)
@pytest.mark.parametrize("pairing", ["interleaved", "halves"])
@pytest.mark.parametrize("dim,axes", [(128, (16, 56, 56)), (64, (16, 24, 24)), (128, (32, 32, 32)), (128, (44, 42, 42)),
                                      (64, (0, 64, 0)), (256, (64, 96, 96)), (72, (8, 32, 30)), (8, (2, 2, 2))])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_grid(tokens, gh, gw, pairing, dim, axes, dtype):
    q, k = _randn((tokens, 6, dim), dtype, 1).cuda(), _randn((tokens, 2, dim), dtype, 2).cuda()
    origin, step = (7.0, -1.5, 0.25), (1.0, 0.5, 2.0)
    yq, yk = AxisRope(dim, axes, pairing=pairing)((q, k), grid=rope_grid(gh, gw, origin, step))
    pos = oracle.grid_positions(tokens, gh, gw, origin, step)
    _check(yq, q, pos, axes, pairing)
    _check(yk, k, pos, axes, pairing)


@pytest.mark.parametrize("pairing", ["interleaved", "halves"])
@pytest.mark.parametrize("heads", [1, 16, 40])
def test_given_positions_far_and_fractional(pairing, heads):
    t = 131
    rng = np.random.default_rng(3)
    pos = np.stack([rng.integers(0, 1 << 24, t), rng.uniform(-300, 300, t), rng.uniform(0, 1, t)], 1).astype(np.float32)
    x = _randn((t, heads, 128), F32, 4).cuda()
    y = AxisRope(128, (16, 56, 56), theta=500.0, pairing=pairing)(x, positions=torch.from_numpy(pos).cuda())
    _check(y, x, pos, (16, 56, 56), pairing, theta=500.0)


@pytest.mark.parametrize("axes,pairing", [((16, 56, 56), "interleaved"), ((32, 48, 48), "halves"), ((44, 42, 42), "halves")])
def test_inverse_is_the_gradient_and_in_place_is_the_same(axes, pairing):
    x = _randn((300, 5, 128), BF16, 5).cuda()
    g = rope_grid(7, 9)
    rope = AxisRope(128, axes, pairing=pairing)
    pos = oracle.grid_positions(300, 7, 9)
    dx = rope(x, grid=g, inverse=True)
    _check(dx, x, pos, axes, pairing, inverse=True)
    again = x.clone()
    assert rope(again, grid=g, inverse=True, out=again) is again
    assert torch.equal(again, dx)
    f = x.float()                                             # <dy, R x> = <R^T dy, x>
    dy = _randn((300, 5, 128), F32, 6).cuda()
    lhs, rhs = (dy.double() * rope(f, grid=g)).sum(), (rope(dy, grid=g, inverse=True).double() * f).sum()
    bound = 2.0 ** -19 * float((dy.abs().sum() * f.abs().max()))
    assert abs(float(lhs - rhs)) <= bound


@pytest.mark.parametrize("pairing,axes", [("interleaved", (16, 56, 56)), ("halves", (32, 48, 32)), ("halves", (16, 40, 56)),
                                          ("halves", (22, 20, 22))])
def test_views_and_untouched_neighbours(pairing, axes):
    t, h, d = 77, 3, 128
    qkv = _randn((t, 3, h, d), BF16, 7).cuda()                # fused projection: q and k are views
    buf = torch.full((h, t + 2, d + 8), 5.0, dtype=BF16, device="cuda")
    out_q = buf[:, 1:t + 1, :d].permute(1, 0, 2)              # [tokens][heads][D] inside a head-major buffer
    out_k = torch.empty((t, h, d), dtype=BF16, device="cuda")
    keep = qkv.clone()
    AxisRope(d, axes, pairing=pairing)((qkv[:, 0], qkv[:, 1]), grid=rope_grid(4, 5), out=(out_q, out_k))
    pos = oracle.grid_positions(t, 4, 5)
    _check(out_q, qkv[:, 0], pos, axes, pairing)
    _check(out_k, qkv[:, 1], pos, axes, pairing)
    assert torch.equal(qkv, keep)
    assert torch.all(buf[:, 0] == 5) and torch.all(buf[:, t + 1:] == 5) and torch.all(buf[..., d:] == 5)
    shared = qkv[:1, 0].expand(t, h, d)                       # one token's values at every position
    y = AxisRope(d, axes, pairing=pairing)(shared, grid=rope_grid(4, 5))
    _check(y, shared, pos, axes, pairing)


@pytest.mark.parametrize("pairing,axes", [("interleaved", (8, 16, 16)), ("interleaved", (6, 14, 18)), ("halves", (16, 16, 16)),
                                          ("halves", (8, 16, 16)), ("halves", (6, 14, 18))])
def test_channels_that_pass_through_keep_every_bit_and_nan_stays_in_its_axis(pairing, axes):
    a, b, c = axes[0], axes[0] + axes[1], sum(axes)
    x = _randn((3, 2, 64), BF16, 8).cuda()
    x[..., c:] = float("inf")
    x[1, 0, c + 1] = float("nan")
    x[0, 1, c + 2] = -0.0
    pos = torch.tensor([[1.0, float("nan"), 2.0], [0.0, 1.0, 3.0], [4.0, 5.0, float("inf")]], device="cuda")
    y = AxisRope(64, axes, pairing=pairing)(x, positions=pos)
    assert torch.equal(y[..., c:].view(torch.int16), x[..., c:].view(torch.int16))
    nan = torch.isnan(y.float()).any(1).cpu()
    assert nan[0, a:b].all() and not nan[0, :a].any() and not nan[0, b:c].any()
    assert nan[2, b:c].all() and not nan[2, :b].any() and not nan[1, :c].any()


def test_offsets_past_32_bits():
    t, stride = 20, (1 << 27) - 64                            # 20 tokens, 5 GB apart in all
    buf = torch.zeros(19 * stride + 512, dtype=BF16, device="cuda")
    x = buf.as_strided((t, 2, 128), (stride, 128, 1))
    x.copy_(_randn((t, 2, 128), BF16, 9).cuda())
    y = AxisRope(128, (16, 56, 56))(x, grid=rope_grid(2, 3))
    _check(y, x, oracle.grid_positions(t, 2, 3), (16, 56, 56), "interleaved")


def test_no_tokens_other_streams_and_a_captured_call():
    rope, g = AxisRope(128, (16, 56, 56)), rope_grid(6, 7)
    assert rope(torch.empty((0, 4, 128), dtype=BF16, device="cuda"), grid=g).shape == (0, 4, 128)
    x = _randn((500, 4, 128), BF16, 10).cuda()
    ref = rope(x, grid=g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = rope(x, grid=g, stream=side)
    side.synchronize()
    assert torch.equal(y, ref)
    graph = torch.cuda.CUDAGraph()
    static = x.clone()
    with torch.cuda.graph(graph):
        out = rope((static, static), grid=g)
    for seed in (11, 12):
        new = _randn((500, 4, 128), BF16, seed).cuda()
        static.copy_(new)
        graph.replay()
        assert torch.equal(out[0], rope(new, grid=g)) and torch.equal(out[1], out[0])


def test_refusals():
    x = torch.zeros((4, 2, 128), dtype=BF16, device="cuda")
    g = rope_grid(2, 2)
    rope = AxisRope(128, (16, 56, 56))
    for bad in (dict(), dict(grid=g, positions=torch.zeros(4, 3, device="cuda")), dict(positions=torch.zeros(3, 3, device="cuda")),
                dict(grid=g, out=torch.zeros((4, 3, 128), dtype=BF16, device="cuda")), dict(grid=g, out=x.float()),
                dict(positions=torch.zeros(4, 3))):
        with pytest.raises(ValueError):
            rope(x, **bad)
    with pytest.raises(ValueError):
        rope(x.cpu(), grid=g)
    with pytest.raises(ValueError):
        rope(x.half(), grid=g)
    for spec in (AxisRope(128, (16, 56, 57)), AxisRope(128, (16, 56, 58)), AxisRope(128, (0, 0, 0)), AxisRope(128, (2, 2, 2), theta=0.0)):
        with pytest.raises(N.NomasError):
            spec(x, grid=g)
    host = torch.zeros((4, 2, 128), dtype=BF16).pin_memory()   # host memory handed to the C call
    args = N.make_rope_tensors([(host.data_ptr(), host.data_ptr(), 256, 128, 256, 128, 2)])
    assert N.nomas_rope(rope.spec, g, 0, 4, args, 1, N.NOMAS_DTYPE_BF16, 0) == N.NOMAS_EINVAL


@pytest.mark.parametrize("pairing", ["interleaved", "halves"])
def test_a_tensor_without_heads_leaves_the_others_turned(pairing):
    rope, g = AxisRope(128, (16, 56, 56), pairing=pairing), rope_grid(2, 3)
    q, none = _randn((9, 16, 128), BF16, 13).cuda(), torch.empty((9, 0, 128), dtype=BF16, device="cuda")
    ref = rope(q, grid=g)
    for xs, at in (((q, none), 0), ((none, q), 1), ((none, q, none), 1)):
        out = tuple(torch.full_like(x, 3.0) for x in xs)
        got = rope(xs, grid=g, out=out)
        assert torch.equal(got[at], ref) and all(y is o for y, o in zip(got, out))
        assert torch.equal(rope(xs, grid=g)[at], ref)
        assert all(y.shape == x.shape for y, x in zip(got, xs))
    assert rope(none, grid=g).shape == none.shape and rope((none, none), grid=g)[1].shape == none.shape


@pytest.mark.parametrize("dtype,pairing", [(F32, "interleaved"), (F32, "halves"), (BF16, "interleaved")])
def test_far_indices_of_a_grid(dtype, pairing):
    # positions up to 1e12, 1.6e11 turns, against 60 digits.  Beside the sines' 2^-20, pair i's turns are off by (1.5 i + 2)
    # 2^-63 of their number (i products and the root's powers, the step's product) and 3000 2^-64 of a turn
    getcontext().prec = 60
    two_pi = Decimal("6.28318530717958647692528676655900576839433879875021164194988918")
    step, origin, t = 1.0e9 / 3.0, -1.0e11 / 7.0, 3001
    x = torch.zeros((t, 1, 16), dtype=dtype, device="cuda")
    first = slice(0, 8) if pairing == "halves" else slice(0, 16, 2)
    second = slice(8, 16) if pairing == "halves" else slice(1, 16, 2)
    x[..., first] = 1.0                                       # y is the cosines and sines themselves
    y = AxisRope(16, (16, 0, 0), pairing=pairing)(x, grid=rope_grid(1, 1, (origin, 0.0, 0.0), (step, 0.0, 0.0)))
    y = y[:, 0].double().cpu().numpy()
    round_off = torch.finfo(dtype).eps / 2
    for n in [0, 1, 2, 3000, *range(7, t, 101)]:
        for i in range(8):
            turns = (Decimal(origin) + n * Decimal(step)) * (-(Decimal(2 * i) / 16) * Decimal(10000).ln()).exp() / two_pi
            size = abs(origin) + n * step
            a = 2 * np.pi * float(turns - turns.to_integral_value())
            slack = 2.0 ** -20 + 2 * np.pi * ((1.5 * i + 2) * 2.0 ** -63 * size * 10000.0 ** (-i / 8) / 6.28 + 3002 * 2.0 ** -64)
            for got, ref in ((y[n, first][i], np.cos(a)), (y[n, second][i], np.sin(a))):
                assert abs(got - ref) <= slack + round_off * (abs(ref) + slack), (n, i)
