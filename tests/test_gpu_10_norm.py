"""Layer norm through the C ABI against the oracle, element by element.  Bounds (u = 2^-24), before the one
rounding to the type (half a step):
  a sum over a row is at most 64 values in a thread and 5 + 16 partial sums: depth below 90;
  mean          off by dm = 90 u mean|x|
  variance      relative 95 u + (dm / sigma)^2, so rstd relative r = 50 u + (dm rstd)^2 / 2
  xhat          off by (dm + 2 u |x - mean|) rstd + |xhat| (r + 2 u)
  y             |f| times that, and 3 u (|xhat f| + |b|)
Backward, with the forward's statistics as given numbers: xhat relative 2 u, g relative 2 u, the row means
95 u of the mean of magnitudes; dw and db: one sum a row of the group, at most (rows + 8) u of the magnitudes."""
import numpy as np
import pytest
import torch

from int8_kv_cache_action_b200 import _nomas as N
from int8_kv_cache_action_b200.runtime import layer_norm, layer_norm_backward
from oracle import norm as oracle

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def _randn(shape, dtype, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).cuda()


def _np(t):
    return None if t is None else t.float().cpu().numpy().astype(np.float64)


def _close(got, ref, slack):
    step = torch.finfo(got.dtype).eps / 2
    err = np.abs(_np(got) - ref)
    assert np.all(err <= step * (np.abs(ref) + slack) + slack + 1e-30), float(np.max(err / (step * np.abs(ref) + slack + 1e-30)))


def _check_forward(x, w, b, rpg, unit, out_dtype, eps=1e-6, **kw):
    y, mean, rstd = layer_norm(x, w, b, eps=eps, rows_per_group=rpg, unit_offset=unit, out_dtype=out_dtype, want_stats=True, **kw)
    xs = _np(x)
    ry, rm, rr = oracle.forward(xs, _np(w), _np(b), eps, rpg, unit)
    dm = 90 * U * np.abs(xs).mean(axis=1)
    r = 50 * U + (dm * rr) ** 2 / 2
    _close(mean, rm, dm)
    _close(rstd, rr, rr * r)
    centred = np.abs(xs - rm[:, None])
    xhat = centred * rr[:, None]
    dx = (dm[:, None] + 2 * U * centred) * rr[:, None] + xhat * (r[:, None] + 2 * U)
    f = np.abs(oracle.factor(_np(w), xs.shape, rpg, unit))
    bias = 0.0 if b is None else np.abs(oracle.factor(_np(b), xs.shape, rpg))
    _close(y, ry, f * dx + 3 * U * (xhat * f + bias))
    return y, mean, rstd


def _check_backward(dy, x, mean, rstd, w, rpg, unit):
    dx, dw, db = layer_norm_backward(dy, x, mean, rstd, w, rows_per_group=rpg, unit_offset=unit)
    m, r = _np(mean), _np(rstd)
    rx, rw, rb = oracle.backward(_np(dy), _np(x), m, r, _np(w), rpg, unit)
    xhat = np.abs((_np(x) - m[:, None]) * r[:, None])
    g = np.abs(_np(dy)) * np.abs(oracle.factor(_np(w), xhat.shape, rpg, unit))
    gx = (g * xhat).mean(axis=1, keepdims=True)
    gm = g.mean(axis=1, keepdims=True)
    slack = np.abs(r[:, None]) * (8 * U * g + 100 * U * gm + 104 * U * xhat * gx)
    _close(dx, rx, slack)
    n = min(rpg or x.shape[0], x.shape[0])
    _close(dw, rw, (n + 8) * U * oracle.group_sums(np.abs(_np(dy)) * xhat, rpg))
    _close(db, rb, (n + 8) * U * oracle.group_sums(np.abs(_np(dy)), rpg))
    return dx, dw, db


SHAPES = [(1, 1), (1, 2048), (3, 8), (5, 7), (700, 64), (2, 16384), (37, 1000), (300, 2048), (33, 1111), (64, 3584),
          (11, 8192), (9, 5003), (900, 40), (7, 16381), (260, 4096)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("xt,yt,pt", [(BF16, BF16, BF16), (BF16, F32, F32), (F32, BF16, BF16), (F32, F32, F32)])
def test_shapes_and_types(rows, cols, xt, yt, pt):
    x = _randn((rows, cols), xt, 1, 2.0) + 0.5
    w, b = _randn((1, cols), pt, 2), _randn((1, cols), pt, 3)
    _, mean, rstd = _check_forward(x, w, b, 0, False, yt)
    _check_backward(_randn((rows, cols), yt, 4), x, mean, rstd, w, 0, False)


@pytest.mark.parametrize("rows,cols,rpg", [(300, 2048, 88), (300, 2048, 1), (1300, 136, 7), (1300, 136, 650), (29, 1111, 10),
                                           (2000, 64, 1999), (641, 520, 128), (50, 2048, 100), (4000, 24, 3)])
@pytest.mark.parametrize("unit", [False, True])
def test_groups(rows, cols, rpg, unit):
    groups = -(-rows // rpg)
    x = _randn((rows, cols), BF16, 5)
    w, b = _randn((groups, cols), BF16, 6, 0.3), _randn((groups, cols), BF16, 7)
    _, mean, rstd = _check_forward(x, w, b, rpg, unit, BF16)
    _check_backward(_randn((rows, cols), BF16, 8), x, mean, rstd, w, rpg, unit)


@pytest.mark.parametrize("cols", [2048, 1001])
def test_without_parameters_and_parts_of_the_gradient(cols):
    x, dy = _randn((50, cols), F32, 9), _randn((50, cols), F32, 10)
    _, mean, rstd = _check_forward(x, None, None, 0, True, F32)
    _check_forward(x, None, _randn((cols,), F32, 11), 0, False, BF16)
    w = _randn((cols,), F32, 12)
    _check_forward(x, w, None, 0, True, F32)
    dx, dw, db = _check_backward(dy, x, mean, rstd, w, 0, False)
    only, none, _ = layer_norm_backward(dy, x, mean, rstd, w, want_params=False)
    assert none is None and torch.equal(only, dx)
    none, ow, ob = layer_norm_backward(dy, x, mean, rstd, w, want_dx=False)
    assert none is None and torch.equal(ow, dw) and torch.equal(ob, db)
    _check_backward(dy, x, mean, rstd, None, 0, True)


def test_rows_far_from_zero_constant_rows_and_loud_channels():
    x = _randn((64, 2048), F32, 13)
    x[0] = 3.0                                             # no variance: y = bias, rstd = 1 / sqrt(eps)
    x[1] += 1.0e4                                          # a mean far above the deviation
    x[2, 5] = 1.0e6
    w, b = _randn((2048,), F32, 14), _randn((2048,), F32, 15)
    y, mean, rstd = _check_forward(x, w, b, 0, False, F32)
    assert torch.equal(y[0], b) and float(mean[0]) == 3.0
    _check_backward(_randn((64, 2048), F32, 16), x, mean, rstd, w, 0, False)


def test_non_finite_rows_stay_alone():
    x = _randn((40, 512), BF16, 17)
    ref = layer_norm(x)
    bad = x.clone()
    bad[3, 7], bad[9, 1] = float("inf"), float("nan")
    y = layer_norm(bad)
    keep = [i for i in range(40) if i not in (3, 9)]
    assert torch.equal(y[keep], ref[keep]) and torch.isnan(y[3]).any() and torch.isnan(y[9]).all()


@pytest.mark.parametrize("cols", [520, 515])
def test_pitches_in_place_and_untouched_neighbours(cols):
    wide = _randn((70, cols + 40), BF16, 18)
    x = wide[:, :cols]
    w = _randn((4, 2 * cols + 16), BF16, 19)[:, :cols]
    buf = torch.full((70, cols + 24), 9.0, dtype=F32, device="cuda")
    out = buf[:, :cols]
    ref, mean, rstd = _check_forward(x, w, w, 20, True, F32)
    assert torch.equal(layer_norm(x, w, w, rows_per_group=20, unit_offset=True, out=out), ref)
    assert torch.all(buf[:, cols:] == 9.0)
    same = x.clone()
    assert torch.equal(layer_norm(same, w, w, rows_per_group=20, unit_offset=True, out=same),
                       layer_norm(x, w, w, rows_per_group=20, unit_offset=True))
    _check_backward(_randn((70, cols + 8), F32, 20)[:, :cols], x, mean, rstd, w, 20, True)


def test_backward_writes_over_its_inputs_and_between_its_rows_nothing():
    x, dy = _randn((90, 2048), BF16, 21), _randn((90, 2048), BF16, 22)
    w = _randn((2048,), BF16, 23)
    _, mean, rstd = layer_norm(x, w, want_stats=True)
    dx, dw, db = layer_norm_backward(dy, x, mean, rstd, w)
    ws = torch.empty(N.nomas_layernorm_workspace_bytes(90, 2048, 0), dtype=torch.uint8, device="cuda")
    grads = torch.full((2, 2100), 4.0, device="cuda")
    for buf, other in ((dy.clone(), x), (x.clone(), dy)):
        ins = (buf, other) if other is x else (other, buf)
        rc = N.nomas_layernorm_bwd(ins[0].data_ptr(), 2048, 1, ins[1].data_ptr(), 2048, 1, 90, 2048, w.data_ptr(), 2048, 1, 0, 0,
                                   mean.data_ptr(), rstd.data_ptr(), buf.data_ptr(), 2048, grads.data_ptr(),
                                   grads[1].data_ptr(), 2100, ws.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert rc == N.NOMAS_OK
        assert torch.equal(buf, dx) and torch.equal(grads[0, :2048], dw[0]) and torch.equal(grads[1, :2048], db[0])
    assert torch.all(grads[:, 2048:] == 4.0)


def test_no_rows():
    x = torch.empty((0, 64), dtype=BF16, device="cuda")
    s = torch.empty(0, device="cuda")
    assert layer_norm(x, want_stats=True)[0].shape == (0, 64)
    dx, dw, db = layer_norm_backward(x, x, s, s)
    assert dx.shape == (0, 64) and torch.all(dw == 0) and torch.all(db == 0) and dw.shape == (1, 64)
    assert layer_norm_backward(x, x, s, s, rows_per_group=4)[1].shape == (0, 64)


def test_same_bits_again_on_two_streams_at_once_and_captured():
    x, dy = _randn((1500, 1032), BF16, 24), _randn((1500, 1032), BF16, 25)
    w = _randn((3, 1032), BF16, 26)
    _, mean, rstd = layer_norm(x, w, rows_per_group=500, want_stats=True)
    ref = layer_norm_backward(dy, x, mean, rstd, w, rows_per_group=500)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [layer_norm_backward(dy, x, mean, rstd, w, rows_per_group=500, stream=s) for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, ref))
    graphs, got = [], []
    for _ in range(2):                                     # two captured graphs, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(layer_norm_backward(dy, x, mean, rstd, w, rows_per_group=500))
        graphs.append(g)
    for _ in range(2):
        for g, o in zip(graphs, got):
            g.replay()
    torch.cuda.synchronize()
    for o in got:
        assert all(torch.equal(a, b) for a, b in zip(o, ref))


def test_rows_past_32_bit_offsets():
    stride = (1 << 26) - 8                                 # 40 rows, 5 GB apart in all
    buf = torch.zeros(39 * stride + 2048, dtype=BF16, device="cuda")
    x = buf.as_strided((40, 1024), (stride, 1))
    x.copy_(_randn((40, 1024), BF16, 27))
    _, mean, rstd = _check_forward(x, None, None, 0, False, BF16)
    _check_backward(x, x, mean, rstd, None, 0, False)


def test_refusals():
    x = torch.zeros((4, 64), dtype=BF16, device="cuda")
    w = torch.zeros(64, device="cuda")
    s = torch.zeros(4, device="cuda")
    for bad in (dict(weight=w[:63]), dict(weight=w.half()), dict(weight=w, bias=w.to(BF16)), dict(weight=w, rows_per_group=2),
                dict(out=torch.zeros((4, 65), device="cuda")), dict(rows_per_group=-1), dict(weight=w.cpu())):
        with pytest.raises(ValueError):
            layer_norm(x, **bad)
    for bad in ((x[:3], x, s, s), (x, x, s[:3], s), (x, x, s, s.double()), (x.cpu(), x, s, s)):
        with pytest.raises(ValueError):
            layer_norm_backward(*bad)
    with pytest.raises(ValueError):
        layer_norm(x.t())
    with pytest.raises(ValueError):
        layer_norm(x.cpu())
    with pytest.raises(N.NomasError):
        layer_norm(torch.zeros((2, N.NOMAS_NORM_MAX_COLS + 1), device="cuda"))
    with pytest.raises(N.NomasError):
        layer_norm(x, eps=-1.0)


def test_expanded_parameters_are_refused():
    x = _randn((8, 64), BF16, 28)
    p = _randn((64,), BF16, 29).expand(4, 64)
    _, mean, rstd = layer_norm(x, want_stats=True)
    for weight, bias in ((p, None), (None, p), (p, p)):
        with pytest.raises(ValueError):
            layer_norm(x, weight, bias, rows_per_group=2)
    with pytest.raises(ValueError):
        layer_norm_backward(x, x, mean, rstd, p, rows_per_group=2)
    _check_forward(x, p.contiguous(), p.contiguous(), 2, True, BF16)


@pytest.mark.parametrize("cols", [71, 72, 1096, 1100, 3000, 3001, 5000, 5001, 9000, 9001])
@pytest.mark.parametrize("xt,yt", [(BF16, BF16), (F32, F32), (F32, BF16)])
def test_backward_of_a_row_whose_mean_times_rstd_overflows(cols, xt, yt):
    # every xhat of the constant row is 0, but (0 - mean) rstd, what padding past the row would have, is -infinity
    x, dy, w = _randn((6, cols), xt, 30), _randn((6, cols), yt, 31), _randn((cols,), F32, 32)
    _, mean, rstd = layer_norm(x, want_stats=True)
    x[2] = 4.0e35
    mean[2], rstd[2] = x[2, 0].float(), 1000.0
    _check_backward(dy, x, mean, rstd, w, 0, False)
    _check_backward(dy, x, mean, rstd, None, 2, True)


def test_a_single_column_of_any_stride():
    def column(seed, dtype=F32):
        return _randn((1, 5), dtype, seed).t()                 # strides (1, 5)
    x, w, out = column(33), column(34)[:3], torch.zeros((1, 5), device="cuda").t()
    y, mean, rstd = _check_forward(x, w, w, 2, False, F32)
    assert torch.equal(layer_norm(x, w, w, rows_per_group=2, out=out), y)
    _check_backward(column(35, BF16), x, mean, rstd, w, 2, False)
