"""The operators together, as a DiT block runs them in front of its attention: frame embeddings -> 4-bit linear
layer (modulation) -> layer norm modulated per frame -> INT8 linear layer (QKV) -> rotary positions in the QKV
buffer -> append of a finished segment and attention of the next.  Each stage is checked against its oracle on
the values that reached it, all on views of the stage before and without a synchronise in between; the same run
is captured and replayed on new inputs.  And the gradient of norm and rotation together, against fp64 autograd."""
import math

import numpy as np
import pytest
import torch

from int8_kv_cache_action_b200.runtime import (AxisRope, Int4Linear, Int8Linear, KVCache, layer_norm, layer_norm_backward,
                                               rope_grid, segment_text)
from int8_kv_cache_action_b200.workloads import SegmentText, Tail
from oracle import attention as att
from oracle import linear as ol
from oracle import linear4 as ol4
from oracle import norm as onorm
from oracle import rope as orope
from oracle.ring import OracleCache
from tests.helpers import TOL_MAX_ABS, TOL_MEAN_REL, attention_errors

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
GH, GW, F, H, D, C, AXES = 5, 7, 3, 2, 128, 320, (16, 56, 56)
T = GH * GW
U = 2.0 ** -24


def _randn(shape, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(BF16).cuda()


def _np(t):
    return t.float().cpu().numpy()


class Block:
    def __init__(self):
        self.mod = Int4Linear.from_weights(_randn((2 * C, 96), 1, 0.05), group=32)
        self.qkv = Int8Linear.from_weights(_randn((3 * H * D, C), 2, 0.05))
        self.rope = AxisRope(D, AXES)

    def __call__(self, x, emb, frame0):
        """x [F T, C], emb [F, 96] -> (modulation, normed, q, k, v before rotation, the buffer after it)."""
        mod = self.mod(emb)
        y = layer_norm(x, mod[:, C:], mod[:, :C], rows_per_group=T, unit_offset=True)
        buf = self.qkv(y).view(x.shape[0], 3, H, D)
        before = buf.clone()
        self.rope((buf[:, 0], buf[:, 1]), grid=rope_grid(GH, GW, origin=(frame0, 0.0, 0.0)), out=(buf[:, 0], buf[:, 1]))
        return mod, y, before, buf


def test_block_in_front_of_the_attention():
    block = Block()
    gc, oc = KVCache(H, D, T, 4, 4, 0), OracleCache(H, D, T, 4, 4, 0)
    seg = segment_text(F, 6, [(4, 0, 2)])
    x = [_randn((F * T, C), 10 + i, 2.0) for i in range(2)]
    emb = [_randn((F, 96), 20 + i) for i in range(2)]
    ktxt, vtxt = _randn((10, 3, H, D), 30)[:, 1], _randn((10, 3, H, D), 31)[:, 2]     # strides of the QKV buffer
    done = block(x[0], emb[0], 0.0)
    gc.append(done[3][:, 1], done[3][:, 2], F)
    now = block(x[1], emb[1], float(F))
    q, k, v = now[3].unbind(1)
    mask, _ = gc.build_mask(seg, q=q, kcur=k)
    out, _ = gc.attention(seg, mask, q, k, v, ktxt, vtxt, 1.0 / math.sqrt(D))
    torch.cuda.synchronize()
    assert gc.status() == 0 and block.mod.status() == 0 and block.qkv.status() == 0

    for (mod, y, before, buf), xi, e, frame0 in ((done, x[0], emb[0], 0.0), (now, x[1], emb[1], float(F))):
        ref, mag = ol4.linear(_np(e), ol4.unpack(block.mod.codes.cpu().numpy()), _np(block.mod.scales), 32)
        bound = 2 * 96 * 2.0 ** -23 * mag
        assert np.all(np.abs(_np(mod) - ref) <= bound + 2.0 ** -8 * (np.abs(ref) + bound))
        m = _np(mod)
        ref, mean, rstd = onorm.forward(_np(xi), m[:, C:], m[:, :C], 1e-6, T, True)
        xhat = np.abs(_np(xi) - mean[:, None]) * rstd[:, None]
        slack = 300 * U * (1 + xhat) * np.abs(onorm.factor(m[:, C:], ref.shape, T, True)) + 8 * U * np.abs(ref)
        assert np.all(np.abs(_np(y) - ref) <= 2.0 ** -8 * (np.abs(ref) + slack) + slack)
        ref = ol.linear(_np(y), block.qkv.codes.cpu().numpy(), block.qkv.scales.cpu().numpy())
        mag = ol.abs_product_sum(_np(y), block.qkv.codes.cpu().numpy(), block.qkv.scales.cpu().numpy())
        bound = 2 * C * 2.0 ** -23 * mag
        assert np.all(np.abs(_np(before).reshape(ref.shape) - ref) <= bound + 2.0 ** -8 * (np.abs(ref) + bound))
        pos = orope.grid_positions(F * T, GH, GW, (frame0, 0.0, 0.0))
        for j in range(2):
            b = _np(before[:, j])
            ref, slack = orope.rotate(b, pos, AXES), 2.0 ** -20 * orope.partner_abs(b, AXES)
            assert np.all(np.abs(_np(buf[:, j]) - ref) <= 2.0 ** -8 * (np.abs(ref) + slack) + slack)
        assert torch.equal(buf[:, 2], before[:, 2])
    oc.append(_np(done[3][:, 1]), _np(done[3][:, 2]), F, None, None)
    ref, _ = att.attention(oc, _np(q), _np(k), _np(v), _np(ktxt), _np(vtxt), SegmentText(F, 6, (Tail(4, 0, 2),)),
                           1.0 / math.sqrt(D))
    worst, mean_rel = attention_errors(out.cpu().numpy(), ref)
    assert worst <= TOL_MAX_ABS and mean_rel <= TOL_MEAN_REL


def test_captured_block_replays_on_new_inputs():
    block = Block()
    x, emb = _randn((F * T, C), 40), _randn((F, 96), 41)
    block(x, emb, 2.0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block(x, emb, 2.0)
    for seed in (42, 43):
        nx, ne = _randn((F * T, C), seed, 3.0), _randn((F, 96), seed + 10)
        x.copy_(nx)
        emb.copy_(ne)
        graph.replay()
        for a, b in zip(out, block(nx, ne, 2.0)):
            assert torch.equal(a, b)


def test_gradient_of_norm_and_rotation_together():
    n = F * T
    x = torch.randn((n, H * D), generator=torch.Generator().manual_seed(50)).cuda()
    w, b = (torch.randn((F, H * D), generator=torch.Generator().manual_seed(s)).cuda() for s in (51, 52))
    dy = torch.randn((n, H, D), generator=torch.Generator().manual_seed(53)).cuda()
    rope, grid = AxisRope(D, AXES, pairing="halves"), rope_grid(GH, GW)
    y, mean, rstd = layer_norm(x, w, b, rows_per_group=T, unit_offset=True, want_stats=True)
    rope(y.view(n, H, D), grid=grid)
    dz = rope(dy, grid=grid, inverse=True).view(n, H * D)
    grads = layer_norm_backward(dz, x, mean, rstd, w, rows_per_group=T, unit_offset=True)

    xs, ws, bs = (t.double().cpu().requires_grad_() for t in (x, w, b))
    rows = torch.arange(n) // T
    xc = xs - xs.mean(1, keepdim=True)
    z = (xc * torch.rsqrt(xc.square().mean(1, keepdim=True) + 1e-6) * (1 + ws[rows]) + bs[rows]).view(n, H, D)
    pos = torch.from_numpy(orope.grid_positions(n, GH, GW))
    parts, c0 = [], 0
    for a, d in enumerate(AXES):
        ang = (pos[:, a, None] * 10000.0 ** (-2.0 * torch.arange(d // 2, dtype=torch.float64) / d))[:, None]
        z1, z2 = z[..., c0:c0 + d // 2], z[..., c0 + d // 2:c0 + d]
        parts += [z1 * ang.cos() - z2 * ang.sin(), z1 * ang.sin() + z2 * ang.cos()]
        c0 += d
    (torch.cat(parts, -1) * dy.double().cpu()).sum().backward()
    # fp32 throughout: rotation under 2^-20 of a pair, norm under 200 roundings of the row's largest terms
    for got, ref, depth in zip(grads, (xs.grad, ws.grad, bs.grad), (H * D, T, T)):
        got, ref = got.double().cpu(), ref
        scale = ref.abs().amax(1, keepdim=True) + ref.abs().mean()
        assert bool(((got - ref).abs() <= 2.0 ** -17 * scale).all()), float(((got - ref).abs() / scale).max())
