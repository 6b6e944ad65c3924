"""Host checks of the rotary positions, the layer norm and the 4-bit linear layer: every refused argument
returns before any CUDA call, so this runs without a GPU."""
import pytest


@pytest.fixture(scope="module")
def N():
    from int8_kv_cache_action_b200 import build
    build.build()
    from int8_kv_cache_action_b200 import _nomas
    return _nomas


A = 0x10000                                                  # 16-byte aligned stand-in address, never read


def test_rope_refusals(N):
    def call(spec=None, grid="grid", positions=0, tokens=4, tensor=None, n=1, dtype=1):
        spec = N.make_rope_spec(*(spec or (128, (16, 56, 56))))
        grid = N.make_rope_grid(2, 2) if grid == "grid" else grid
        t = dict(x=A, y=A, xt=256, xh=128, yt=256, yh=128, heads=2)
        t.update(tensor or {})
        return N.nomas_rope(spec, grid, positions, tokens, N.make_rope_tensors([tuple(t.values())] * max(n, 1)), n, dtype, 0)
    assert call(tokens=0) == N.NOMAS_OK
    for spec in ((120 + 4, (16, 56, 56)), (264, (16, 56, 56)), (0, (0, 0, 0)), (128, (16, 56, 58)), (128, (15, 1, 2)), (128, (0, 0, 0)),
                 (128, (-2, 4, 4)), (128, (2, 2, 2), 0.0), (128, (2, 2, 2), float("nan")), (128, (2, 2, 2), float("inf")),
                 (128, (2, 2, 2), 100.0, 2)):
        assert call(spec=spec) == N.NOMAS_EINVAL, spec
    for kw in (dict(grid=None), dict(positions=A), dict(grid=None, positions=A + 2), dict(tokens=-1), dict(n=0), dict(n=5), dict(dtype=2),
               dict(grid=N.make_rope_grid(0, 2)), dict(grid=N.make_rope_grid(1 << 16, 1 << 15)),
               dict(grid=N.make_rope_grid(2, 2, (float("nan"), 0, 0))), dict(grid=N.make_rope_grid(2, 2, step=(1, float("inf"), 1)))):
        assert call(**kw) == N.NOMAS_EINVAL, kw
    for t in (dict(x=0), dict(y=0), dict(x=A + 8), dict(heads=0), dict(xt=260), dict(xh=-8), dict(y=A + 16, yh=64), dict(y=A + 16, yt=0),
              dict(y=A + 16, yt=128, yh=192),                   # y's tokens and heads meet
              dict(yt=512)):                                    # in place with other strides
        assert call(tensor=t) == N.NOMAS_EINVAL, t
    assert call(n=2) == N.NOMAS_EINVAL                           # two results in one place
    assert call(n=2, tensor=dict(y=A + 16)) == N.NOMAS_EINVAL
    spec, grid = N.make_rope_spec(128, (16, 56, 56)), N.make_rope_grid(2, 2)
    first = (A, A + 16, 256, 128, 256, 128, 2)
    for x, y in ((A + 16, A + 32), (A + 32, A)):                # the second reads the first one's result, writes what it reads
        pair = N.make_rope_tensors([first, (x, y, 256, 128, 256, 128, 2)])
        assert N.nomas_rope(spec, grid, 0, 4, pair, 2, N.NOMAS_DTYPE_BF16, 0) == N.NOMAS_EINVAL
    assert call(spec=(128, (2, 2, 64), 1e-300), grid=N.make_rope_grid(2, 2, (0, 0, 1e300))) == N.NOMAS_EINVAL
    assert call(tokens=1 << 31) == N.NOMAS_EUNSUPPORTED


def test_layernorm_refusals(N):
    fwd = dict(x=A, rows=4, cols=64, ldx=64, xt=1, w=A, b=A, ldp=64, pt=1, rpg=0, unit=0, eps=1e-6, y=A + 4096, ldy=64, yt=1)
    bwd = dict(dy=A, lddy=64, yt=1, x=A, ldx=64, xt=1, rows=4, cols=64, w=A, ldp=64, pt=1, rpg=0, unit=0, mean=A, rstd=A, dx=A + 4096,
               lddx=64, dw=A, db=A, ldg=64, ws=A)
    f = lambda **kw: N.nomas_layernorm_fwd(*{**fwd, **kw}.values())          # noqa: E731
    g = lambda **kw: N.nomas_layernorm_bwd(*{**bwd, **kw}.values())          # noqa: E731
    assert f(rows=0) == N.NOMAS_OK
    for kw in (dict(x=0), dict(y=0), dict(x=A + 1), dict(xt=2), dict(yt=-1), dict(pt=7), dict(rows=-1), dict(cols=0), dict(ldx=63), dict(ldy=63),
               dict(ldp=63), dict(w=A + 1), dict(rpg=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(y=A, yt=0), dict(y=A, ldy=72)):
        assert f(**kw) == N.NOMAS_EINVAL, kw
    for kw in (dict(dy=0), dict(x=0), dict(mean=0), dict(rstd=0), dict(dx=0, dw=0, db=0), dict(lddx=63), dict(ldg=63), dict(rows=4096, ws=0),
               dict(ws=A + 8), dict(dw=A + 2), dict(rpg=-1), dict(lddy=63), dict(dx=A, lddx=72), dict(dx=A, yt=0)):
        assert g(**kw) == N.NOMAS_EINVAL, kw
    assert f(cols=N.NOMAS_NORM_MAX_COLS + 1) == N.NOMAS_EUNSUPPORTED and g(rows=1 << 31) == N.NOMAS_EUNSUPPORTED
    assert N.nomas_layernorm_workspace_bytes(4, 0, 0) == 0 and N.nomas_layernorm_workspace_bytes(0, 8, 0) >= 16


def test_w4_refusals(N):
    ok = dict(x=A, m=4, k=64, ldx=64, codes=A, scales=A, group=64, n=16, y=A, ldy=16, yt=0, ws=0, st=A)
    call = lambda **kw: N.nomas_w4a16_linear(*{**ok, **kw}.values())         # noqa: E731
    assert call(m=0) == N.NOMAS_OK
    for kw in (dict(x=0), dict(x=A + 2), dict(m=-1), dict(k=48, ldx=48), dict(k=0), dict(ldx=56), dict(ldx=68), dict(codes=0), dict(codes=A + 8),
               dict(scales=0), dict(scales=A + 2), dict(group=16), dict(group=96), dict(n=0), dict(y=0), dict(ldy=15), dict(yt=2), dict(st=0),
               dict(m=1000, n=1 << 16, ldy=1 << 16), dict(m=1000, n=1 << 16, ldy=1 << 16, ws=A + 4)):
        assert call(**kw) == N.NOMAS_EINVAL, kw
    assert N.nomas_w4a16_workspace_bytes(1, 4096, 4096) == 0
    assert N.nomas_w4a16_workspace_bytes(1000, 4096, 2048) == 4096 * 2048 * 2
    assert N.nomas_w4a16_workspace_bytes(1000, 4095, 2048, N.NOMAS_DTYPE_F32) == 4095 * 2048 * 2 + 2 * 1000 * 4096 * 4
    assert N.nomas_w4a16_workspace_bytes(1000, 4096, 1024, N.NOMAS_DTYPE_F32) == 4096 * 1024 * 2
    for size in ((0, 4096, 2048), (1000, 0, 2048), (1000, 4096, 2040), (1000, 1 << 31, 64), (1 << 31, 4096, 2048)):
        assert N.nomas_w4a16_workspace_bytes(*size) == 0
    assert N.nomas_w4_quantize(0, 16, 64, 64, 64, A, A) == N.NOMAS_EINVAL
    assert N.nomas_w4_quantize(A, 16, 64, 63, 64, A, A) == N.NOMAS_EINVAL
    assert N.nomas_w4_dequant(A, A, 64, 16, 64, A + 8) == N.NOMAS_EINVAL


def test_layernorm_parameter_rows_that_overlap_are_refused(N):
    # a group's row is read at its pitch from the first, so an expanded row (stride 0) must never reach a launch
    import torch
    from int8_kv_cache_action_b200.runtime import _norm_params
    x, row = torch.zeros((8, 64)), torch.zeros(64)
    expanded, overlapping = row.expand(4, 64), torch.zeros(4 * 63 + 1).as_strided((4, 64), (63, 1))
    for p in (expanded, overlapping):
        for weight, bias in ((p, None), (None, p), (p, p)):
            with pytest.raises(ValueError):
                _norm_params(x, weight, bias, 2)
    assert _norm_params(x, row.expand(1, 64), row, 0) == (64, N.NOMAS_DTYPE_F32, 1)      # one group: its only row
    views = torch.zeros((4, 128), dtype=torch.bfloat16)
    assert _norm_params(x, views[:, 64:], views[:, :64], 2) == (128, N.NOMAS_DTYPE_BF16, 4)
    assert _norm_params(x, None, None, 2) == (64, N.NOMAS_DTYPE_F32, 4)
    assert _norm_params(x[:0], expanded[:0], None, 2)[2] == 0


def test_a_single_column_has_contiguous_rows(N):
    import torch
    from int8_kv_cache_action_b200.runtime import _norm_params
    column = torch.zeros((1, 5)).t()                          # [5, 1], contiguous, strides (1, 5)
    assert column.is_contiguous() and column.stride(1) == 5
    assert _norm_params(column, None, None, 0) == (1, N.NOMAS_DTYPE_F32, 1)
    assert _norm_params(column, column[:3], column[:3], 2) == (1, N.NOMAS_DTYPE_F32, 3)
    for bad in (torch.zeros((5, 4)).t(), torch.zeros((5, 8))[:, ::2]):
        with pytest.raises(ValueError):
            _norm_params(bad, None, None, 0)
    with pytest.raises(ValueError):
        _norm_params(column, torch.zeros(1).expand(3, 1), None, 2)
