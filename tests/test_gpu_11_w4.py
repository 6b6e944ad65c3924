"""4-bit linear layer through the C ABI against the oracle: codes, scales and bf16 weights bit for bit,
y = x W^T within the fp32 accumulation bound 2 K 2^-23 sum |x| |w| (any order, truncating adds) and, for bf16
outputs, half a step of the result."""
import numpy as np
import pytest
import torch

from int8_kv_cache_action_b200 import _nomas as N
from int8_kv_cache_action_b200.runtime import Int4Linear
from oracle import linear4 as oracle

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _weights(n, k, seed):
    w = torch.randn(n, k, generator=torch.Generator().manual_seed(seed)) * 0.02
    w[:: max(1, n // 7)] *= 30.0
    w[1 % n, :32] = 0.0
    return w.to(BF16)


def _acts(m, k, seed):
    return torch.randn(m, k, generator=torch.Generator().manual_seed(seed)).to(BF16)


def _codes(n, k, group, seed):
    """Every code -8 .. 7, arbitrary scales."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.int32).to(torch.uint8)
    scales = (torch.randn(n, -(-k // group), generator=g) * 0.05).to(BF16)
    return Int4Linear(codes.cuda(), scales.cuda(), group)


def _check(y, x, lin):
    ref, mag = oracle.linear(x.float().cpu().numpy(), oracle.unpack(lin.codes.cpu().numpy()), lin.scales.float().cpu().numpy(), lin.group)
    bound = 2.0 * lin.k_in * 2.0 ** -23 * mag + 1e-30
    if y.dtype == BF16:
        bound = bound + torch.finfo(BF16).eps / 2 * (np.abs(ref) + bound)
    err = np.abs(y.float().cpu().numpy() - ref)
    assert np.all(err <= bound), float(np.max(err / bound))


@pytest.mark.parametrize("n,k,group", [(1, 32, 32), (7, 96, 64), (300, 160, 128), (513, 2048, 64), (40, 1024, 32), (33, 3584, 128)])
def test_quantise_and_dequantise_bit_exact(n, k, group):
    w = _weights(n, k, 1)
    lin = Int4Linear.from_weights(w.cuda(), group)
    q, s = oracle.quantize(w.float().numpy(), group)
    assert np.array_equal(lin.codes.cpu().numpy(), oracle.pack(q))
    assert np.array_equal(lin.scales.float().cpu().numpy().view(np.uint32), s.view(np.uint32))
    assert np.array_equal(lin.dequantized().float().cpu().numpy().view(np.uint32), oracle.dequantize(q, s, group).view(np.uint32))


def test_every_code_times_every_scale_is_rounded_once():
    # all positive and negative finite bf16 scales (their bit patterns), each with the 16 codes
    bits = np.concatenate([np.arange(0, 0x7F80), np.arange(0x8000, 0xFF80)]).astype(np.uint16)
    scales = torch.from_numpy(bits.view(np.int16).copy()).view(BF16)[:, None].cuda()
    codes = torch.tensor([[(i % 8) * 2 | ((i % 8) * 2 + 1) << 4 for i in range(16)]], dtype=torch.uint8).repeat(len(bits), 1).cuda()
    lin = Int4Linear(codes, scales, 32)
    got = lin.dequantized().cpu()
    want = ((torch.tensor([c - 8.0 for c in range(16)] * 2)[None] * scales.cpu().double()).float()).to(BF16)
    assert torch.equal(got, want)                              # an overflow rounds to infinity in both


def test_non_finite_weights_show():
    w = _weights(4, 128, 2)
    w[1, 70], w[2, 3] = float("inf"), float("nan")
    lin = Int4Linear.from_weights(w.cuda(), 64)
    nan = torch.isnan(lin.scales).cpu()
    assert nan.nonzero().tolist() == [[1, 1], [2, 0]]
    y = lin(torch.ones((1, 128), dtype=BF16, device="cuda"))
    assert torch.isnan(y)[0].tolist() == [False, True, True, False]


ROWS = [1, 2, 7, 8, 9, 16, 17, 30, 33, 63, 64, 65, 130, 257]


@pytest.mark.parametrize("m", ROWS)
@pytest.mark.parametrize("n,k,group", [(1, 32, 32), (15, 96, 128), (300, 1056, 64), (520, 2080, 128), (1000, 4096, 32)])
@pytest.mark.parametrize("out_dtype", [F32, BF16])
def test_linear_within_the_accumulation_bound(m, n, k, group, out_dtype):
    x = _acts(m, k, 3).cuda()
    lin = _codes(n, k, group, 4)
    y = lin(x, out_dtype=out_dtype)
    assert lin.status() == N.NOMAS_OK
    _check(y, x, lin)


@pytest.mark.parametrize("m,n,k,group", [(1, 12288, 2048, 64), (30, 12288, 2048, 64), (5, 2048, 8192, 128), (2, 28001, 8192, 32),
                                         (1, 17, 24576, 64), (3, 40000, 64, 64), (64, 64, 16384, 128)])
def test_large(m, n, k, group):
    x = _acts(m, k, 5).cuda()
    lin = _codes(n, k, group, 6)
    _check(lin(x, out_dtype=F32), x, lin)


# tcgen05 tiles: clusters of 1 to 8, ragged rows and columns, a long row whose scales come in parts, idle ranks
@pytest.mark.parametrize("m,n,k,group", [(33, 4100, 2080, 64), (64, 1000, 8416, 32), (100, 4096, 4128, 128), (20, 16500, 4128, 32),
                                         (40, 130, 65568, 64), (128, 2048, 2304, 64), (47, 20000, 448, 128)])
@pytest.mark.parametrize("out_dtype", [F32, BF16])
def test_tiles(m, n, k, group, out_dtype):
    x = _acts(m, k, 16).cuda()
    lin = _codes(n, k, group, 17)
    y = lin(x, out_dtype=out_dtype)
    assert lin.status() == N.NOMAS_OK
    _check(y, x, lin)
    assert torch.equal(lin(x, out_dtype=out_dtype), y)


@pytest.mark.parametrize("m", [5, 40, 100, 300])
@pytest.mark.parametrize("n,k", [(520, 2080), (2050, 8192)])
def test_fp32_results_keep_fp32_precision(m, n, k):
    # runs of at most 1024 columns in the tensor core, truncated: each run's 65 sums lose under 65 2^-23 of the run's largest
    # partial sum, about sqrt(1024 / k) of the result's size, and the rounded sums of the runs far less
    x, lin = _acts(m, k, 20).cuda(), _codes(n, k, 64, 21)
    y = lin(x, out_dtype=F32).double()
    ref = x.double() @ lin.dequantized().double().t()
    assert float((y - ref).norm() / ref.norm()) <= 65 * 2.0 ** -23
    edge = torch.full((m, n + 3), 5.0, device="cuda")
    lin(x, out=edge[:, :n])
    assert torch.equal(edge[:, :n].double(), y) and torch.all(edge[:, n:] == 5.0)


@pytest.mark.parametrize("n,k", [(4096, 4096), (2048, 32768)])          # one and two loads of a CTA's scales
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(n, k):
    x = _acts(64, k, 18).cuda()
    lin = _codes(n, k, 64, 19)
    ref = lin(x)
    prev = N.nomas_set_wait_limit_ns(0)
    try:
        lin(x)
        torch.cuda.synchronize()
        status = lin.status()
    finally:
        N.nomas_set_wait_limit_ns(prev)
    assert status == N.NOMAS_ETIMEOUT
    assert torch.equal(lin(x), ref) and lin.status() == N.NOMAS_OK


def test_each_weight_reaches_its_place():
    # x = rows of the identity: y is the dequantised weights themselves, exactly
    k = 256
    lin = _codes(70, k, 64, 7)
    w = lin.dequantized()
    eye = torch.eye(k, dtype=BF16, device="cuda")
    for c0 in range(0, k, 64):
        assert torch.equal(lin(eye[c0:c0 + 64]), w.t()[c0:c0 + 64])
    assert torch.equal(lin(eye), w.t())


@pytest.mark.parametrize("m", [3, 40, 100])
def test_pitches_and_untouched_neighbours(m):
    k, n = 160, 77
    xb = _acts(m, 2 * k, 8).cuda()
    lin = _codes(n, k, 32, 9)
    buf = torch.full((m, n + 11), 7.0, device="cuda")
    out = buf[:, :n]
    assert lin(xb[:, k:], out=out) is out
    _check(out, xb[:, k:], lin)
    assert torch.all(buf[:, n:] == 7.0)
    edge = torch.full((m + 1, n), 7.0, dtype=BF16, device="cuda")
    lin(xb[:, :k], out=edge[:m])
    _check(edge[:m], xb[:, :k], lin)
    assert torch.all(edge[m] == 7.0)


@pytest.mark.parametrize("m", [2, 20])
def test_rows_of_x_do_not_meet(m):
    lin = _codes(100, 512, 64, 10)
    x = _acts(m, 512, 11).cuda()
    ref = lin(x)
    x[1, 5] = float("nan")
    y = lin(x)
    keep = [i for i in range(m) if i != 1]
    assert torch.equal(y[keep], ref[keep]) and torch.isnan(y[1]).all()


def test_no_rows_streams_and_captured_calls():
    lin = _codes(300, 1024, 64, 12)
    assert lin(torch.empty((0, 1024), dtype=BF16, device="cuda")).shape == (0, 300)
    for m in (4, 200):                                         # few rows, and the GEMM with its own workspace
        x = _acts(m, 1024, 13).cuda()
        ref = lin(x)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        outs = [lin(x, stream=s) for _ in range(4) for s in streams]
        torch.cuda.synchronize()
        assert all(torch.equal(o, ref) for o in outs)
        graph = torch.cuda.CUDAGraph()
        static = x.clone()
        with torch.cuda.graph(graph):
            y = lin(static)
        new = _acts(m, 1024, 14).cuda()
        static.copy_(new)
        graph.replay()
        assert torch.equal(y, lin(new))
    assert lin.status() == N.NOMAS_OK


def test_refusals():
    lin = _codes(16, 64, 32, 15)
    x = torch.zeros((4, 64), dtype=BF16, device="cuda")
    for bad in (x[:, :32], x.float(), x.t(), x.cpu(), x[0]):
        with pytest.raises(ValueError):
            lin(bad)
    for out in (torch.zeros((4, 15), device="cuda"), torch.zeros((4, 16), dtype=torch.float16, device="cuda"), torch.zeros((4, 16))):
        with pytest.raises(ValueError):
            lin(x, out=out)
    for bad in ((lin.codes[:, :8], lin.scales, 32), (lin.codes, lin.scales, 64), (lin.codes, lin.scales, 16),
                (lin.codes, lin.scales.float(), 32), (lin.codes.to(torch.int8), lin.scales, 32)):
        with pytest.raises(ValueError):
            Int4Linear(*bad)
    with pytest.raises(ValueError):
        Int4Linear.from_weights(torch.zeros((4, 48), dtype=BF16, device="cuda"))


@pytest.mark.parametrize("m,n,k,group", [(64, 4096, 4128, 64), (64, 4096, 4160, 128), (100, 1030, 4128, 128), (20, 16500, 4128, 64),
                                         (8, 200, 96, 64), (30, 300, 1056, 128), (200, 2100, 1056, 128)])
@pytest.mark.parametrize("out_dtype", [F32, BF16])
def test_scales_near_the_largest_of_a_last_group_that_columns_end_in(m, n, k, group, out_dtype):
    # codes of at most 4 in size: every weight is at most 2e38 and finite; past column K, 8 times the scale is not
    g = torch.Generator().manual_seed(22)
    c = torch.randint(4, 13, (n, k), generator=g, dtype=torch.int32)
    codes = (c[:, 0::2] | c[:, 1::2] << 4).to(torch.uint8)
    lin = Int4Linear(codes.cuda(), torch.full((n, -(-k // group)), 5.0e37, dtype=BF16, device="cuda"), group)
    x = (torch.randn(m, k, generator=g) * 1e-20).to(BF16).cuda()
    y = lin(x, out_dtype=out_dtype)
    assert lin.status() == N.NOMAS_OK
    _check(y, x, lin)


def test_a_single_row_of_weights_with_any_stride():
    w = _weights(64, 1, 23).cuda().t()                         # [1, 64], strides (1, 1)
    assert w.stride() == (1, 1)
    lin, ref = Int4Linear.from_weights(w, 32), Int4Linear.from_weights(w.reshape(64).clone()[None], 32)
    assert torch.equal(lin.codes, ref.codes) and torch.equal(lin.scales, ref.scales)
    x = _acts(3, 64, 24).cuda()
    _check(lin(x), x, lin)


def test_a_single_column_of_results_with_any_stride():
    lin, x = _codes(1, 96, 32, 25), _acts(5, 96, 26).cuda()
    out = torch.zeros((1, 5), device="cuda").t()
    assert lin(x, out=out) is out and torch.equal(out, lin(x, out_dtype=F32))
