"""The bf16 GEMM at sizes that take each of its tile widths: 256, 224 and 192 columns on SM pairs, 256 and 128 on
one SM (the width that needs the least time in rounds of tiles), with rows, columns and inner dimensions that end
inside a tile, results next to untouched memory, and the calls captured and on another stream.

Tolerance: an fp32 sum of K products in any order with truncated additions loses at most 2 K 2^-23 of the sum of the
products' sizes; a bf16 result adds half a step, 2^-8 of its size."""
import pytest
import torch

from int8_kv_cache_action_b200 import _nomas as N

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32

# about 148 SMs: one SM 256 and 128; pairs 192, 224, 256 and 192 columns
SHAPES = [(77, 28001, 264), (128, 12285, 328), (129, 8190, 72), (1757, 6141, 200), (9000, 2043, 72), (1280, 8192, 512), (300, 2041, 8)]


def _call(x, w, y):
    st = torch.zeros(4, dtype=torch.int32, device="cuda")
    m, k = x.shape
    stream = torch.cuda.current_stream().cuda_stream
    rc = N.nomas_linear_bf16(x.data_ptr(), m, k, x.stride(0), w.data_ptr(), w.shape[0], w.stride(0), y.data_ptr(), y.stride(0),
                             N.NOMAS_DTYPE_F32 if y.dtype == F32 else N.NOMAS_DTYPE_BF16, st.data_ptr(), stream)
    assert rc == N.NOMAS_OK
    return st


def _inputs(m, n, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(m, k, generator=g, device="cuda").to(BF16), torch.randn(n, k, generator=g, device="cuda").to(BF16))


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_widths_within_the_accumulation_bound(m, n, k, dtype):
    x, w = _inputs(m, n, k, 1)
    buf = torch.full((m + 1, n + 13), 7.0, dtype=dtype, device="cuda")
    st = _call(x, w, buf[:m, :n])
    for r0 in range(0, m, 1024):                              # the 64-bit product in parts
        xs = x[r0:r0 + 1024].double()
        ref, mag = xs @ w.double().t(), xs.abs() @ w.double().abs().t()
        bound = 2.0 * k * 2.0 ** -23 * mag + (2.0 ** -8 * ref.abs() if dtype == BF16 else 0.0) + 1e-30
        assert torch.all((buf[r0:min(m, r0 + 1024), :n].double() - ref).abs() <= bound)
    assert torch.all(buf[:, n:] == 7.0) and torch.all(buf[m] == 7.0)
    assert not st.any()


@pytest.mark.parametrize("m,n,k", [(96, 4096, 128), (640, 8192, 128)])
def test_calls_behind_one_another_see_each_other(m, n, k):
    # the result of a product is the next one's input, in a captured chain: each waits for the one before it
    x, w = _inputs(m, n, k, 2)
    back = (torch.randn(k, n, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda") / 64).to(BF16)
    mid, out = torch.empty((m, n), dtype=BF16, device="cuda"), torch.empty((m, k), dtype=BF16, device="cuda")
    expect = []
    at = x.clone()
    for _ in range(3):
        _call(at, w, mid)
        torch.cuda.synchronize()
        _call(mid, back, out)
        torch.cuda.synchronize()
        at = (out.float() / out.float().abs().max()).to(BF16)
        expect.append(out.clone())
    assert all(torch.isfinite(e.float()).all() for e in expect)
    static = x.clone()
    graph = torch.cuda.CUDAGraph()
    states = []
    with torch.cuda.graph(graph):
        states += [_call(static, w, mid), _call(mid, back, out)]
    for i in range(3):
        if i:
            static.copy_((expect[i - 1].float() / expect[i - 1].float().abs().max()).to(BF16))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, expect[i])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _call(x, w, mid)
        _call(mid, back, out)
    side.synchronize()
    assert torch.equal(out, expect[0]) and not any(s.any() for s in states)


@pytest.mark.parametrize("m,n,k", [(96, 12288, 1024), (640, 8192, 1024), (1300, 6144, 2048)])
def test_products_directly_behind_one_another(m, n, k):
    # nothing stands between the products of a chain: a product is launched as the one that writes its input retires.  All
    # that they need is allocated, and their results are overwritten, before the chain starts
    x, w = _inputs(m, n, k, 4)
    g = torch.Generator(device="cuda").manual_seed(5)
    back = (torch.randn(k, n, generator=g, device="cuda") / (k * n) ** 0.5).to(BF16)
    links, status = 4, torch.zeros(4, dtype=torch.int32, device="cuda")
    bufs = [torch.empty((m, n if i % 2 == 0 else k), dtype=BF16, device="cuda") for i in range(2 * links)]

    def product(x, w, y):
        rc = N.nomas_linear_bf16(x.data_ptr(), m, x.shape[1], x.stride(0), w.data_ptr(), w.shape[0], w.stride(0), y.data_ptr(),
                                 y.stride(0), N.NOMAS_DTYPE_BF16, status.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert rc == N.NOMAS_OK

    def chain(after=lambda: None):
        for i, y in enumerate(bufs):
            product(x if i == 0 else bufs[i - 1], w if i % 2 == 0 else back, y)
            after()

    def overwrite():
        for y in bufs:
            y.fill_(float("nan"))
        torch.cuda.synchronize()

    overwrite()
    chain(torch.cuda.synchronize)
    expect = [y.clone() for y in bufs]
    assert all(torch.isfinite(e).all() for e in expect)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    side = torch.cuda.Stream()

    def aside():
        with torch.cuda.stream(side):
            chain()

    for run in (chain, aside, graph.replay, graph.replay):
        overwrite()
        run()
        torch.cuda.synchronize()
        assert all(torch.equal(y, e) for y, e in zip(bufs, expect))
    assert not status.any()
