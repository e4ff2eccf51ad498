"""rms_norm and its gradient on the GPU: against the definition in 64 bits, and
outputs of 8 bits code for code."""
import math

import pytest
import torch

import mixed_precision_dense_tiled_amd as mp
from layers_ref import HALF, TINY, U, norm_backward, norm_rows, norm_rstd, norm_sum, quantise

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]
# every width of the kernels, both ends of each, odd ones
DIMS = [1, 2, 7, 8, 9, 63, 64, 100, 128, 129, 511, 512, 513, 1000, 1024, 1025, 2047, 2048, 2049, 4096, 4097, 5120,
        8191, 8192, 8200, 16384, 16385, 32767, 32768]


def rows_like(rows, dim, dtype, seed, pad=0, shift=0):
    """Strided, unaligned rows of a larger buffer of NaN, and the buffer."""
    g = torch.Generator().manual_seed(seed)
    buf = torch.full((rows * (dim + pad) + shift + 8,), float("nan"), dtype=dtype)
    view = buf[shift:shift + rows * (dim + pad)].view(rows, dim + pad)[:, :dim]
    view.copy_(torch.randn((rows, dim), generator=g))
    gpu = buf.cuda()
    return gpu[shift:shift + rows * (dim + pad)].view(rows, dim + pad)[:, :dim], view


def near(got, want, off, dtype):
    err = (got.cpu().double() - want).abs()
    bound = off + HALF[dtype] * want.abs() * (1 + 2.0 ** -7) + TINY[dtype]
    assert (err <= bound).all(), (err - bound).max()


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("dtype", TYPES)
def test_plain(dtype, dim):
    rows = 5 if dim < 5000 else 2
    for pad, shift, w_type, res in ((0, 0, dtype, True), (3, 1, torch.float32, False)):
        x, xc = rows_like(rows, dim, dtype, dim + pad, pad, shift)
        r, rc = rows_like(rows, dim, dtype, dim + pad + 1, pad, shift) if res else (None, None)
        w = (1 + 0.3 * torch.randn(dim, generator=torch.Generator().manual_seed(dim))).to(w_type)
        got = mp.rms_norm(x, w.cuda(), eps=1e-5, residual=r, return_rstd=True)
        h = norm_sum(xc, rc)
        if res:
            assert torch.equal(got.residual.cpu(), h)
        else:
            assert got.residual is None
        assert got.scales is None and torch.equal(got.rstd.cpu(), norm_rstd(h, 1e-5))
        y = h.double() * (h.double().square().mean(-1, keepdim=True) + 1e-5).rsqrt() * w.double()
        near(got.out, y, 3 * U * y.abs(), dtype)
        assert torch.equal(got.out.cpu(), norm_rows(h, w, 1e-5).to(dtype))


@pytest.mark.parametrize("quant", ["int8", "fp8_rows", "fp8_blocks"])
@pytest.mark.parametrize("dim", DIMS)
def test_codes(quant, dim):
    for dtype, pad, shift, res in ((torch.bfloat16, 0, 0, True), (torch.float16, 5, 1, False),
                                   (torch.float32, 0, 0, True)):
        x, xc = rows_like(3, dim, dtype, dim, pad, shift)
        r, rc = rows_like(3, dim, dtype, dim + 1, pad, shift) if res else (None, None)
        w = torch.randn(dim, generator=torch.Generator().manual_seed(dim)).to(dtype)
        got = mp.rms_norm(x, w.cuda(), residual=r, quant=quant)
        values, scales = quantise(norm_rows(norm_sum(xc, rc), w, 1e-6), quant)
        codes = got.out.cpu() if quant == "int8" else got.out.cpu().view(torch.float8_e4m3fn)
        assert torch.equal(got.scales.cpu(), scales)
        assert torch.equal(codes.float(), values)


@pytest.mark.parametrize("quant", [None, "int8", "fp8_rows", "fp8_blocks"])
def test_numbers_that_are_none(quant):
    """Rows of zeros, NaN and infinities; a row beside them is as it is alone."""
    dim = 300
    x = torch.randn((5, dim), generator=torch.Generator().manual_seed(1))
    x[0] = 0
    x[1, 140] = float("nan")
    x[2, 5] = float("inf")
    x[3] = torch.linspace(-1e-38, 1e-38, dim)
    w = torch.ones(dim)
    w[7] = 0
    got = mp.rms_norm(x.cuda(), w.cuda(), eps=1e-6, quant=quant)
    y = norm_rows(x, w, 1e-6)
    if quant is None:
        assert torch.equal(got.out.cpu().nan_to_num(7.5), y.nan_to_num(7.5))
        return
    values, scales = quantise(y, quant)
    codes = got.out.cpu().float() if quant == "int8" else got.out.cpu().view(torch.float8_e4m3fn).float()
    assert torch.equal(got.scales.cpu().nan_to_num(-1), scales.nan_to_num(-1))
    assert torch.equal(codes.nan_to_num(999), values.nan_to_num(999))
    assert got.scales[0].eq(1).all() and got.scales[1].isnan().all()


@pytest.mark.parametrize("dim", [2560, 4096, 5120, 6144, 6150, 8192])
def test_many_rows(dim):
    """More rows than CUs: as in few."""
    w = (1 + 0.3 * torch.randn(dim, generator=torch.Generator().manual_seed(6))).cuda()
    x, r = rows_like(600, dim, torch.bfloat16, 1, 0, 0)[0], rows_like(600, dim, torch.bfloat16, 2, 0, 0)[0]
    for quant in (None, "int8", "fp8_rows", "fp8_blocks"):
        many = mp.rms_norm(x, w, residual=r, quant=quant)
        few = [mp.rms_norm(x[i:i + 200], w, residual=r[i:i + 200], quant=quant) for i in (0, 200, 400)]
        assert torch.equal(many.out, torch.cat([f.out for f in few]))
        assert torch.equal(many.residual, torch.cat([f.residual for f in few]))
        if quant is not None:
            assert torch.equal(many.scales, torch.cat([f.scales for f in few]))


def test_in_place_and_apart():
    """x and residual updated in place; buffers around the rows stay."""
    dim, rows, dtype = 1000, 7, torch.bfloat16
    w = torch.randn(dim, generator=torch.Generator().manual_seed(5)).to(dtype)
    want = None
    for where in ("new", "residual", "x"):
        x, xc = rows_like(rows, dim, dtype, 1, 8, 0)
        r, rc = rows_like(rows, dim, dtype, 2, 8, 0)
        big = torch.full((rows + 2, dim + 4), 3.0, dtype=dtype, device="cuda")
        out = {"new": big[1:-1, 2:-2], "residual": x, "x": r}[where]
        res = {"new": None, "residual": r, "x": x}[where]
        got = mp.rms_norm(x, w.cuda(), residual=r, out=out, residual_out=res)
        h = norm_sum(xc, rc)
        want = norm_rows(h, w, 1e-6).to(dtype) if want is None else want
        assert got.out is out and torch.equal(out.cpu(), want) and torch.equal(got.residual.cpu(), h)
        if where == "new":
            big[1:-1, 2:-2] = 3.0
            assert (big == 3.0).all()


def test_far_sizes():
    """Values whose squares leave FP32, and a weight that brings them back."""
    x = torch.tensor([[3e37, -1e37, 2e37, 0.0], [1e-30, 2e-30, -3e-30, 0.0]])
    w = torch.tensor([1.0, 2.0, 3.0, 4.0])
    got = mp.rms_norm(x.cuda(), w.cuda(), eps=0.0).out.cpu()
    h = x.double()
    y = h * h.square().mean(-1, keepdim=True).rsqrt() * w.double()
    near(got, y, 3 * U * y.abs(), torch.float32)


def test_no_rows_and_more_rows_than_groups():
    w = torch.ones(64, device="cuda")
    got = mp.rms_norm(torch.empty((0, 64), device="cuda"), w, quant="fp8_blocks", return_rstd=True)
    assert got.out.shape == (0, 64) and got.scales.shape == (0, 1) and got.rstd.shape == (0,)
    gh, gw = mp.rms_norm_backward(torch.empty((0, 64), device="cuda"), torch.empty((0, 64), device="cuda"), w,
                                  torch.empty(0, device="cuda"))
    assert gh.shape == (0, 64) and torch.equal(gw, torch.zeros_like(gw))
    x = torch.randn((70001, 64), generator=torch.Generator().manual_seed(3))
    got = mp.rms_norm(x.cuda(), w).out.cpu()
    assert torch.equal(got, norm_rows(x, torch.ones(64), 1e-6))


@pytest.mark.parametrize("dim", [1, 7, 8, 100, 512, 513, 2048, 2050, 4096, 4100, 8192, 9001, 16384, 32768])
@pytest.mark.parametrize("dtype", TYPES)
def test_backward(dtype, dim):
    for rows, pad, shift, w_type, res in ((1, 0, 0, dtype, False), (6, 3, 1, torch.float32, True),
                                          (1500 if dim <= 513 else 9, 0, 0, dtype, True)):
        h, hc = rows_like(rows, dim, dtype, dim, pad, shift)
        g, gc = rows_like(rows, dim, dtype, dim + 1, pad, shift)
        r, rc = rows_like(rows, dim, dtype, dim + 2, pad, shift) if res else (None, None)
        w = (1 + 0.3 * torch.randn(dim, generator=torch.Generator().manual_seed(dim))).to(w_type)
        rstd = norm_rstd(hc, 1e-6)
        gh, gw = mp.rms_norm_backward(g, h, w.cuda(), rstd.cuda(), grad_residual=r)
        dh, off, dw, off_w = norm_backward(gc, hc, w, rstd, rc)
        near(gh, dh, off, dtype)
        assert gw.dtype == torch.float32
        assert ((gw.cpu().double() - dw).abs() <= off_w + 2.0 ** -149).all()
        again = mp.rms_norm_backward(g, h, w.cuda(), rstd.cuda(), grad_residual=r)
        assert torch.equal(again[0], gh) and torch.equal(again[1], gw)
        # in place of the gradient
        mp.rms_norm_backward(g, h, w.cuda(), rstd.cuda(), grad_residual=r, out=g)
        assert torch.equal(g, gh)


@pytest.mark.parametrize("rows, dim", [(2500, 513), (5000, 1001), (3300, 1500), (1601, 2200), (1600, 5000), (800, 9001),
                                       (300, 32768)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_backward_many_rows(dtype, rows, dim):
    """More rows than are held at a time."""
    (h, hc), (g, gc), (r, rc) = (rows_like(rows, dim, dtype, dim + i, 0, 0) for i in range(3))
    w = (1 + 0.3 * torch.randn(dim, generator=torch.Generator().manual_seed(dim))).to(dtype)
    rstd = norm_rstd(hc, 1e-6)
    gh, gw = mp.rms_norm_backward(g, h, w.cuda(), rstd.cuda(), grad_residual=r, out=g)
    dh, off, dw, off_w = norm_backward(gc, hc, w, rstd, rc)
    near(gh, dh, off, dtype)
    assert ((gw.cpu().double() - dw).abs() <= off_w + 2.0 ** -149).all()


def test_backward_against_differences():
    """The gradient along a direction, from outputs of the forward kernel at both sides."""
    rows, dim, step = 3, 96, 2.0 ** -8
    g = torch.Generator().manual_seed(11)
    x, d, up, w = (torch.randn((rows, dim), generator=g) for _ in range(4))
    w = 1 + 0.2 * w[0]
    dw = torch.randn(dim, generator=g)

    def loss64(a, b):
        a, b = a.double(), b.double()
        return (up.double() * a * (a.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * b).sum()

    def loss(a, b):
        y = mp.rms_norm(a.cuda(), b.cuda(), eps=1e-6).out.cpu().double()
        return (up.double() * y).sum(), (up.double() * y).abs().sum()

    f = mp.rms_norm(x.cuda(), w.cuda(), return_rstd=True)
    gh, gw = (t.cpu().double() for t in mp.rms_norm_backward(up.cuda(), x.cuda(), w.cuda(), f.rstd))
    dh, off, _, off_w = norm_backward(up, x, w, f.rstd.cpu(), None)
    for (xa, wa), (xb, wb), got, own in (
            ((x + step * d, w), (x - step * d, w), (gh * d.double()).sum(), ((off + U * dh.abs()) * d.abs()).sum()),
            ((x, w + step * dw), (x, w - step * dw), (gw * dw.double()).sum(), (off_w * dw.abs()).sum())):
        (a, na), (b, nb) = loss(xa, wa), loss(xb, wb)
        diff = (a - b) / (2 * step)
        bent = ((loss64(xa, wa) - loss64(xb, wb)) / (2 * step) - got).abs()     # the difference's own error
        assert bent < 1e-3 * (1 + got.abs())
        # three FP32 roundings in every output
        assert (diff - got).abs() <= bent + 3 * U * (na + nb) / (2 * step) + own


def test_stream_and_graph():
    """On a stream of its own, and replayed from a graph with new inputs."""
    dim = 5120
    w = torch.randn(dim, device="cuda")
    x, r, g = (torch.randn((33, dim), device="cuda") for _ in range(3))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        one = mp.rms_norm(x, w, residual=r, quant="int8")
    s.synchronize()
    assert torch.equal(one.out, mp.rms_norm(x, w, residual=r, quant="int8").out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = mp.rms_norm(x, w, residual=r, return_rstd=True)
        gh, gw = mp.rms_norm_backward(g, f.residual, w, f.rstd, grad_residual=g)
    for seed in range(3):
        for t in (x, r, g):
            t.normal_(generator=torch.Generator(device="cuda").manual_seed(seed))
        graph.replay()
        torch.cuda.synchronize()
        e = mp.rms_norm(x, w, residual=r, return_rstd=True)
        eh, ew = mp.rms_norm_backward(g, e.residual, w, e.rstd, grad_residual=g)
        for a, b in ((f.out, e.out), (f.residual, e.residual), (gh, eh), (gw, ew)):
            assert torch.equal(a, b)
    assert math.isfinite(float(gw.sum()))
