"""rms_norm and its gradient where values leave the usual ranges: against the
definition in 64 bits, and codes byte for byte."""
import pytest
import torch

import mixed_precision_dense_tiled_amd as mp
from layers_ref import HALF, TINY, norm_backward, norm_rows, norm_rstd, quantise

pytestmark = pytest.mark.gpu
# a width of every launch, none a whole number of a thread's elements
WIDTHS = [5, 300, 700, 1501, 3001, 5003, 7001, 9001, 20001]


def randn(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def close(got, want, off, dtype):
    err = (got.cpu().double() - want).abs()
    bound = off + HALF[dtype] * want.abs() * (1 + 2.0 ** -7) + TINY[dtype]
    assert (err <= bound).all(), (err - bound).max()


@pytest.mark.parametrize("dim", [4] + WIDTHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size", [1e37, 1e20, 1e-20, 1e-30])
def test_backward_far_sizes(size, dtype, dim):
    """Rows whose squares, and whose rstd's square, leave FP32: the projection on the row stays."""
    rows = 7
    h = (randn((rows, dim), dim) * size).to(dtype)
    if dim == 4:
        h[0] = torch.tensor([3e37, -1e37, 2e37, 0.5e37]).to(dtype) if size == 1e37 else h[0]
    g = randn((rows, dim), dim + 1).to(dtype)
    w = (1 + 0.3 * randn(dim, dim + 2)).to(dtype)
    rstd = norm_rstd(h, 0.0)
    gh, gw = mp.rms_norm_backward(g.cuda(), h.cuda(), w.cuda(), rstd.cuda())
    dh, off, dw, off_w = norm_backward(g, h, w, rstd, None)
    close(gh, dh, off, dtype)
    assert ((gw.cpu().double() - dw).abs() <= off_w).all()


@pytest.mark.parametrize("dim", WIDTHS)
@pytest.mark.parametrize("size", [1e4, 1e-3, 1e-6])
def test_backward_far_sizes_of_fp16(size, dim):
    """FP16's largest values and its subnormals."""
    h = (randn((7, dim), dim) * size).to(torch.float16)
    g = (randn((7, dim), dim + 1) * min(1.0, 100 * size)).to(torch.float16)
    w = (1 + 0.3 * randn(dim, dim + 2)).to(torch.float16)
    rstd = norm_rstd(h, 0.0)
    gh, gw = mp.rms_norm_backward(g.cuda(), h.cuda(), w.cuda(), rstd.cuda())
    dh, off, dw, off_w = norm_backward(g, h, w, rstd, None)
    close(gh, dh, off, torch.float16)
    assert ((gw.cpu().double() - dw).abs() <= off_w).all()


@pytest.mark.parametrize("dim", [5, 700, 3001, 20001])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_backward_of_zeros(dtype, dim):
    """A row of zeros under an eps whose rstd's square leaves FP32: rstd * grad * weight."""
    g, w = randn((3, dim), dim).to(dtype), (1 + 0.3 * randn(dim, dim + 1)).to(dtype)
    h = torch.zeros((3, dim), dtype=dtype)
    rstd = norm_rstd(h, 1e-45)
    assert float(rstd[0]) > 2.0 ** 70
    gh, gw = mp.rms_norm_backward(g.cuda(), h.cuda(), w.cuda(), rstd.cuda())
    assert torch.equal(gh.cpu(), (rstd[:, None] * (g.float() * w.float())).to(dtype))
    assert not gw.any()


def same_numbers(a, b):
    assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(-1), b.nan_to_num(-1)), (a, b)


@pytest.mark.parametrize("quant", ["int8", "fp8_rows", "fp8_blocks"])
@pytest.mark.parametrize("dim", [1, 9, 100, 128, 130] + WIDTHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rstd_of_infinity(dtype, dim, quant):
    """Rows of FP32's subnormals without an eps: every y is infinite, or NaN from a 0; scales are
    one or the other, and the values that the codes stand for are NaN."""
    x = torch.full((3, dim), 2.0 ** -133).to(dtype)
    x[1] = -x[1]
    x[2, dim // 2] = 0
    w = torch.ones(dim, dtype=dtype)
    got = mp.rms_norm(x.cuda(), w.cuda(), eps=0.0, quant=quant)
    values, scales = quantise(norm_rows(x, w, 0.0), quant)
    assert scales[:2].isinf().all() and scales[2].isnan().any()
    mine = got.scales.cpu()
    assert not mine.isfinite().any() and mine[scales.isnan()].isnan().all()
    out = got.out.cpu() if quant == "int8" else got.out.cpu().view(torch.float8_e4m3fn)
    same_numbers(out.float(), values)
    block = 128 if quant == "fp8_blocks" else dim
    each = mine.view(3, -1).repeat_interleave(block, 1)[:, :dim]
    assert (out.float() * each).isnan().all()


@pytest.mark.parametrize("quant", ["fp8_rows", "fp8_blocks"])
@pytest.mark.parametrize("dim", [128] + WIDTHS)
def test_minus_zero(quant, dim):
    """E4M3 codes keep the sign of a 0, as the division by the scale does: of -0 in x, of a
    negative x under a weight of 0, in rows of zeros, and of what is rounded to 0."""
    x = randn((4, dim), dim)
    x[:, ::3] = -0.0
    x[1] = -0.0
    x[2, 1::3] *= 1e-6
    w = 1 + 0.3 * randn(dim, dim + 1)
    w[2::5] = 0
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        h, v = x.to(dtype), w.to(dtype)
        got = mp.rms_norm(h.cuda(), v.cuda(), quant=quant)
        values, _ = quantise(norm_rows(h, v, 1e-6), quant)
        want = values.to(torch.float8_e4m3fn).view(torch.uint8)
        assert (want == 0x80).any() and torch.equal(got.out.cpu(), want)


def test_backward_of_more_rows_than_a_norm_takes():
    """The workgroups of the gradient walk rows, of any number."""
    rows, dim = (1 << 22) + 3, 8
    h, g = (randn((rows, dim), i).to(torch.bfloat16) for i in (1, 2))
    w = 1 + 0.3 * randn(dim, 3)
    rstd = norm_rstd(h, 1e-6)
    gh, gw = mp.rms_norm_backward(g.cuda(), h.cuda(), w.cuda(), rstd.cuda())
    dh, off, dw, off_w = norm_backward(g, h, w, rstd, None)
    close(gh, dh, off, torch.bfloat16)
    assert ((gw.cpu().double() - dw).abs() <= off_w).all()


@pytest.mark.parametrize("quant", [None, "int8", "fp8_rows", "fp8_blocks"])
@pytest.mark.parametrize("dim", [128] + WIDTHS + [16384, 32768])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_weights_of_fp32(dtype, dim, quant):
    """16-bit rows under FP32 weights that 16 bits do not hold, few rows and more than CUs."""
    w = 1 + 0.3 * randn(dim, dim + 1)
    for rows in (3, 300) if dim <= 8192 else (3,):
        x, r = randn((rows, dim), dim).to(dtype), randn((rows, dim), dim + 2).to(dtype)
        h = (x.float() + r.float()).to(dtype)
        got = mp.rms_norm(x.cuda(), w.cuda(), residual=r.cuda(), quant=quant)
        y = norm_rows(h, w, 1e-6)
        if quant is None:
            assert torch.equal(got.out.cpu(), y.to(dtype))
            continue
        values, scales = quantise(y, quant)
        codes = got.out.cpu() if quant == "int8" else got.out.cpu().view(torch.float8_e4m3fn)
        assert torch.equal(got.scales.cpu(), scales) and torch.equal(codes.float(), values)


@pytest.mark.parametrize("quant", [None, "int8", "fp8_blocks"])
@pytest.mark.parametrize("dim", [128] + WIDTHS + [16384, 32768])
def test_in_place_at_every_width(dim, quant):
    """x and the residual replaced by what comes of them, where a row is a wave's and where many
    waves share it; and a gradient in place of its gradients."""
    dtype = torch.bfloat16
    w = (1 + 0.3 * randn(dim, dim + 1)).to(dtype)
    for rows in (3, 300) if dim <= 8192 else (3,):
        xc, rc, gc = (randn((rows, dim), dim + i).to(dtype) for i in (2, 3, 4))
        want = mp.rms_norm(xc.cuda(), w.cuda(), residual=rc.cuda(), quant=quant, return_rstd=True)
        for first in ("x", "residual"):
            x, r = xc.cuda(), rc.cuda()
            h, out = (x, r) if first == "x" else (r, x)
            got = mp.rms_norm(x, w.cuda(), residual=r, quant=quant, residual_out=h, out=out if quant is None else None)
            assert torch.equal(h, want.residual) and torch.equal(got.out, want.out)
            if quant is not None:
                assert torch.equal(got.scales, want.scales)
        if quant is None:
            gh, gw = mp.rms_norm_backward(gc.cuda(), want.residual, w.cuda(), want.rstd, grad_residual=rc.cuda())
            for where in ("grad", "grad_residual"):
                g, r = gc.cuda(), rc.cuda()
                a, b = mp.rms_norm_backward(g, want.residual, w.cuda(), want.rstd, grad_residual=r,
                                            out=g if where == "grad" else r)
                assert torch.equal(a, gh) and torch.equal(b, gw)


@pytest.mark.parametrize("rows, dim", [(1, 700), (3, 5003), (127, 64), (500, 513), (2500, 1000), (20000, 209), (1000, 3001),
                                       (900, 5120), (3001, 1501), (1200, 7001), (1100, 9001), (700, 20001)])
def test_weights_gradient_by_its_sums(rows, dim):
    """The weight's gradient within the roundings of the additions that it takes: a workgroup's (up
    to 1024 columns a wave's) rows one after the other, four waves' sums where they share a
    workgroup, then the workgroups' in 64 lines and a tree of 6; and of the product (h * rstd) * grad,
    whose last rounding is the addition's."""
    h, g = (randn((rows, dim), dim + i).to(torch.float16) for i in (0, 1))
    w = torch.ones(dim, dtype=torch.float16)
    rstd = norm_rstd(h, 1e-6)
    _, gw = mp.rms_norm_backward(g.cuda(), h.cuda(), w.cuda(), rstd.cuda())
    size = mp.layers._lib().rms_norm_backward_workspace(rows, dim)
    groups, waves = max(size // (4 * dim), 1), 4 if dim <= 1024 else 1
    deep = -(-rows // (groups * waves)) + waves - 1 + (-(-groups // 64) + 6 if groups > 1 else 0)
    each = g.double() * h.double() * rstd.double()[:, None]
    bound = 2.0 ** -24 * (deep + 2) * each.abs().sum(0) * (1 + 1e-4)
    assert ((gw.cpu().double() - each.sum(0)).abs() <= bound).all(), (gw.cpu().double() - each.sum(0)).abs().max()


@pytest.mark.parametrize("quant", [None, "int8", "fp8_blocks"])
def test_more_rows_than_a_launch(quant):
    """In place and apart; each row as by itself."""
    most, dim = 4194303, 8
    rows = most + 5
    x, r = (randn((rows, dim), i).to(torch.bfloat16).cuda() for i in (1, 2))
    w = (1 + 0.3 * randn(dim, 3)).to(torch.bfloat16).cuda()
    parts = [mp.rms_norm(x[a:b], w, residual=r[a:b], quant=quant, return_rstd=True) for a, b in ((0, most), (most, rows))]
    want = [None if a is None else torch.cat([a, b]) for a, b in zip(*parts)]
    for place in (False, True):
        got = mp.rms_norm(x, w, residual=r, quant=quant, return_rstd=True, residual_out=r if place else None,
                          out=x if place and quant is None else None)
        for a, b in zip(got, want):
            assert a is b is None or torch.equal(a, b)


def test_overlaps_across_launches():
    """An output that lies on rows of another launch's is refused as one on its own is."""
    most, dim = 4194303, 8
    buf = torch.zeros((2 * most + 10, dim), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(dim, dtype=torch.bfloat16, device="cuda")
    x, far = buf[:most + 5], buf[most:2 * most + 5]
    with pytest.raises(ValueError, match="overlaps"):
        mp.rms_norm(x, w, out=far)
    with pytest.raises(ValueError, match="overlaps"):
        mp.rms_norm(x, w, residual=torch.zeros_like(x), residual_out=far)
    with pytest.raises(mp.MpdtError):       # (the same buffer, both written)
        mp.rms_norm(x, w, residual=torch.zeros_like(x), residual_out=x, out=x)
