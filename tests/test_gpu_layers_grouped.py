"""Products grouped by expert on the GPU: bit for bit with whole numbers, within the
roundings of FP32 sums otherwise, over ragged, empty and broken groups."""
import pytest
import torch

import mixed_precision_dense_tiled_amd as mp
from layers_ref import HALF, TINY, U, groups_of

pytestmark = pytest.mark.gpu
bf16, f16, f32 = torch.bfloat16, torch.float16, torch.float32
GUARD = 7.0


def offs(sizes, first=0):
    out = [first]
    for s in sizes:
        out.append(out[-1] + s)
    return out


def mats(shape, dtype, seed, whole, pad=0, shift=0):
    """(GPU view, CPU copy) of [.., rows, cols] inside a buffer of NaN (rows pad apart)."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(-3, 4, shape, generator=g).float() if whole else torch.randn(shape, generator=g)
    wide = (*shape[:-1], shape[-1] + pad)
    n = 1
    for s in wide:
        n *= s
    fill = float("nan") if dtype.is_floating_point else 99
    buf = torch.full((n + shift + 16,), fill, dtype=dtype)
    view = buf[shift:shift + n].view(wide)[..., :shape[-1]]
    view.copy_(x.to(dtype))
    return buf.cuda()[shift:shift + n].view(wide)[..., :shape[-1]], view.clone()


def close(got, want, mass, dtype, k):
    """Sums of k products of `mass` in all, FP32 in any order, rounded once."""
    got = got.cpu().double()
    bound = (k + 1) * U * mass + HALF[dtype] * want.abs() * (1 + 2 ** -6) + TINY[dtype]
    assert ((got - want).abs() <= bound).all(), ((got - want).abs() - bound).max()


SIZES = [
    # rows of the groups, K, N
    ([1], 1, 1),
    ([1, 1, 1], 8, 8),
    ([3, 0, 5], 7, 9),
    ([0, 0, 64, 1], 31, 33),
    ([65, 63], 32, 64),
    ([127, 0, 128, 129], 33, 127),
    ([16] * 9, 64, 128),
    ([200, 1, 55], 100, 129),
    ([256], 128, 256),
    ([257, 255, 0], 136, 264),
    ([300, 30, 3], 192, 520),
    ([1] * 70, 40, 48),                 # more groups than lanes
    ([700, 0, 1301], 136, 200),         # few tiles of D, long sums
    ([5, 0, 70] * 24, 131, 263),        # many tiles of D that end inside
    ([0] * 65 + [5] + [0] * 80 + [600], 72, 260),
    ([513, 511], 520, 257),
    ([40, 260], 1000, 1000),
    ([700], 2056, 300),
    ([300, 0, 200], 1003, 611),         # rows that end inside a vector, along and across the sum
    ([130, 70], 77, 301),
    ([260, 1], 33, 259),
    ([129, 255, 64], 47, 1025),
    ([700, 0, 900, 513, 129, 65, 1, 800], 200, 1032),
    ([700, 0, 900, 513, 129, 65, 1, 800], 1003, 1501),
    ([2000, 2200], 33, 1025),
    ([1500, 1600, 90, 64], 72, 1288),
    ([4000, 17, 250], 520, 2056),
    ([70000], 16, 264),                 # more whole tiles than two rounds of the card
    ([300, 20000, 90, 40000, 5, 70, 8000], 24, 300),
    ([257, 0, 100] * 40, 8, 16),        # whole and part tiles past the 64th group
    # the same with sums that are not short
    ([700, 0, 900, 513, 129, 65, 1, 800], 1100, 1032),
    ([700, 0, 900, 513, 129, 65, 1, 800], 2061, 1501),
    ([4000, 17, 250], 2056, 2056),
    ([70000], 1064, 264),
    ([300, 20000, 90, 40000, 5, 70, 8000], 1048, 300),
    ([257, 0, 100] * 40, 2064, 528),
    ([9000, 300, 9, 8000], 1064, 4104),     # four rounds of the card
]


@pytest.mark.parametrize("dtype", [bf16, f16])
@pytest.mark.parametrize("trans_b", [False, True])
@pytest.mark.parametrize("sizes, K, N", SIZES)
def test_product(sizes, K, N, trans_b, dtype):
    o = offs(sizes)
    rows, e = o[-1], len(sizes)
    off = torch.tensor(o, dtype=torch.int32, device="cuda")
    for whole, d16, pad, shift in ((True, False, 0, 0), (False, True, 0, 0), (True, True, 8, 0), (False, False, 3, 1)):
        a, ac = mats((rows, K), dtype, 1, whole, pad, shift)
        b, bc = mats((e, N, K) if trans_b else (e, K, N), dtype, 2, whole, pad, shift)
        got = mp.gemm_grouped(a, b, off, trans_b=trans_b, d16=d16)
        kind = dtype if d16 else f32
        assert got.dtype == kind and got.shape == (rows, N)
        for i, (lo, hi) in enumerate(groups_of(o, rows)):
            x, w = ac[lo:hi].double(), bc[i].double()
            w = w.T if trans_b else w
            if whole:
                assert torch.equal(got[lo:hi].cpu(), (x @ w).float().to(kind)), i
            else:
                close(got[lo:hi], x @ w, x.abs() @ w.abs(), kind, K)


@pytest.mark.parametrize("dtype", [bf16, f16])
@pytest.mark.parametrize("sizes, K, N", SIZES)
def test_weights_gradient(sizes, K, N, dtype):
    o = offs(sizes)
    rows, e = o[-1], len(sizes)
    off = torch.tensor(o, dtype=torch.int32, device="cuda")
    for whole, d16, pad, shift in ((True, False, 0, 0), (False, True, 0, 0), (True, True, 8, 0), (False, False, 3, 1)):
        a, ac = mats((rows, K), dtype, 1, whole, pad, shift)
        g, gc = mats((rows, N), dtype, 2, whole, pad, shift)
        kind = dtype if d16 else f32
        out, _ = mats((e, K, N), kind, 3, False, pad, shift)
        got = mp.gemm_grouped_wgrad(a, g, off, out=out if pad else None, d16=d16)
        assert got.dtype == kind and got.shape == (e, K, N)
        for i, (lo, hi) in enumerate(groups_of(o, rows)):
            x, y = ac[lo:hi].double(), gc[lo:hi].double()
            want = x.T @ y
            if whole:
                assert torch.equal(got[i].cpu(), want.float().to(kind)), i
            else:
                close(got[i], want, x.abs().T @ y.abs(), kind, hi - lo)
            if lo == hi:
                assert not got[i].any()


@pytest.mark.parametrize("sizes, K, N", SIZES)
def test_w8a8(sizes, K, N):
    """Bit for bit, and gemm_w8a8's own bits for each group."""
    o = offs(sizes)
    rows, e = o[-1], len(sizes)
    off = torch.tensor(o, dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(4)
    sx = 0.01 + torch.rand(rows, generator=g)
    sw = 0.01 + torch.rand((e, N), generator=g)
    bias = torch.randn((e, N), generator=g)
    for pad, shift, with_bias in ((0, 0, False), (16, 0, True), (3, 1, True)):
        x, xc = mats((rows, K), torch.int8, 1, True, pad, shift)
        w, wc = mats((e, N, K), torch.int8, 2, True, pad, shift)
        big = torch.randint(-128, 128, (rows, K), generator=g).to(torch.int8)
        x.copy_(big)
        got = mp.gemm_grouped_w8a8(x, sx.cuda(), w, sw.cuda(), off, bias=bias.cuda() if with_bias else None)
        for i, (lo, hi) in enumerate(groups_of(o, rows)):
            z = (big[lo:hi].long() @ wc[i].long().T).float()
            y = (z * sx[lo:hi, None]) * sw[i]
            y = y + bias[i] if with_bias else y
            assert torch.equal(got[lo:hi].cpu(), y.to(bf16)), i
            if hi > lo:
                one = mp.gemm_w8a8(x[lo:hi], sx[lo:hi].cuda(), w[i], sw[i].cuda(),
                                   bias=bias[i].cuda() if with_bias else None)
                assert torch.equal(one, got[lo:hi])


@pytest.mark.parametrize("o, rows", [
    ([5, 9, 9, 30], 40),                # rows before the first and past the last group
    ([0, 20, 10, 35], 40),              # descending: groups never share a row
    ([-7, 12, 90, 95], 40),             # outside the rows
    ([50, 60, 70, 80], 40),             # nothing at all
    ([2 ** 31 - 1, -2 ** 31, 5, 40], 40),
    ([0, 0, 0, 0], 40),
])
def test_broken_offsets(o, rows):
    off = torch.tensor(o, dtype=torch.int32, device="cuda")
    K, N = 72, 136
    a, ac = mats((rows, K), f16, 1, True)
    b, bc = mats((3, K, N), f16, 2, True)
    x8, w8 = a.to(torch.int8), b.mT.contiguous().to(torch.int8)
    ones = torch.ones(rows, device="cuda")
    out = torch.full((rows + 2, N), GUARD, device="cuda")
    y8 = torch.full((rows, N), GUARD, dtype=bf16, device="cuda")
    mp.gemm_grouped(a, b, off, out=out[1:-1])
    mp.gemm_grouped_w8a8(x8, ones, w8, torch.ones((3, N), device="cuda"), off, out=y8)
    grad = mp.gemm_grouped_wgrad(a, a[:, :64].contiguous(), off)
    want = torch.full((rows, N), GUARD)
    for i, (lo, hi) in enumerate(groups_of(o, rows)):
        want[lo:hi] = ac[lo:hi].float() @ bc[i].float()
        assert torch.equal(grad[i].cpu(), ac[lo:hi].float().T @ ac[lo:hi, :64].float())
    assert torch.equal(out[1:-1].cpu(), want) and (out[0] == GUARD).all() and (out[-1] == GUARD).all()
    assert torch.equal(y8.cpu(), want.to(bf16))


def test_strided_outputs_and_guards():
    """Rows of D inside a wider buffer: nothing beside them is written."""
    o = offs([70, 0, 59])
    off = torch.tensor(o, dtype=torch.int32, device="cuda")
    for dtype, N, lo in ((bf16, 130, 3), (bf16, 128, 8), (f16, 257, 1)):
        a, ac = mats((o[-1], 96), dtype, 1, True)
        b, bc = mats((3, 96, N), dtype, 2, True)
        want = torch.cat([ac[x:y].float() @ bc[i].float() for i, (x, y) in enumerate(groups_of(o, o[-1]))])
        for kind in (dtype, f32):
            big = torch.full((o[-1] + 4, N + 24), GUARD, dtype=kind, device="cuda")
            mp.gemm_grouped(a, b, off, out=big[2:-2, lo:lo + N])
            assert torch.equal(big[2:-2, lo:lo + N].cpu(), want.to(kind))
            big[2:-2, lo:lo + N] = GUARD
            assert (big == GUARD).all()


def test_empty_axes():
    off = torch.tensor([0, 3, 5], dtype=torch.int32, device="cuda")
    z = lambda *s, dtype=bf16: torch.zeros(s, dtype=dtype, device="cuda")
    d = mp.gemm_grouped(z(5, 0), z(2, 0, 6), off)
    assert d.shape == (5, 6) and not d.any()
    assert mp.gemm_grouped(z(5, 4), z(2, 4, 0), off).shape == (5, 0)
    assert mp.gemm_grouped(z(0, 4), z(2, 4, 6), off).shape == (0, 6)
    assert mp.gemm_grouped(z(5, 4), z(0, 4, 6), off[:1]).shape == (5, 6)
    g = mp.gemm_grouped_wgrad(z(0, 4), z(0, 6), off)
    assert g.shape == (2, 4, 6) and not g.any()
    assert mp.gemm_grouped_wgrad(z(5, 0), z(5, 6), off).shape == (2, 0, 6)
    y = mp.gemm_grouped_w8a8(z(5, 0, dtype=torch.int8), torch.ones(5, device="cuda"), z(2, 6, 0, dtype=torch.int8),
                             torch.ones((2, 6), device="cuda"), off, bias=torch.ones((2, 6), device="cuda"))
    assert (y == 1).all()


def test_numbers_that_are_none_stay_in_their_rows():
    """NaN and infinities in one group's rows or matrix reach nobody else."""
    o = offs([30, 41, 5])
    off = torch.tensor(o, dtype=torch.int32, device="cuda")
    a, ac = mats((o[-1], 100), bf16, 1, True)
    b, bc = mats((3, 100, 72), bf16, 2, True)
    clean = mp.gemm_grouped(a, b, off)
    grad = mp.gemm_grouped_wgrad(a, clean.to(bf16), off)
    a[40, 99] = float("nan")
    b[2, 0, 0] = float("inf")
    got = mp.gemm_grouped(a, b, off)
    assert got[40].isnan().all()
    rest = torch.ones(o[-1], dtype=torch.bool)
    rest[40] = False
    rest[71:] = False
    assert torch.equal(got[rest.cuda()], clean[rest.cuda()]) and torch.equal(got[71:, 1:], clean[71:, 1:])
    again = mp.gemm_grouped_wgrad(a, clean.to(bf16), off)
    assert torch.equal(again[0], grad[0]) and torch.equal(again[2], grad[2])
    assert again[1][99].isnan().all() and torch.equal(again[1][:99], grad[1][:99])


@pytest.mark.parametrize("sizes, K, N", [([300, 513, 7], 264, 520), ([40, 0, 90] * 30, 131, 263),
                                         ([600, 41, 700], 72, 100)])
def test_numbers_that_are_none_beside_tiles(sizes, K, N):
    """A group of nothing but NaN, and NaN behind the last group, next to groups that
    tiles of every size take."""
    o = offs(sizes)
    rows = o[-1] + 100
    off = torch.tensor(o, dtype=torch.int32, device="cuda")
    bad = 1 if sizes[1] else 2
    for dtype in (bf16, f16):
        a, ac = mats((rows, K), dtype, 1, True)
        g, gc = mats((rows, N), dtype, 2, True)
        b, bc = mats((len(sizes), K, N), dtype, 3, True)
        for t in (a, g):
            t[o[bad]:o[bad + 1]] = float("nan")
            t[o[-1]:] = float("nan")
        b[bad] = float("inf")
        d, dt = mp.gemm_grouped(a, b, off), mp.gemm_grouped(g, b, off, trans_b=True)
        dw = mp.gemm_grouped_wgrad(a, g, off)
        for i, (lo, hi) in enumerate(groups_of(o, rows)):
            if i == bad:
                assert d[lo:hi].isnan().all() and dt[lo:hi].isnan().all() and dw[i].isnan().all()
                continue
            assert torch.equal(d[lo:hi].cpu(), ac[lo:hi].float() @ bc[i].float())
            assert torch.equal(dt[lo:hi].cpu(), gc[lo:hi].float() @ bc[i].float().T)
            assert torch.equal(dw[i].cpu(), ac[lo:hi].float().T @ gc[lo:hi].float())


def test_rows_past_4_gib():
    """Rows of one group more than 2^32 bytes apart."""
    o = [0, 1, 1400, 1500]
    off = torch.tensor(o, dtype=torch.int32, device="cuda")
    wide = torch.zeros((1500, 1 << 21), dtype=bf16, device="cuda")     # 4 MiB a row
    a, g = wide[:, 8:80], wide[:, 1 << 20:(1 << 20) + 136]
    x, y = mats((1500, 72), bf16, 1, True)[1], mats((1500, 136), bf16, 2, True)[1]
    a.copy_(x)
    g.copy_(y)
    b, bc = mats((3, 72, 136), bf16, 3, True)
    got, back = mp.gemm_grouped(a, b, off), mp.gemm_grouped(g, b, off, trans_b=True)
    grad = mp.gemm_grouped_wgrad(a, g, off)
    for i, (lo, hi) in enumerate(zip(o, o[1:])):
        assert torch.equal(got[lo:hi].cpu(), x[lo:hi].float() @ bc[i].float())
        assert torch.equal(back[lo:hi].cpu(), y[lo:hi].float() @ bc[i].float().T)
        assert torch.equal(grad[i].cpu(), x[lo:hi].float().T @ y[lo:hi].float())


def test_matrices_past_4_gib():
    """Groups whose matrices lie more than 2^32 bytes apart."""
    K, N, e = 1024, 4096, 600
    b = torch.zeros((e, K, N), dtype=bf16, device="cuda")
    for i in (0, 511, 599):
        b[i].normal_(generator=torch.Generator(device="cuda").manual_seed(i))
    sizes = [0] * e
    for i in (0, 511, 599):
        sizes[i] = 5
    off = torch.tensor(offs(sizes), dtype=torch.int32, device="cuda")
    a, ac = mats((15, K), bf16, 1, False)
    got = mp.gemm_grouped(a, b, off)
    for j, i in enumerate((0, 511, 599)):
        x, w = ac[5 * j:5 * j + 5].double(), b[i].cpu().double()
        close(got[5 * j:5 * j + 5], x @ w, x.abs() @ w.abs(), f32, K)


def test_rows_far_apart():
    """Leading dimensions past what the direct loads' offsets hold."""
    off = torch.tensor([0, 4, 9], dtype=torch.int32, device="cuda")
    wide = torch.zeros((9, 1 << 23), dtype=bf16, device="cuda")     # 16 MiB a row
    a, g = wide[:, 8:80], wide[:, 1 << 20:(1 << 20) + 136]
    x, y = mats((9, 72), bf16, 1, True)[1], mats((9, 136), bf16, 2, True)[1]
    a.copy_(x)
    g.copy_(y)
    b, bc = mats((2, 72, 136), bf16, 3, True)
    got, grad = mp.gemm_grouped(a, b, off), mp.gemm_grouped_wgrad(a, g, off)
    for i, (lo, hi) in enumerate(((0, 4), (4, 9))):
        assert torch.equal(got[lo:hi].cpu(), x[lo:hi].float() @ bc[i].float())
        assert torch.equal(grad[i].cpu(), x[lo:hi].float().T @ y[lo:hi].float())


def test_one_matrix_for_all_groups():
    """A stride of 0 between groups."""
    off = torch.tensor([0, 100, 100, 190], dtype=torch.int32, device="cuda")
    a, ac = mats((190, 128), f16, 1, True)
    b, bc = mats((1, 128, 264), f16, 2, True)
    assert torch.equal(mp.gemm_grouped(a, b.expand(3, -1, -1), off).cpu(), ac.float() @ bc[0].float())


def test_gradients_against_differences():
    """Both gradients along a direction, from the forward product (linear in each side,
    so a difference of whole steps is exact but for roundings)."""
    o = offs([37, 0, 64, 12])
    rows, K, N = o[-1], 96, 80
    off = torch.tensor(o, dtype=torch.int32, device="cuda")
    for trans_b in (False, True):
        a, ac = mats((rows, K), f16, 1, True)
        b, bc = mats((4, N, K) if trans_b else (4, K, N), f16, 2, True)
        up, upc = mats((rows, N), f16, 3, True)
        da, _ = mats((rows, K), f16, 4, True)
        db, _ = mats(tuple(b.shape), f16, 5, True)
        loss = lambda x, w: (mp.gemm_grouped(x, w, off, trans_b=trans_b).double() * up.double()).sum()
        ga = mp.gemm_grouped(up, b, off, trans_b=not trans_b)
        gb = mp.gemm_grouped_wgrad(up, a, off) if trans_b else mp.gemm_grouped_wgrad(a, up, off)
        # (whole numbers: everything is exact)
        assert loss(a + da, b) - loss(a - da, b) == 2 * (ga.double() * da.double()).sum()
        assert loss(a, b + db) - loss(a, b - db) == 2 * (gb.double() * db.double()).sum()


def test_stream_and_graph():
    o = torch.tensor(offs([100, 0, 28, 300]), dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    a = torch.randn((428, 256), generator=g, device="cuda").to(bf16)
    b = torch.randn((4, 256, 512), generator=g, device="cuda").to(bf16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mp.gemm_grouped(a, b, o)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d = mp.gemm_grouped(a, b, o, d16=True)
        da = mp.gemm_grouped(d, b, o, trans_b=True, d16=True)
        db = mp.gemm_grouped_wgrad(a, d, o)
    for sizes in ([100, 0, 28, 300], [0, 428, 0, 0], [1, 2, 400, 25]):
        o.copy_(torch.tensor(offs(sizes), dtype=torch.int32))
        a.normal_(generator=g)
        graph.replay()
        torch.cuda.synchronize()
        e = mp.gemm_grouped(a, b, o, d16=True)
        assert torch.equal(d, e) and torch.equal(da, mp.gemm_grouped(e, b, o, trans_b=True, d16=True))
        assert torch.equal(db, mp.gemm_grouped_wgrad(a, e, o))
