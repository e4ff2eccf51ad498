"""A decoder layer's operators in more than one place at a time: on two streams at once, and in
two captured graphs replayed in turns, each with the bits of a call by itself."""
import pytest
import torch

import mixed_precision_dense_tiled_amd as mp

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16


class Work:
    """Inputs of every operator from a seed, and one pass through all of them."""

    def __init__(self, seed, rows, dim):
        g = torch.Generator(device="cuda").manual_seed(seed)
        randn = lambda *s: torch.randn(s, generator=g, device="cuda").to(bf16)
        cut = torch.randint(0, rows + 1, (5,), generator=g, device="cuda").sort().values.to(torch.int32)
        zero, all_ = (torch.tensor([n], dtype=torch.int32, device="cuda") for n in (0, rows))
        self.offsets = torch.cat([zero, cut, all_])
        self.x, self.r, self.g = randn(rows, dim), randn(rows, dim), randn(rows, dim)
        self.w, self.b, self.up = randn(dim), randn(6, dim, 264), randn(rows, 264)
        self.w8 = torch.randint(-127, 128, (6, 264, dim), generator=g, device="cuda").to(torch.int8)
        self.s8 = torch.rand((6, 264), generator=g, device="cuda")
        self.q, self.k, self.v = randn(rows, 4, 64), randn(rows, 2, 64), randn(rows, 2, 64)
        self.freq = torch.rand(32, generator=g, device="cuda")
        pages = -(-rows // 16)
        self.cache = [randn(pages, 16, 2, 64) for _ in range(2)]
        self.where = (torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None], torch.cat([zero, all_]),
                      all_)

    def __call__(self):
        n = mp.rms_norm(self.x, self.w, residual=self.r, return_rstd=True)
        gh, gw = mp.rms_norm_backward(self.g, n.residual, self.w, n.rstd, grad_residual=self.r)
        i8 = mp.rms_norm(self.x, self.w, residual=self.r, quant="int8")
        f8 = mp.rms_norm(self.x, self.w, quant="fp8_blocks")
        q = mp.paged_kv_append_rope(self.q, self.k, self.v, *self.cache, *self.where, self.freq)
        d = mp.gemm_grouped(n.out, self.b, self.offsets, d16=True)
        return [n.out, n.residual, n.rstd, gh, gw, i8.out, i8.scales, f8.out, f8.scales, q, d,
                mp.gemm_grouped(self.up, self.b, self.offsets, trans_b=True),
                mp.gemm_grouped_wgrad(n.out, self.up, self.offsets),
                mp.gemm_grouped_w8a8(i8.out, i8.scales, self.w8, self.s8, self.offsets), *self.cache]


def same(a, b):
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


SIZES = [((300, 1000), (70, 5000)), ((2000, 520), (1, 128)), ((1500, 3000), (900, 9000))]


@pytest.mark.parametrize("one, two", SIZES)
def test_two_streams(one, two):
    works = [Work(1, *one), Work(2, *two)]
    want = [[t.clone() for t in w()] for w in works]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in works]
    for _ in range(3):
        got = [None, None]
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                for _ in range(4):
                    got[i] = works[i]()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            same(a, b)


@pytest.mark.parametrize("one, two", SIZES)
def test_two_graphs(one, two):
    works = [Work(3, *one), Work(4, *two)]
    for w in works:
        w()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for w in works:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(w())
    for seed in range(3):
        for w in works:
            for t in (w.x, w.r, w.g, w.up, w.q, w.k, w.v):
                t.normal_(generator=torch.Generator(device="cuda").manual_seed(seed))
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        held = [[t.clone() for t in o] for o in outs]
        for w, h in zip(works, held):
            same(w(), h)
