"""paged_kv_append_rope on the GPU: turned keys and queries against the rotation in
64 bits, values and everything else in the cache bit for bit."""
import math

import pytest
import torch

import mixed_precision_dense_tiled_amd as mp
from layers_ref import HALF, TINY, U, rope
from serving_ref import Batch

pytestmark = pytest.mark.gpu
bf16, f16 = torch.bfloat16, torch.float16


def positions(b):
    pos = torch.empty(b.tokens, dtype=torch.int64)
    for i, (q, n) in enumerate(b.seqs):
        lo = int(b.cu[i])
        pos[lo:lo + q] = torch.arange(n - q, n)
    return pos


def freqs(pairs, base=10000.0):
    return (base ** (-torch.arange(pairs) / pairs)).float()


def bits(t):
    return t.cpu().view(torch.uint8 if t.element_size() == 1 else torch.int16)


def check(b, k, v, inv_freq, interleaved, gpu, got_q, q=None, pos=None):
    """The cache and q after a call, against the definition."""
    pos = positions(b) if pos is None else pos
    want, off = rope(k, pos, inv_freq, interleaved)
    for name, (new, err), before, after, scale in (("k", (want, off), b.caches[0], gpu[0], b.scales[0]),
                                                   ("v", (v.double(), torch.zeros_like(off)), b.caches[1], gpu[1],
                                                    b.scales[1])):
        after = after.cpu()
        rest = torch.ones(before.shape[:2], dtype=torch.bool)
        for i, (nq, n) in enumerate(b.seqs):
            lo = int(b.cu[i])
            for t in range(nq):
                p = n - nq + t
                if p < 0:
                    continue
                page, slot = int(b.table[i, p // b.page]), p % b.page
                rest[page, slot] = False
                x, e, y = new[lo + t], err[lo + t], after[page, slot].double()
                if scale is not None:
                    s = scale.double()[:, None]
                    x, e = x / s, e / s + 2 * U * (x / s).abs()
                    x = x.clamp(-448, 448)
                    # half a step of E4M3: 2^-4 of a value, 2^-10 among the subnormals
                    assert ((y - x).abs() <= e * (1 + 2 ** -3) + (2.0 ** -4 * x.abs()).clamp_min(2.0 ** -10)).all(), name
                elif name == "v":
                    assert torch.equal(bits(after[page, slot]), bits(v[lo + t]))
                else:
                    assert ((y - x).abs() <= e + HALF[b.dtype] * x.abs() * (1 + 2 ** -6) + TINY[b.dtype]).all()
        assert torch.equal(bits(after[rest]), bits(before[rest])), name
    if q is not None:
        want, off = rope(q, pos, inv_freq, interleaved)
        y = got_q.cpu().double()
        assert ((y - want).abs() <= off + HALF[b.dtype] * want.abs() * (1 + 2 ** -6) + TINY[b.dtype]).all()
        assert torch.equal(bits(got_q[..., 2 * len(inv_freq):].contiguous()),
                           bits(q[..., 2 * len(inv_freq):].contiguous()))


CASES = [
    # seqs, heads, kv_heads, dim, page, pairs, interleaved, dtype, fp8
    ([(1, 1)], 1, 1, 16, 16, 8, False, bf16, False),
    ([(1, 517)], 32, 8, 128, 16, 64, False, bf16, False),
    ([(1, 9), (1, 70), (1, 33)], 4, 2, 64, 32, 32, True, f16, False),
    ([(5, 5), (0, 7), (17, 40), (3, 3)], 8, 8, 80, 16, 40, False, f16, False),
    ([(33, 100)], 7, 1, 128, 7, 16, False, bf16, False),
    ([(33, 100), (8, 8)], 3, 3, 112, 24, 24, True, bf16, False),
    ([(20, 21)], 4, 2, 48, 16, 1, False, f16, False),
    ([(20, 21)], 4, 2, 48, 16, 3, True, bf16, False),
    ([(20, 21)], 4, 2, 48, 16, 11, False, bf16, False),
    ([(40, 90), (1, 5)], 8, 4, 128, 16, 64, False, bf16, True),
    ([(9, 90), (1, 5)], 8, 4, 96, 64, 48, True, f16, True),
    ([(9, 90), (64, 64)], 2, 1, 64, 64, 5, False, f16, True),
    ([(2, 5)] * 70, 2, 2, 32, 16, 16, False, bf16, False),          # more sequences than lanes
]


@pytest.mark.parametrize("seqs, heads, kv_heads, dim, page, pairs, interleaved, dtype, fp8", CASES)
def test_against_the_rotation(seqs, heads, kv_heads, dim, page, pairs, interleaved, dtype, fp8):
    for with_q, heads_first in ((True, False), (False, True)):
        b = Batch(seqs, heads, kv_heads, dim, page, dtype, fp8, seed=dim + pairs, heads_first=heads_first)
        g = torch.Generator().manual_seed(7)
        k, v = (torch.randn((b.tokens, kv_heads, dim), generator=g).to(dtype) for _ in range(2))
        f = freqs(pairs)
        caches = [c.cuda() for c in b.caches]
        if heads_first:
            caches = [c.transpose(1, 2).contiguous().transpose(1, 2) for c in caches]
        scale = [None if s is None else s.cuda() for s in b.scales]
        got = mp.paged_kv_append_rope(b.q.cuda() if with_q else None, k.cuda(), v.cuda(), *caches, b.table.cuda(),
                                      b.cu.cuda(), b.lens.cuda(), f.cuda(), interleaved=interleaved,
                                      k_scale=scale[0], v_scale=scale[1])
        check(b, k, v, f, interleaved, caches, got, b.q if with_q else None)
        if not with_q:
            assert got is None


@pytest.mark.parametrize("interleaved", [False, True])
def test_one_wide_row_in_place(interleaved):
    """q, k and v side by side in a token's row, q turned where it is."""
    b = Batch([(6, 30), (1, 9), (12, 12)], 4, 2, 64, 16, bf16, seed=3)
    g = torch.Generator().manual_seed(8)
    qkv = torch.randn((b.tokens, 8 * 64 + 16), generator=g).to(bf16)
    gpu = qkv.cuda()
    split = lambda t: [t[:, a * 64:c * 64].unflatten(1, (c - a, 64)) for a, c in ((0, 4), (4, 6), (6, 8))]
    q, k, v = split(gpu)
    caches = [c.cuda() for c in b.caches]
    f = freqs(32)
    got = mp.paged_kv_append_rope(q, k, v, *caches, b.table.cuda(), b.cu.cuda(), b.lens.cuda(), f.cuda(),
                                  interleaved=interleaved, out=q)
    cq, ck, cv = split(qkv)
    assert got is q
    check(b, ck, cv, f, interleaved, caches, got, cq)
    assert torch.equal(bits(gpu[:, 256:].contiguous()), bits(qkv[:, 256:].contiguous()))


def test_far_positions():
    """Angles of positions far out (FP32 would lose them whole). The cache is small:
    nearly all of a sequence lies on pages that do not exist."""
    page, width = 1024, 1 << 20
    for p0 in (1 << 17, 1 << 20, (1 << 24) + 5, (1 << 30) - 9):
        lens = torch.tensor([p0 + 8], dtype=torch.int32)
        table = torch.full((1, width), -1, dtype=torch.int32)
        cu = torch.tensor([0, 8], dtype=torch.int32)
        q = torch.randn((8, 2, 64), generator=torch.Generator().manual_seed(p0 % 1000)).to(f16)
        cache = torch.zeros((1, page, 2, 64), dtype=f16, device="cuda")
        f = freqs(32)
        got = mp.paged_kv_append_rope(q.cuda(), q.cuda(), q.cuda(), cache, cache.clone(), table.cuda(), cu.cuda(),
                                      lens.cuda(), f.cuda())
        want, off = rope(q, torch.arange(p0, p0 + 8), f, False)
        err = (got.cpu().double() - want).abs()
        assert (err <= off + HALF[f16] * want.abs() * (1 + 2 ** -6) + TINY[f16]).all()
        assert not cache.any()


def test_tokens_without_a_place():
    """Rows past the last sequence stay; tokens before position 0, on missing pages or
    past the table are turned but not stored."""
    b = Batch([(9, 4), (5, 40)], 2, 1, 32, 16, bf16, seed=4)
    b.table[1, 2] = 77                      # no such page: positions 32 to 39
    tokens = b.tokens + 3
    g = torch.Generator().manual_seed(9)
    q, k, v = (torch.randn((tokens, h, 32), generator=g).to(bf16) for h in (2, 1, 1))
    out = torch.full((tokens, 2, 32), 5.0, dtype=bf16, device="cuda")
    caches = [c.cuda() for c in b.caches]
    f = freqs(16)
    mp.paged_kv_append_rope(q.cuda(), k.cuda(), v.cuda(), *caches, b.table.cuda(), b.cu.cuda(), b.lens.cuda(),
                            f.cuda(), out=out)
    pos = positions(b)
    want, off = rope(q[:b.tokens], pos, f, False)
    assert pos[0] == -5 and (out[b.tokens:] == 5.0).all()
    err = (out[:b.tokens].cpu().double() - want).abs()
    assert (err <= off + HALF[bf16] * want.abs() * (1 + 2 ** -6) + TINY[bf16]).all()
    stored = torch.zeros(b.caches[0].shape[:2], dtype=torch.bool)
    for p in range(4):
        stored[b.table[0, 0].long(), p] = True
    for i in range(2):
        assert torch.equal(bits(caches[i].cpu()[~stored]), bits(b.caches[i][~stored]))
    assert not torch.equal(bits(caches[1].cpu()[stored]), bits(b.caches[1][stored]))


def test_numbers_that_are_none():
    """NaN and infinities stay in their pair; a pair that is not turned (position 0)
    keeps what it can."""
    b = Batch([(2, 2)], 1, 1, 32, 16, f16, seed=5)
    q = torch.randn((2, 1, 32), generator=torch.Generator().manual_seed(1)).to(f16)
    q[1, 0, 3], q[1, 0, 5] = math.nan, math.inf
    caches = [c.cuda() for c in b.caches]
    got = mp.paged_kv_append_rope(q.cuda(), q.cuda(), q.cuda(), *caches, b.table.cuda(), b.cu.cuda(), b.lens.cuda(),
                                  freqs(16).cuda()).cpu()
    assert torch.equal(got[0], q[0])
    bad = torch.zeros(32, dtype=torch.bool)
    bad[[3, 19, 5, 21]] = True
    assert torch.equal(~got[1, 0].isfinite(), bad)


def test_same_as_without_rotation():
    """At frequencies of 0 the keys land as paged_kv_append lands them, in every type."""
    for dtype, fp8 in ((bf16, False), (f16, False), (bf16, True), (f16, True)):
        b = Batch([(33, 90), (1, 7), (20, 20)], 2, 2, 80, 16, dtype, fp8, seed=6)
        g = torch.Generator().manual_seed(10)
        k, v = (torch.randn((b.tokens, 2, 80), generator=g).to(dtype).cuda() for _ in range(2))
        scale = [None if s is None else s.cuda() for s in b.scales]
        one, two = [c.cuda() for c in b.caches], [c.cuda() for c in b.caches]
        where = (b.table.cuda(), b.cu.cuda(), b.lens.cuda())
        mp.paged_kv_append(k, v, *one, *where, k_scale=scale[0], v_scale=scale[1])
        mp.paged_kv_append_rope(None, k, v, *two, *where, torch.zeros(40, device="cuda"), k_scale=scale[0],
                                v_scale=scale[1])
        for x, y in zip(one, two):
            assert torch.equal(bits(x), bits(y))


def test_stream_and_graph():
    b = Batch([(3, 40), (1, 9), (30, 30)], 4, 2, 64, 16, bf16, seed=7)
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn((b.tokens, h, 64), generator=g, device="cuda").to(bf16) for h in (4, 2, 2))
    where = (b.table.cuda(), b.cu.cuda(), b.lens.cuda(), freqs(32).cuda())
    caches = [c.cuda() for c in b.caches]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mp.paged_kv_append_rope(q, k, v, *caches, *where)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = mp.paged_kv_append_rope(q, k, v, *caches, *where)
    for seed in range(3):
        for t in (q, k, v):
            t.normal_(generator=g)
        where[2].copy_(b.lens + seed % 2)       # (one more token at the end of every sequence)
        graph.replay()
        torch.cuda.synchronize()
        other = [c.clone() for c in caches]
        for c in other:
            c.zero_()
        want = mp.paged_kv_append_rope(q, k, v, *other, *where)
        assert torch.equal(got, want)
        for x, y in zip(caches, other):
            used = y.view(torch.int16) != 0
            assert torch.equal(x.view(torch.int16)[used], y.view(torch.int16)[used])
