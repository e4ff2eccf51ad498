"""paged_kv_append_rope at the precision that it states, over more tokens than one to a
workgroup, and E4M3 caches byte for byte."""
import math

import pytest
import torch

import mixed_precision_dense_tiled_amd as mp
from layers_ref import HALF, TINY, U, rope
from serving_ref import Batch
from test_gpu_layers_rope import bits, freqs, positions

pytestmark = pytest.mark.gpu
bf16, f16 = torch.bfloat16, torch.float16


@pytest.mark.parametrize("dtype", [bf16, f16])
@pytest.mark.parametrize("pairs, interleaved", [(8, False), (16, False), (5, False), (12, True), (40, False)])
@pytest.mark.parametrize("scale", [None, 0.75, 2.0 ** -59, 2.0 ** 59])
def test_zeros_keep_their_sign(scale, pairs, interleaved, dtype):
    """Values, and elements of keys that do not turn, land byte for byte as paged_kv_append lands
    them (which divides), -0 among them."""
    fp8 = scale is not None
    b = Batch([(33, 90), (1, 7), (0, 3), (20, 20)], 2, 2, 80, 16, dtype, fp8, seed=6)
    g = torch.Generator().manual_seed(10)
    k, v = (torch.randn((b.tokens, 2, 80), generator=g) for _ in range(2))
    if fp8 and dtype == bf16:
        k, v = k * (100 * scale), v * (100 * scale)
    for t in (k, v):
        t[..., ::3] = -0.0
        t[3], t[4] = -0.0, 0.0
    k, v = k.to(dtype).cuda(), v.to(dtype).cuda()
    scales = [None if not fp8 else torch.full((2,), scale, device="cuda")] * 2
    one, two = [c.cuda() for c in b.caches], [c.cuda() for c in b.caches]
    where = (b.table.cuda(), b.cu.cuda(), b.lens.cuda())
    mp.paged_kv_append(k, v, *one, *where, k_scale=scales[0], v_scale=scales[1])
    mp.paged_kv_append_rope(None, k, v, *two, *where, freqs(pairs).cuda(), interleaved=interleaved,
                            k_scale=scales[0], v_scale=scales[1])
    assert torch.equal(bits(one[1]), bits(two[1]))
    assert torch.equal(bits(one[0][..., 2 * pairs:].contiguous()), bits(two[0][..., 2 * pairs:].contiguous()))
    if fp8:
        assert (one[1].view(torch.uint8) == 0x80).any()


def test_angles_to_half_a_step():
    """Where a token's angle is an odd number of eighths of a turn, a (cos -+ sin) cancels: the
    result of a = b = 1024 shows cos and sin to their last bits.  Each is a value of 64 bits
    rounded once to FP32, off by at most 2^-25 below 1 (and the series' 1e-11); the difference
    of two such numbers is exact, their sum is rounded, and both go once to FP16."""
    m = torch.arange(32)
    f = ((2 * m + 1) * (math.pi / 4)).float()
    q = torch.full((64, 1, 64), 1024.0).to(f16)
    cache = torch.zeros((4, 16, 1, 64), dtype=f16, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    angle = torch.arange(64).double()[:, None] * f.double()
    c, s = torch.cos(angle), torch.sin(angle)
    for near in (False, True):
        got = mp.paged_kv_append_rope(q.cuda(), q.cuda(), q.cuda(), cache, cache.clone(), i32([[0, 1, 2, 3]]),
                                      i32([0, 64]), i32([64]), f.cuda(), interleaved=near).cpu().double()[:, 0]
        first, second = (got[:, 0::2], got[:, 1::2]) if near else (got[:, :32], got[:, 32:])
        for x, want in ((first, 1024 * (c - s)), (second, 1024 * (c + s))):
            bound = 1024 * 2 * (2.0 ** -25 + 1e-11) + (HALF[f16] + U) * want.abs() * (1 + 2.0 ** -10) + TINY[f16]
            assert ((x - want).abs() <= bound).all(), ((x - want).abs() - bound).max()


def ragged(tokens, seqs, seed):
    """[(new, all)] of `seqs` sequences with `tokens` new ones in all, every fifth without any."""
    g = torch.Generator().manual_seed(seed)
    part = torch.rand(seqs, generator=g) + 0.1
    part[::5] = 0
    ends = (part.cumsum(0) / part.sum() * tokens).round().long()
    ends[-1] = tokens
    new = torch.diff(ends, prepend=torch.zeros(1, dtype=torch.long)).tolist()
    past = torch.randint(0, 60, (seqs,), generator=g).tolist()
    return [(q, q + n) for q, n in zip(new, past)]


def check(b, k, v, f, interleaved, caches, q, got):
    """All of a call's outputs against the definition; the rest of the cache as it was."""
    pos = positions(b)
    seq = torch.repeat_interleave(torch.arange(len(b.seqs)), torch.tensor([n for n, _ in b.seqs]))
    page, slot = b.table[seq, pos // b.page].long(), pos % b.page
    turned, off = rope(k[:b.tokens], pos, f, interleaved)
    for i, (new, err) in enumerate(((turned, off), (v[:b.tokens].double(), torch.zeros_like(off)))):
        before, after = b.caches[i], caches[i].cpu()
        y = after[page, slot].double()
        if b.scales[i] is not None:
            s = b.scales[i].double()[:, None]
            x, e = (new / s).clamp(-448, 448), err / s + 2 * U * (new / s).abs()
            # half a step of E4M3: 2^-4 of a value, 2^-10 among the subnormals
            assert ((y - x).abs() <= e * (1 + 2 ** -3) + (2.0 ** -4 * x.abs()).clamp_min(2.0 ** -10)).all()
        else:
            assert ((y - new).abs() <= err + HALF[b.dtype] * new.abs() * (1 + 2 ** -6) + TINY[b.dtype]).all()
        rest = torch.ones(before.shape[:2], dtype=torch.bool)
        rest[page, slot] = False
        assert torch.equal(bits(after[rest]), bits(before[rest]))
    if q is not None:
        want, off = rope(q[:b.tokens], pos, f, interleaved)
        y = got[:b.tokens].cpu()
        assert ((y.double() - want).abs() <= off + HALF[b.dtype] * want.abs() * (1 + 2 ** -6) + TINY[b.dtype]).all()
        still = slice(2 * len(f), None)
        assert torch.equal(bits(y[..., still].contiguous()), bits(q[:b.tokens, :, still].contiguous()))


# Few heads and over 512 (1024, 2048) pairs of tokens: 2, 4 and 8 tokens to a workgroup, and
# token counts that leave a part of the last one.
MANY = [
    # tokens, seqs, heads, kv_heads, dim, page, pairs, interleaved, dtype, fp8
    (1030, 9, 4, 2, 128, 16, 64, False, bf16, False),
    (1031, 90, 4, 2, 64, 16, 32, True, f16, False),         # (more sequences than lanes)
    (1030, 9, 2, 1, 48, 16, 8, False, bf16, True),          # (threads that have no part of a row)
    (2050, 9, 2, 1, 80, 32, 20, True, f16, False),
    (2051, 70, 1, 1, 16, 16, 8, False, bf16, False),
    (2053, 7, 4, 2, 64, 64, 16, False, f16, True),
    (4801, 24, 4, 2, 64, 64, 16, False, bf16, True),
    (4801, 100, 2, 1, 96, 16, 24, True, f16, True),
    (4099, 5, 2, 2, 112, 24, 56, False, f16, False),
    (4100, 200, 4, 1, 128, 16, 40, True, bf16, False),
    (1030, 9, 4, 2, 96, 16, 12, False, f16, False),         # (pairs that fill no piece)
    (2050, 80, 2, 1, 64, 16, 5, False, bf16, True),
]


@pytest.mark.parametrize("tokens, seqs, heads, kv_heads, dim, page, pairs, interleaved, dtype, fp8", MANY)
def test_many_tokens(tokens, seqs, heads, kv_heads, dim, page, pairs, interleaved, dtype, fp8):
    b = Batch(ragged(tokens, seqs, tokens), heads, kv_heads, dim, page, dtype, fp8, seed=dim + pairs)
    g = torch.Generator().manual_seed(7)
    behind = 5          # rows behind the last sequence
    k, v = (torch.randn((tokens + behind, kv_heads, dim), generator=g).to(dtype) for _ in range(2))
    q = torch.cat([b.q, torch.full((behind, heads, dim), 3.0, dtype=dtype)])
    f = freqs(pairs)
    scale = [None if s is None else s.cuda() for s in b.scales]
    where = (b.table.cuda(), b.cu.cuda(), b.lens.cuda(), f.cuda())
    first = None
    for how in ("apart", "in place", "without"):
        caches = [c.cuda() for c in b.caches]
        mine = None if how == "without" else q.cuda()
        out = mine if how == "in place" else None if how == "without" else torch.full_like(q, 9.0).cuda()
        got = mp.paged_kv_append_rope(mine, k.cuda(), v.cuda(), *caches, *where, interleaved=interleaved,
                                      k_scale=scale[0], v_scale=scale[1], out=out)
        check(b, k, v, f, interleaved, caches, None if how == "without" else q, got)
        if how != "without":
            assert (got[tokens:] == (3.0 if how == "in place" else 9.0)).all()
        # the same bits however q is given
        now = [bits(c) for c in caches] + ([] if how == "without" else [bits(got[:tokens])])
        first = now if first is None else first
        assert all(torch.equal(x, y) for x, y in zip(first, now))


@pytest.mark.parametrize("pairs, interleaved", [(16, False), (12, True), (5, False)])
@pytest.mark.parametrize("scale", [2.0 ** -61, 2.0 ** -70, 2.0 ** -100, 2.0 ** 61, 2.0 ** 100, 0.99 * 2.0 ** -60,
                                   1.01 * 2.0 ** 60])
def test_unusual_scales(scale, pairs, interleaved):
    """Cache scales that the codes' quick division does not take, each beside one that it does;
    BF16 rows of their size, some past E4M3's range."""
    b = Batch([(33, 90), (1, 7), (20, 20)], 2, 2, 64, 16, bf16, True, seed=6)
    b.scales = [torch.tensor([scale, 0.75]), torch.tensor([0.75, scale])]
    g = torch.Generator().manual_seed(10)
    k, v = (torch.randn((b.tokens, 2, 64), generator=g) * (200 * s[:, None]) for s in b.scales)
    k, v = k.to(bf16), v.to(bf16)
    f = freqs(pairs)
    caches = [c.cuda() for c in b.caches]
    mp.paged_kv_append_rope(None, k.cuda(), v.cuda(), *caches, b.table.cuda(), b.cu.cuda(), b.lens.cuda(), f.cuda(),
                            interleaved=interleaved, k_scale=b.scales[0].cuda(), v_scale=b.scales[1].cuda())
    check(b, k, v, f, interleaved, caches, None, None)
    plain = [c.cuda() for c in b.caches]
    mp.paged_kv_append(k.cuda(), v.cuda(), *plain, b.table.cuda(), b.cu.cuda(), b.lens.cuda(),
                       k_scale=b.scales[0].cuda(), v_scale=b.scales[1].cuda())
    assert torch.equal(bits(plain[1]), bits(caches[1]))
    assert torch.equal(bits(plain[0][..., 2 * pairs:].contiguous()), bits(caches[0][..., 2 * pairs:].contiguous()))


@pytest.mark.parametrize("seqs", [1, 9, 64, 65, 90])
@pytest.mark.parametrize("tokens", [30, 1030, 4801])
def test_broken_batches(tokens, seqs):
    """Borders and lengths that descend, are negative or leave the batch: tokens land where
    paged_kv_append lands them, whatever the number of tokens to a workgroup."""
    g = torch.Generator().manual_seed(tokens + seqs)
    width, page = 8, 16
    table = torch.randperm(seqs * width, generator=g).to(torch.int32).view(seqs, width)
    cu = torch.randint(-tokens // 4, tokens + tokens // 4, (seqs + 1,), generator=g).to(torch.int32)
    if seqs % 2:
        cu = cu.sort().values
        cu[seqs // 2] = -5
    lens = torch.randint(-20, 2 * width * page, (seqs,), generator=g).to(torch.int32)
    k, v, q = (torch.randn((tokens, h, 32), generator=g).to(bf16).cuda() for h in (1, 1, 2))
    one, two = ([torch.zeros((seqs * width, page, 1, 32), dtype=bf16, device="cuda") for _ in range(2)] for _ in range(2))
    where = (table.cuda(), cu.cuda(), lens.cuda())
    mp.paged_kv_append(k, v, *one, *where)
    out = torch.full_like(q, 9.0)
    mp.paged_kv_append_rope(q, k, v, *two, *where, torch.zeros(16, device="cuda"), out=out)
    for x, y in zip(one, two):
        assert torch.equal(bits(x), bits(y))
    # an angle of 0 leaves a row as it is; a row of no sequence is not written
    same, left = (out == q).flatten(1).all(1), (out == 9.0).flatten(1).all(1)
    assert (same | left).all()
