"""paged_kv_append_rope at the precision that it states, and E4M3 caches byte for byte."""
import math

import pytest
import torch

import mixed_precision_dense_tiled_amd as mp
from layers_ref import HALF, TINY, U
from serving_ref import Batch
from test_gpu_layers_rope import bits, freqs

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
