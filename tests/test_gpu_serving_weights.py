"""Single tokens: the weights keep 16 bits and more in the second product, whatever
the cache's type.  Values of one size and both signs cancel in the output, so that
a weight's rounding to FP16 (2^-12 of it) would stand out against the output's own."""
import pytest
import torch

import mixed_precision_dense_tiled_amd as mp
from serving_ref import EPS, Batch, close

pytestmark = pytest.mark.gpu
bf16, f16 = torch.bfloat16, torch.float16
U = EPS[torch.float32]


@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("dtype, fp8", [(bf16, False), (f16, False), (bf16, True), (f16, True)])
@pytest.mark.parametrize("longest", [40, 1500], ids=["one_launch", "shared_out"])
def test_weights_are_not_rounded_to_16_bits(gpu_ok, dim, dtype, fp8, longest):
    b = Batch([(1, n) for n in (2, 3, 5, 8, 13, 21, 32, 40, longest)], 8, 2, dim, 16, dtype, fp8, seed=dim + 90)
    g = torch.Generator().manual_seed(7)
    v = b.caches[1]
    v.copy_((torch.randint(0, 2, v.shape, generator=g) * 2 - 1).to(v.dtype))
    b.scales = [b.scales[0], torch.ones(2) if fp8 else None]
    out = mp.paged_attention(**b.gpu(), scale=0.5 * dim ** -0.5)
    o, _, tol, _ = b.attention(scale=0.5 * dim ** -0.5)
    # the definition's bound holds half a step of 16 bits for each weight: |v| = 1, so
    # that much of the whole.  Of it stays what the second part leaves: half a step
    # (BF16, its smallest) of half a step
    ep = EPS[f16] if fp8 else EPS[dtype]
    tol = tol - 1.01 * ep + 1.01 * EPS[bf16] ** 2
    assert (tol > 0).all()
    close(out, o, tol, "out")
