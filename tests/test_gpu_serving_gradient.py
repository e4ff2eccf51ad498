"""The log probabilities' gradient with factors at the ends of their range."""
import math

import pytest
import torch

import mixed_precision_dense_tiled_amd as mp
from serving_ref import logprobs

pytestmark = pytest.mark.gpu
bf16, f32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [bf16, torch.float16, f32])
@pytest.mark.parametrize("factor", [1e9, 1e20, 1e30])
def test_large_gradients_leave_impossible_tokens_at_zero(gpu_ok, dtype, factor):
    """A gradient of the entropy past 3.4e8 on rows with logits of -inf and of the
    type's lowest value."""
    x = (torch.randn(4, 500, generator=torch.Generator().manual_seed(3)) * 2.5).to(dtype).cuda()
    x[:, 10:200] = -math.inf
    x[1, 200:300] = torch.finfo(dtype).min
    x[2, 1:] = -math.inf
    t = torch.tensor([0, 1, 0, -100], device="cuda")
    r = mp.token_logprobs(x, t)
    ge = torch.tensor([factor, -factor, factor, factor], device="cuda")
    got = mp.token_logprobs_backward(x, t, r.lse, r.entropy, None, ge).cpu().double()
    assert not got.isnan().any()
    assert not got[:, 10:200].any() and not got[1, 200:300].any()
    _, lse, h, _, _ = logprobs(x, t)
    lp = x.double().cpu() - lse[:, None]
    p = lp.exp()
    want = -ge.double().cpu()[:, None] * p * (lp.masked_fill(p == 0, 0.0) + h[:, None])
    if dtype == f32 or dtype == bf16 and factor < 1e30:
        # FP32: exponent, lse and entropy are off by some hundred roundings of values up to 20
        tol = factor * p * 2e-4 + 2.0 ** -8 * want.abs()
        assert ((got - want).abs() <= tol).all()
