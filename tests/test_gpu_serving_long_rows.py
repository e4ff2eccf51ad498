"""token_logprobs over rows of many chunks in one workgroup (rows enough that none
is cut): ties, masked prefixes, few possible tokens, NaN in early and late
chunks."""
import math

import pytest
import torch

import mixed_precision_dense_tiled_amd as mp
from test_gpu_serving_logprobs import check

pytestmark = pytest.mark.gpu
bf16, f32 = torch.bfloat16, torch.float32
ROWS = 300


def noise(vocab, dtype, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(ROWS, vocab, device="cuda", generator=g) * 2.5).to(dtype)


def check_some(x, t, top, rows):
    """The kernel over all rows, the definition over some of them."""
    r = mp.token_logprobs(x, t, top_k=top)
    check(x[rows], t[rows], top, mp.TokenLogprobs(*(v[rows] for v in r)))
    return r


@pytest.mark.parametrize("dtype, vocab", [(bf16, 65001), (f32, 40003)])
@pytest.mark.parametrize("top", [1, 20, 64])
def test_ties_and_masks(gpu_ok, dtype, vocab, top):
    x = noise(vocab, dtype, 1)
    x[0] = 0.0                                            # all equal
    x[1, :40000] = -math.inf                              # nothing in the first chunks
    x[2] = -math.inf
    x[2, torch.arange(10) * 4000 + 3] = torch.arange(10, device="cuda").to(dtype)     # ten possible tokens
    x[3] = -math.inf                                      # none
    x[4] = (torch.arange(vocab, device="cuda") // 5000).to(dtype)                     # rising steps
    x[5] = -(torch.arange(vocab, device="cuda") // 5000).to(dtype)                    # falling steps
    x[6] = torch.arange(vocab, device="cuda").remainder(3).to(dtype)
    x[7, 30000:] = 9.0                                    # a tie above all that came before
    x[8, :8200] = -math.inf
    x[9, vocab - 1] = 50.0
    x[10] = -math.inf
    x[10, vocab - 1] = 1.0
    x[11, 100:] = -math.inf
    t = torch.arange(ROWS, device="cuda") * 100
    check_some(x, t, top, list(range(13)) + [299])


@pytest.mark.parametrize("dtype, vocab", [(bf16, 65001), (f32, 40003), (f32, 3500), (f32, 3400)])
@pytest.mark.parametrize("top", [1, 20, 64])
@pytest.mark.parametrize("where", [0, 8, 1500, 9000, 33000, -1])
def test_alternatives_of_a_row_with_nan(gpu_ok, dtype, vocab, top, where):
    """NaN results, but the indices keep their order: NaN first (lower index first),
    then the largest."""
    x = noise(vocab, dtype, 2)
    first = vocab - 1 if where < 0 else min(where, vocab - 100)
    for row, n in ((0, 1), (1, 3), (2, 40), (3, 70), (4, 2000)):
        x[row, first:first + n] = math.nan
    x[5, first] = math.inf
    t = torch.arange(ROWS, device="cuda")
    r = check_some(x, t, top, [6, 7, 299])
    for row in range(6):
        for v in (r.logprob, r.lse, r.entropy, r.top_logprobs):
            assert v[row].isnan().all()
        y = x[row].double().cpu()
        order = torch.sort(torch.where(y.isnan(), math.inf, y), descending=True, stable=True).indices[:top]
        if row < 5:
            assert r.top_indices[row].tolist() == order.tolist(), row
        else:
            assert int(r.top_indices[row, 0]) == first and len(set(r.top_indices[row].tolist())) == top
