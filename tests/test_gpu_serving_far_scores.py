"""Scores at the far ends of FP32: the largest one takes all the weight, however low
it lies."""
import pytest
import torch

import mixed_precision_dense_tiled_amd as mp
from serving_ref import EPS, Batch, close

pytestmark = pytest.mark.gpu
bf16, f16 = torch.bfloat16, torch.float16


@pytest.mark.parametrize("dtype, size", [(bf16, 1e3), (bf16, 1e5), (bf16, 1e10), (bf16, 1e16), (bf16, 1e18), (f16, 1e3),
                                         (f16, 3e4)])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("seqs", [[(1, 1), (1, 40), (1, 700)], [(1, 1), (1, 40), (1, 1500)], [(1, 1), (40, 40), (90, 700)]],
                         ids=["one_launch", "shared_out", "chunks"])
def test_the_largest_score_takes_all(gpu_ok, dtype, size, sign, seqs):
    """q is `size` in every place, key j of a sequence sign * size * (1 + (j * 37 % 64) / 64):
    steps of 1 / 64 apart.  (q . k stays below 2^127, FP32's own end.)"""
    b = Batch(seqs, 2, 1, 64, 16, dtype, seed=3)
    size = float(torch.tensor(size, dtype=dtype))
    b.q.fill_(size)
    for s, (_, n) in enumerate(seqs):
        for j in range(n):
            b.caches[0][b.table[s, j // 16].long(), j % 16] = sign * size * (1 + j * 37 % 64 / 64)
    out, lse = mp.paged_attention(**b.gpu(), return_lse=True, scale=0.125)
    # (by the softmax itself: e^(s - lse) of such scores has lost the sum)
    want, z = torch.empty(b.q.shape, dtype=torch.float64), torch.empty(b.q.shape[:2], dtype=torch.float64)
    for s, (nq, n) in enumerate(seqs):
        k, v = b.keys(s, 0, 0), b.keys(s, 0, 1)
        for t in range(nq):
            seen = n - nq + t + 1
            sc = 0.125 * (k[:seen] @ b.q[int(b.cu[s]) + t, 0].double())
            want[int(b.cu[s]) + t], z[int(b.cu[s]) + t] = torch.softmax(sc, 0) @ v[:seen], torch.logsumexp(sc, 0)
    # any error of a score is far below a step between keys, but far above 1: where
    # keys share the largest score their weights are the same all the same
    close(lse, z, 70 * EPS[torch.float32] * z.abs(), "lse")
    p = torch.tensor(2.02 * EPS[dtype])
    close(out, want, p + p * want.abs(), "out")
