"""Rows whose dim is below the kernels' own widths (64, 96, 128): what fills them up
does not take part."""
import pytest
import torch

import mixed_precision_dense_tiled_amd as mp
from serving_ref import Batch, close

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16


@pytest.mark.parametrize("dim", [16, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("page", [16, 24])
@pytest.mark.parametrize("seqs", [[(1, 100), (1, 40)], [(1, 1500), (1, 40)], [(70, 400), (1, 40)]],
                         ids=["one_launch", "shared_out", "chunks"])
def test_a_key_at_minus_infinity_has_no_weight(gpu_ok, dim, page, seqs):
    """q . k = -inf takes a key out, whatever the row is padded to."""
    b = Batch(seqs, 4, 2, dim, page, bf16, seed=dim)
    b.q[..., 0] = b.q[..., 0].abs() + 0.5
    out_of = {0: [0, 5, 17, 60], 1: [3]}
    for s, keys in out_of.items():
        for j in keys:
            b.caches[0][b.table[s, j // page].long(), j % page, :, 0] = float("-inf")

    def hidden(s):
        m = torch.zeros(b.seqs[s][1], dtype=torch.bool)
        m[out_of[s]] = True
        return m

    got = mp.paged_attention(**b.gpu(), return_lse=True)
    out, lse, tol, tol_lse = b.attention(hidden=hidden)
    close(got[1], lse, tol_lse, "lse")
    close(got[0], out, tol, "out")
