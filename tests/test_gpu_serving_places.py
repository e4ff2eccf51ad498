"""Where a new token lies: paged_kv_append and paged_attention cut lengths and
offsets that leave the batch in the same way, so that the keys one writes are
the keys the other reads."""
import pytest
import torch

import mixed_precision_dense_tiled_amd as mp
from serving_ref import Batch

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# (cu_q, lens) as given, and as cut to 9 tokens and 4 pages of 16
CUT = [([0, 4, 9], [20, 10 ** 9], [0, 4, 9], [20, 64]),
       ([0, 4, 9], [65, 2 ** 31 - 1], [0, 4, 9], [64, 64]),
       ([-3, 4, 10 ** 9], [20, 30], [0, 4, 9], [20, 30]),
       ([-5, 4, 12], [40, 64], [0, 4, 9], [40, 64]),
       ([0, 9, 9], [70, 5], [0, 9, 9], [64, 5]),
       ([0, 20, 30], [50, 5], [0, 9, 9], [50, 5]),
       ([0, 4, 9], [-7, 30], [0, 4, 9], [0, 30])]


@pytest.mark.parametrize("cu, lens, cu_cut, lens_cut", CUT)
@pytest.mark.parametrize("copies", [1, 40], ids=["few", "many"])
def test_append_cuts_as_attention_does(gpu_ok, cu, lens, cu_cut, lens_cut, copies):
    """copies: 80 sequences are looked up another way than two (the others are empty)."""
    b = Batch([(4, 60), (5, 64)] + [(0, 0)] * (2 * copies - 2), 2, 2, 64, 16, seed=5)
    b.table = b.table[:, :4].contiguous()
    more = 2 * copies - 2
    cu, cu_cut = cu + [cu[-1]] * more, cu_cut + [9] * more
    lens, lens_cut = lens + [0] * more, lens_cut + [0] * more
    g = b.gpu()
    q = g.pop("q")
    k, v = (torch.randn(9, 2, 64, device="cuda").to(bf16) for _ in range(2))
    a, c = ({**g, "k_cache": g["k_cache"].clone(), "v_cache": g["v_cache"].clone()} for _ in range(2))
    a.update(cu_q=i32(cu), lens=i32(lens))
    c.update(cu_q=i32(cu_cut), lens=i32(lens_cut))
    for x in (a, c):
        mp.paged_kv_append(k, v, **x)
    # by the definition: row i of sequence s at position n - nq + i
    want = g["k_cache"].clone(), g["v_cache"].clone()
    for s in range(2):
        n, start, nq = lens_cut[s], cu_cut[s], cu_cut[s + 1] - cu_cut[s]
        for i in range(nq):
            pos = n - nq + i
            if pos >= 0:
                pg = int(b.table[s, pos // 16])
                if pg >= 0:
                    want[0][pg, pos % 16], want[1][pg, pos % 16] = k[start + i], v[start + i]
    for x in (a, c):
        assert torch.equal(x["k_cache"], want[0]) and torch.equal(x["v_cache"], want[1])
    one, two = (mp.paged_attention(q, **x, return_lse=True) for x in (a, c))
    last = cu_cut[-1]
    assert torch.equal(one[0][:last], two[0][:last]) and torch.equal(one[1][:last], two[1][:last])
