"""Capped scores over the whole range of caps, from one that flattens every
score to one that is as good as none, through every kernel of paged_attention,
with bounds that follow the score and not the cap."""
import math

import pytest
import torch

import mixed_precision_dense_tiled_amd as mp
from serving_ref import EPS, Batch, close

pytestmark = pytest.mark.gpu
bf16, f16 = torch.bfloat16, torch.float16
U = EPS[torch.float32]


def capped(b, softcap, scale, window=0):
    """out, lse and their bounds in FP64.  A score s = scale * (q . k) is off by
    (dim + 4) roundings of its products' sizes and four of its own; the cap's slope
    is at most 1, and its evaluation adds 16 roundings of the capped score c = cap
    * tanh(s / cap): up to 0.5 of y = s / cap a polynomial (half a rounding) whose
    argument, constants and products add 8; above it 1 - 2 / (e^2y + 1), where the
    exponent's five roundings weigh y (1 - tanh^2) / tanh <= 0.85 each, exponential and
    reciprocal (two each) 0.85 and 1.2, the sum and the difference 1.2 and 1, the
    factor 1."""
    out = torch.zeros(b.q.shape, dtype=torch.float64)
    lse = torch.full(b.q.shape[:2], -math.inf, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    ep = EPS[torch.float16] if b.scales[0] is not None else EPS[b.dtype]
    for i, (nq, n) in enumerate(b.seqs):
        if not nq or not n:
            continue
        rows = slice(int(b.cu[i]), int(b.cu[i + 1]))
        pos, tok = torch.arange(n - nq, n)[:, None], torch.arange(n)
        see = tok <= pos
        if window:
            see &= tok > pos - window
        some = see.any(-1)
        for h in range(b.heads):
            kvh = h // (b.heads // b.kv_heads)
            q, k, v = b.q[rows, h].double(), b.keys(i, kvh, 0), b.keys(i, kvh, 1)
            s = scale * (q @ k.T)
            c = softcap * torch.tanh(s / softcap)
            ds = (b.dim + 4) * U * abs(scale) * (q.abs() @ k.abs().T) + 4 * U * s.abs() + 16 * U * c.abs()
            # (a score's size where the cap holds it down adds nothing: both ends of the error are below the cap)
            ds = torch.minimum(ds, 2 * c.abs() + 16 * U * c.abs())
            c = c.masked_fill(~see, -math.inf)
            z = torch.logsumexp(c, -1)
            p = torch.where(see, torch.exp(c - z.masked_fill(~some, 0.0)[:, None]), torch.zeros_like(c))
            d = torch.where(see, ds, torch.zeros_like(ds)).amax(-1)
            o = p @ v
            out[rows, h], lse[rows, h] = o, z
            rel = 2 * d + (2 * n + 16) * U
            tol[rows, h] = (p @ v.abs()) * (ep + rel)[:, None] * 1.01 + EPS[b.dtype] * o.abs() * 1.01 + 1e-7
            tol_lse[rows, h] = d + (n + 16) * U + 4 * U * z.masked_fill(~some, 0.0).abs()
    return out, lse, tol, tol_lse


ONE_LAUNCH = [(1, 1), (1, 2), (1, 33), (1, 300), (1, 0), (1, 64)]
SHARED_OUT = ONE_LAUNCH + [(1, 1200)]
CHUNKS = [(40, 40), (1, 300), (130, 400), (0, 21), (9, 4), (65, 64)]


@pytest.mark.parametrize("softcap", [1e-38, 1e-3, 0.5, 5.0, 50.0, 1e3, 1e5, 1e7, 1e9, 1e30, 3e38])
@pytest.mark.parametrize("seqs", [ONE_LAUNCH, SHARED_OUT, CHUNKS], ids=["one_launch", "shared_out", "chunks"])
@pytest.mark.parametrize("dtype, fp8", [(bf16, False), (f16, True)])
def test_caps(gpu_ok, softcap, seqs, dtype, fp8):
    b = Batch(seqs, 4, 2, 64, 16, dtype, fp8, seed=40)
    scale = 0.25
    got = mp.paged_attention(**b.gpu(), return_lse=True, scale=scale, softcap=softcap)
    out, lse, tol, tol_lse = capped(b, softcap, scale)
    close(got[1], lse, tol_lse, f"cap {softcap} lse")
    close(got[0], out, tol, f"cap {softcap} out")


@pytest.mark.parametrize("scale", [20.0, -3.0])
@pytest.mark.parametrize("softcap", [1e-38, 30.0, 1e4])
@pytest.mark.parametrize("seqs", [SHARED_OUT, CHUNKS], ids=["singles", "chunks"])
def test_scores_of_every_size_under_one_cap(gpu_ok, scale, softcap, seqs):
    """Scores in the hundreds, near zero and exactly zero side by side."""
    b = Batch(seqs, 4, 2, 80, 16, f16, seed=41)
    g = torch.Generator().manual_seed(42)
    b.q = (b.q.float() * 2.0 ** -torch.randint(0, 12, b.q.shape[:2], generator=g)[..., None].float()).to(f16)
    b.q[::3, 1] = 0
    got = mp.paged_attention(**b.gpu(), return_lse=True, scale=scale, softcap=softcap, window=500)
    out, lse, tol, tol_lse = capped(b, softcap, scale, window=500)
    close(got[1], lse, tol_lse, "lse")
    close(got[0], out, tol, "out")


@pytest.mark.parametrize("dim", [80, 96, 112, 128])
@pytest.mark.parametrize("dtype, fp8", [(bf16, False), (f16, False), (bf16, True), (f16, True)])
@pytest.mark.parametrize("seqs", [ONE_LAUNCH, SHARED_OUT, CHUNKS], ids=["one_launch", "shared_out", "chunks"])
def test_caps_over_wide_heads(gpu_ok, dim, dtype, fp8, seqs):
    b = Batch(seqs, 4, 2, dim, 16, dtype, fp8, seed=dim + 1)
    got = mp.paged_attention(**b.gpu(), return_lse=True, scale=0.2, softcap=4.0, window=250)
    out, lse, tol, tol_lse = capped(b, 4.0, 0.2, window=250)
    close(got[1], lse, tol_lse, "lse")
    close(got[0], out, tol, "out")


@pytest.mark.parametrize("softcap", [0.0, 5.0, 1e4])
@pytest.mark.parametrize("seqs", [ONE_LAUNCH, SHARED_OUT, CHUNKS], ids=["one_launch", "shared_out", "chunks"])
def test_a_head_whose_scale_is_no_number(gpu_ok, softcap, seqs):
    """Its outputs are none, with a cap as without one; the other head's are as ever."""
    b = Batch(seqs, 4, 2, 64, 16, bf16, True, seed=43)
    some = torch.cat([torch.arange(n - nq, n) >= 0 for nq, n in seqs if nq])
    g = b.gpu()
    want = mp.paged_attention(**g, return_lse=True, softcap=softcap)
    g["k_scale"][1] = math.nan
    out, lse = mp.paged_attention(**g, return_lse=True, softcap=softcap)
    assert torch.equal(out[:, :2], want[0][:, :2]) and torch.equal(lse[:, :2], want[1][:, :2])
    assert out[some][:, 2:].isnan().all() and lse[some][:, 2:].isnan().all()
    assert (out[~some] == 0).all() and (lse[~some] == -math.inf).all()
