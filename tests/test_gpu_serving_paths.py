"""paged_attention's ways that long tables and pages of 16 tokens do not take: one
launch over short caches in every type, pages whose size is no multiple of 16
with places that do not exist, and the beam search example over an FP8 cache at
the bound of the rounding that it really has."""
import math
import os
import sys

import pytest
import torch

import mixed_precision_dense_tiled_amd as mp
from serving_ref import Batch, close, e4m3

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu
bf16, f16 = torch.bfloat16, torch.float16
TYPES = [(bf16, False), (f16, False), (bf16, True), (f16, True)]

SHORT = [(1, 1), (1, 2), (1, 31), (1, 33), (1, 517), (1, 0), (1, 64), (1, 900), (2, 700), (3, 2)]


def check(b, **k):
    out, lse = mp.paged_attention(**b.gpu(), return_lse=True, **k)
    o, z, tol, tol_z = b.attention(**k)
    close(lse, z, tol_z, "lse")
    close(out, o, tol, "out")
    return out, lse


@pytest.mark.parametrize("dim", [16, 64, 80, 96, 128])
@pytest.mark.parametrize("dtype, fp8", TYPES)
@pytest.mark.parametrize("how", ["plain", "cap", "window", "junk"])
def test_one_launch(gpu_ok, dim, dtype, fp8, how):
    b = Batch(SHORT, 8, 2, dim, 16, dtype, fp8, seed=dim + 50, junk=how == "junk")
    assert b.table.shape[1] * b.page <= 1024
    out, lse = check(b, softcap=20.0 if how == "cap" else 0.0, window=77 if how == "window" else 0)
    assert not out.isnan().any() and not lse.isnan().any()


@pytest.mark.parametrize("page", [1, 3, 24, 100])
@pytest.mark.parametrize("dtype, fp8", TYPES)
def test_one_launch_page_sizes(gpu_ok, page, dtype, fp8):
    check(Batch(SHORT, 4, 1, 64, page, dtype, fp8, seed=page + 60))


@pytest.mark.parametrize("heads", [1, 7, 16, 24])
def test_one_launch_head_sharing(gpu_ok, heads):
    check(Batch([(1, 200), (1, 90), (1, 0)], heads, 1, 64, 16, f16, seed=heads))


LONG = [(1, 1300), (1, 7), (1, 90), (2, 400)]
CHUNKS = [(70, 1300), (33, 50), (9, 4), (120, 500)]


@pytest.mark.parametrize("page", [3, 24, 100])
@pytest.mark.parametrize("seqs", [SHORT, LONG, CHUNKS], ids=["one_launch", "shared_out", "chunks"])
@pytest.mark.parametrize("dtype, fp8", [(bf16, False), (f16, True)])
@pytest.mark.parametrize("window", [0, 50])
def test_odd_pages_beyond_a_sequence_are_not_read(gpu_ok, page, seqs, dtype, fp8, window):
    out, lse = check(Batch(seqs, 4, 2, 80, page, dtype, fp8, seed=page + 70, junk=True), window=window)
    assert not out.isnan().any() and not lse.isnan().any()


@pytest.mark.parametrize("page", [3, 16, 24])
@pytest.mark.parametrize("seqs", [[(1, 300), (1, 600), (1, 40)], [(1, 300), (1, 1600), (1, 40)],
                                  [(60, 300), (100, 600), (30, 40)]], ids=["one_launch", "shared_out", "chunks"])
@pytest.mark.parametrize("dtype, fp8", [(bf16, False), (bf16, True)])
def test_odd_pages_that_do_not_exist_hold_no_keys(gpu_ok, page, seqs, dtype, fp8):
    b = Batch(seqs, 4, 2, 64, page, dtype, fp8, seed=page + 80)
    gone = {0: [3, 7], 1: [0, 11], 2: list(range(-(-40 // page)))}
    for s, (entries, value) in enumerate(zip(gone.values(), (-1, b.pages, 2 ** 31 - 1))):
        for e in entries:
            b.table[s, e] = value

    def hidden(i):
        m = torch.zeros(b.seqs[i][1], dtype=torch.bool)
        for p in gone[i]:
            m[page * p:page * p + page] = True
        return m

    got = mp.paged_attention(**b.gpu(), return_lse=True)
    b.table = torch.where((b.table < 0) | (b.table >= b.pages), 0, b.table)     # for the definition's own reads
    out, lse, tol, tol_z = b.attention(hidden=hidden)
    close(got[1], lse, tol_z, "lse")
    close(got[0], out, tol, "out")
    assert (got[0][b.cu[2]:] == 0).all() and (got[1][b.cu[2]:] == -math.inf).all()


def plain_logprob(model, text, start, scale):
    """Sum of log probabilities of text[start:] without a cache; keys and values are
    what an E4M3 cache holds of their BF16 values."""
    import beam_search as bs
    f = lambda t: t.float().cpu()  # noqa: E731
    x = f(model.embed)[torch.tensor(text)]
    y = (x @ f(model.qkv)).to(bf16).float().view(-1, bs.HEADS + 2 * bs.KV_HEADS, bs.DIM)
    q = y[:, :bs.HEADS]
    k, v = (e4m3(t.double() / scale).float() * scale
            for t in (y[:, bs.HEADS:bs.HEADS + bs.KV_HEADS], y[:, bs.HEADS + bs.KV_HEADS:]))
    out = torch.empty(len(text), bs.HEADS, bs.DIM)
    hide = torch.ones(len(text), len(text)).triu(1).bool()
    for h in range(bs.HEADS):
        kv = h // (bs.HEADS // bs.KV_HEADS)
        s = (q[:, h] @ k[:, kv].T * bs.DIM ** -0.5).masked_fill(hide, -math.inf)
        out[:, h] = s.softmax(-1) @ v[:, kv]
    x = out.reshape(len(text), -1) @ f(model.out) + x
    lp = torch.log_softmax(x @ f(model.head), -1)
    return sum(float(lp[i - 1, text[i]]) for i in range(start, len(text)))


def test_beams_over_fp8(gpu_ok):
    import beam_search as bs
    model, steps, beams = bs.Decoder(), 20, 4
    prompts = [[5, 17, 200, 3, 9], list(range(100, 137)), [7] * 16]
    text, score, _ = bs.search(model, prompts, beams, steps, fp8=True)
    # what is left besides the cache's own rounding: q, k, v, the attended values and the
    # hidden state in BF16, 2^-8 of values of order one, through logits' weights of
    # size 4, in each of `steps` log probabilities
    tol = steps * 4 * 2.0 ** -8
    for i, t in enumerate(text):
        p = prompts[i // beams]
        assert abs(plain_logprob(model, t, len(p), 1.0 / 64) - float(score[i])) < tol
