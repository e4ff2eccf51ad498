"""The beam search example end to end: the log probability of each beam, as the
cache's operators gave it step by step, against a plain recomputation of the
whole text in FP32; and the cache's bookkeeping at the end."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def plain_logprob(model, text, start):
    """Sum of log probabilities of text[start:], without a cache."""
    import beam_search as bs
    f = lambda t: t.float().cpu()  # noqa: E731
    tokens = torch.tensor(text)
    x = f(model.embed)[tokens]
    y = (x @ f(model.qkv)).view(-1, bs.HEADS + 2 * bs.KV_HEADS, bs.DIM)
    q, k, v = y[:, :bs.HEADS], y[:, bs.HEADS:bs.HEADS + bs.KV_HEADS], y[:, bs.HEADS + bs.KV_HEADS:]
    out = torch.empty(len(text), bs.HEADS, bs.DIM)
    hide = torch.ones(len(text), len(text)).triu(1).bool()
    for h in range(bs.HEADS):
        kv = h // (bs.HEADS // bs.KV_HEADS)
        s = (q[:, h] @ k[:, kv].T * bs.DIM ** -0.5).masked_fill(hide, float("-inf"))
        out[:, h] = s.softmax(-1) @ v[:, kv]
    x = out.reshape(len(text), -1) @ f(model.out) + x
    lp = torch.log_softmax(x @ f(model.head), -1)
    return sum(float(lp[i - 1, text[i]]) for i in range(start, len(text)))


@pytest.mark.parametrize("fp8", [False, True])
def test_beams(gpu_ok, fp8):
    import beam_search as bs
    model = bs.Decoder()
    prompts = [[5, 17, 200, 3, 9], list(range(100, 137)), [7] * 16]
    steps, beams = 20, 4
    text, score, cache = bs.search(model, prompts, beams, steps, fp8=fp8)
    assert len(text) == len(prompts) * beams and len({tuple(t) for t in text}) == len(text)
    # q, k, v, the attended values and the hidden state are rounded to BF16 (2^-8 of
    # values of order one; an FP8 cache: 2^-4 of keys and values), which the
    # logits' weights of size 4 carry into each of `steps` log probabilities
    tol = steps * 4 * 2.0 ** -8 if not fp8 else steps * 4 * 2.0 ** -4
    for i, t in enumerate(text):
        p = prompts[i // beams]
        assert t[:len(p)] == p and len(t) == len(p) + steps
        assert abs(plain_logprob(model, t, len(p)) - float(score[i])) < tol
    # what the cache holds: every page of a row counted, compacted to the front
    refs = torch.zeros_like(cache.refs)
    for row, n in zip(cache.table.tolist(), cache.lens.tolist()):
        for pg in row[:-(-n // bs.PAGE)]:
            refs[pg] += 1
    assert torch.equal(refs, cache.refs)
    live = int((refs > 0).sum())
    assert (refs[:live] > 0).all() and (refs[live:] == 0).all()
    assert sorted(cache.lens.tolist()) == sorted([0] * len(text) + [len(t) - 1 for t in text])
