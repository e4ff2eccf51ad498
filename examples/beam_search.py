"""Beam search over a paged cache: the serving operators as a program uses them.

A one-layer decoder with random weights takes in prompts (their keys and values
appended to the cache, attention over it), forks each prompt into beams that
share its pages, and lets them grow token by token: cache_extend makes room,
paged_kv_append and paged_attention run the layer, token_logprobs names the
best continuations, cache_fork moves beams to their parents' pages and
cache_free gives up the old ones.  At the end cache_compact brings what is left
together.

    python examples/beam_search.py [--fp8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mixed_precision_dense_tiled_amd as mp  # noqa: E402

VOCAB, WIDTH, HEADS, KV_HEADS, DIM, PAGE = 1000, 512, 8, 2, 64, 16


class Decoder:
    """Embedding, one attention layer, logits; BF16 weights from a seed."""

    def __init__(self, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=g, device=device) * rows ** -0.5).to(torch.bfloat16)

        self.embed = torch.randn(VOCAB, WIDTH, generator=g, device=device).to(torch.bfloat16)
        self.qkv = weight(WIDTH, (HEADS + 2 * KV_HEADS) * DIM)
        self.out = weight(HEADS * DIM, WIDTH)
        self.head = weight(WIDTH, VOCAB) * 4

    def split(self, tokens):
        """Hidden state, and q, k, v of the tokens."""
        x = self.embed[tokens]
        y = mp.gemm_bf16_bf16out(x, self.qkv).view(-1, HEADS + 2 * KV_HEADS, DIM)
        return x, y[:, :HEADS], y[:, HEADS:HEADS + KV_HEADS], y[:, HEADS + KV_HEADS:]

    def logits(self, x, attended):
        x = mp.gemm_bf16_bf16out(attended.reshape(-1, HEADS * DIM), self.out, x.float())
        return mp.gemm_bf16(x, self.head)


class Cache:
    """The pages of one layer (plane 0: K, plane 1: V) and who holds them.  Rows
    come in two halves, so that a step forks beams from one half into the other."""

    def __init__(self, rows, pages=256, width=16, fp8=False, device="cuda"):
        dtype = torch.float8_e4m3fn if fp8 else torch.bfloat16
        self.kv = torch.zeros(2, pages, PAGE, KV_HEADS, DIM, device=device).to(dtype)
        self.scale = torch.full((KV_HEADS,), 1.0 / 64, device=device) if fp8 else None
        self.refs = torch.zeros(pages, dtype=torch.int32, device=device)
        self.table = torch.full((2 * rows, width), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(2 * rows, dtype=torch.int32, device=device)
        self.rows, self.device = rows, device

    def ints(self, values):
        return torch.tensor(values, dtype=torch.int32, device=self.device)

    def grow(self, add):
        return mp.cache_extend(self.refs, self.table, self.lens, self.ints(add), PAGE)

    def attend(self, q, k, v, cu):
        args = dict(table=self.table, cu_q=self.ints(cu), lens=self.lens, k_scale=self.scale, v_scale=self.scale)
        mp.paged_kv_append(k, v, self.kv[0], self.kv[1], **args)
        return mp.paged_attention(q, self.kv[0], self.kv[1], **args)

    def move(self, parent):
        """Rows of the other half become copies of their parents; the old half is
        given up."""
        short = mp.cache_fork(self.kv, self.refs, self.table, self.lens, self.ints(parent), PAGE)
        mp.cache_free(self.refs, self.table, self.lens, self.ints([int(p < 0) for p in parent]), PAGE)
        return short


def search(model, prompts, beams, steps, fp8=False):
    """The best `beams` continuations of each prompt: (tokens, log probability)."""
    n = len(prompts) * beams
    cache = Cache(n, fp8=fp8)
    half = 0                                   # where the live rows are
    rows = 2 * n

    def offsets(counts):
        cu = [0]
        for c in counts:
            cu.append(cu[-1] + c)
        return cu

    # the prompts, each as the first row of its beams
    counts = [0] * rows
    for i, p in enumerate(prompts):
        counts[i * beams] = len(p)
    missing = cache.grow(counts)
    tokens = torch.tensor([t for p in prompts for t in p], device="cuda")
    x, q, k, v = model.split(tokens)
    last = torch.tensor(offsets([len(p) for p in prompts])[1:], device="cuda") - 1
    logits = model.logits(x[last], cache.attend(q, k, v, offsets(counts))[last])
    none = torch.full((len(prompts),), -100, device="cuda")
    best = mp.token_logprobs(logits, none, top_k=beams)
    score = best.top_logprobs.reshape(-1)
    text = [list(prompts[i]) + [t] for i, row in enumerate(best.top_indices.tolist()) for t in row]
    parents = [i * beams for i in range(len(prompts)) for _ in range(beams)]

    for step in range(steps - 1):
        # every beam into the other half, as a copy of its parent
        other = n - half
        parent = [-1] * rows
        for r, p in enumerate(parents):
            parent[other + r] = half + p
        missing = missing + cache.move(parent)
        half = other
        counts = [0] * rows
        counts[half:half + n] = [1] * n
        missing = missing + cache.grow(counts)
        x, q, k, v = model.split(torch.tensor([t[-1] for t in text], device="cuda"))
        logits = model.logits(x, cache.attend(q, k, v, offsets(counts)))
        best = mp.token_logprobs(logits, torch.full((n,), -100, device="cuda"), top_k=beams)
        total = (score[:, None] + best.top_logprobs).view(len(prompts), beams * beams)
        score, pick = total.topk(beams, dim=-1)
        score = score.reshape(-1)
        pick = pick.tolist()
        choice = best.top_indices.view(len(prompts), beams * beams).tolist()
        parents = [i * beams + c // beams for i, row in enumerate(pick) for c in row]
        text = [text[p] + [choice[i][c]] for (i, c), p in
                zip([(i, c) for i, row in enumerate(pick) for c in row], parents)]
    mp.cache_compact(cache.kv, cache.refs, cache.table, cache.lens, PAGE)
    assert int(missing) == 0, "the cache has too few pages"
    return text, score, cache


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--fp8", action="store_true", help="cache in 8 bits")
    args = ap.parse_args()
    prompts = [[5, 17, 200, 3, 9], list(range(100, 137))]
    text, score, cache = search(Decoder(), prompts, beams=3, steps=12, fp8=args.fp8)
    for t, s in zip(text, score.tolist()):
        print(f"{s:9.3f}  {t[-12:]}")
    print("pages in use:", int((cache.refs > 0).sum()), "of", cache.refs.numel())


if __name__ == "__main__":
    main()
