"""A decoder layer of experts: the layer operators as a program uses them.

Serving, in 8 bits: rms_norm adds the residual and hands INT8 rows with their
scales to the W8A8 projection; paged_kv_append_rope turns the queries where they
lie in the projection's rows and puts the keys, turned too, and the values into
the paged cache; paged_attention reads it; and each token's rows go through the
experts that the router picks, by gemm_grouped_w8a8.  Nothing comes back to the
host on the way.

Training: one step through the norm and the experts in BF16, with the gradients
of the rows, the norm's weight and every expert's matrices.

    python examples/expert_layer.py
"""
import os
import sys
from collections import namedtuple

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mixed_precision_dense_tiled_amd as mp  # noqa: E402

WIDTH, HEADS, KV_HEADS, DIM, PAGE = 512, 8, 2, 64, 16
EXPERTS, TOP, INNER = 8, 2, 384

Routed = namedtuple("Routed", "token offsets gate place")


def route(logits):
    """Rows sorted by expert: which token each is, where each expert's begin, the
    tokens' gates, and where a token's rows are."""
    tokens = logits.shape[0]
    best = logits.float().topk(TOP, dim=-1)
    gate = best.values.softmax(-1)
    expert = best.indices.reshape(-1)
    order = torch.argsort(expert, stable=True)
    counts = (expert[:, None] == torch.arange(EXPERTS, device=logits.device)).sum(0)
    offsets = torch.zeros(EXPERTS + 1, dtype=torch.int32, device=logits.device)
    offsets[1:] = counts.cumsum(0)
    place = torch.empty_like(order)
    place[order] = torch.arange(tokens * TOP, device=logits.device)
    return Routed(order // TOP, offsets, gate, place.view(tokens, TOP))


def in_8_bits(w):
    """A weight [.., out, in] as INT8 with a scale for each output channel."""
    scale = w.abs().amax(-1) / 127
    return torch.round(w / scale[..., None]).to(torch.int8), scale


class Cache:
    """Pages of one layer and which sequence has which."""

    def __init__(self, seqs, pages=64, width=16, device="cuda"):
        self.k, self.v = (torch.zeros(pages, PAGE, KV_HEADS, DIM, dtype=torch.bfloat16, device=device)
                          for _ in range(2))
        self.refs = torch.zeros(pages, dtype=torch.int32, device=device)
        self.table = torch.full((seqs, width), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(seqs, dtype=torch.int32, device=device)

    def grow(self, add):
        return mp.cache_extend(self.refs, self.table, self.lens, add, PAGE)


class Layer:
    """Weights from a seed, in 8 bits; norms in BF16."""

    def __init__(self, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape):
            return in_8_bits(torch.randn(*shape, generator=g, device=device) * shape[-1] ** -0.5)

        self.norm1, self.norm2 = (1 + 0.1 * torch.randn(2, WIDTH, generator=g, device=device)).to(torch.bfloat16)
        self.qkv = weight((HEADS + 2 * KV_HEADS) * DIM, WIDTH)
        self.out = weight(WIDTH, HEADS * DIM)
        self.router = weight(EXPERTS, WIDTH)
        self.up = weight(EXPERTS, 2 * INNER, WIDTH)
        self.down = weight(EXPERTS, WIDTH, INNER)
        self.inv_freq = (10000.0 ** (-torch.arange(0, DIM, 2, device=device) / DIM)).float()

    def __call__(self, x, residual, cache, cu, trace=None):
        """The layer's output and residual for new tokens x [tokens, WIDTH] (rows cu[b] to
        cu[b + 1] of sequence b, whose cache has room for them)."""
        keep = {} if trace is None else trace
        where = dict(table=cache.table, cu_q=cu, lens=cache.lens)
        n1 = keep["n1"] = mp.rms_norm(x, self.norm1, residual=residual, quant="int8")
        qkv = mp.gemm_w8a8(n1.out, n1.scales, *self.qkv).view(-1, HEADS + 2 * KV_HEADS, DIM)
        keep["qkv"] = None if trace is None else qkv.clone()
        q, k, v = qkv.split([HEADS, KV_HEADS, KV_HEADS], dim=1)
        keep["q"] = mp.paged_kv_append_rope(q, k, v, cache.k, cache.v, inv_freq=self.inv_freq, out=q, **where)
        att = keep["att"] = mp.paged_attention(q, cache.k, cache.v, **where)
        y = keep["y"] = mp.gemm_w8a8(*mp.quantize_i8_rows(att.view(-1, HEADS * DIM)), *self.out)
        n2 = keep["n2"] = mp.rms_norm(y, self.norm2, residual=n1.residual, quant="int8")
        r = keep["r"] = route(mp.gemm_w8a8(n2.out, n2.scales, *self.router))
        h = keep["h"] = mp.gemm_grouped_w8a8(n2.out[r.token], n2.scales[r.token], *self.up, r.offsets)
        gate, up = h.float().split(INNER, dim=-1)
        a = keep["a"] = mp.quantize_i8_rows((torch.nn.functional.silu(gate) * up).to(torch.bfloat16))
        z = keep["z"] = mp.gemm_grouped_w8a8(*a, *self.down, r.offsets)
        return (z[r.place].float() * r.gate[..., None]).sum(1).to(torch.bfloat16), n2.residual


def serve(layer, prompts, steps, seed=1):
    """Prompts in one call, then single tokens; random rows in the place of a model's.
    Returns the outputs of every call and the cache."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    cache = Cache(len(prompts))
    missing, outs, counts = 0, [], prompts
    for _ in range(1 + steps):
        add = torch.tensor(counts, dtype=torch.int32, device="cuda")
        cu = torch.zeros(len(counts) + 1, dtype=torch.int32, device="cuda")
        cu[1:] = add.cumsum(0)
        missing = missing + cache.grow(add)
        x, residual = torch.randn(2, sum(counts), WIDTH, generator=g, device="cuda").to(torch.bfloat16)
        outs.append(layer(x, residual, cache, cu))
        counts = [1] * len(prompts)
    assert int(missing) == 0, "the cache has too few pages"
    return outs, cache


Grads = namedtuple("Grads", "x weight up down")


def train_step(x, residual, weight, up, down, routed, grad_out, grad_residual):
    """y = sum over a token's experts of gate * silu(norm(x + residual) . up) . down in BF16, and
    the gradients from those in y and in x + residual.  up [EXPERTS, WIDTH, INNER], down
    [EXPERTS, INNER, WIDTH]; the routing is given."""
    n = mp.rms_norm(x, weight, residual=residual, return_rstd=True)
    rows = n.out[routed.token]
    h = mp.gemm_grouped(rows, up, routed.offsets, d16=True)
    a = torch.nn.functional.silu(h.float()).to(h.dtype)
    z = mp.gemm_grouped(a, down, routed.offsets, d16=True)
    y = (z[routed.place].float() * routed.gate[..., None]).sum(1).to(x.dtype)

    gate = torch.empty(rows.shape[0], 1, device=x.device)
    gate[routed.place.reshape(-1)] = routed.gate.reshape(-1, 1)
    gz = (grad_out[routed.token].float() * gate).to(x.dtype)
    ga = mp.gemm_grouped(gz, down, routed.offsets, trans_b=True)
    s = torch.sigmoid(h.float())
    gh = (ga * (s + h.float() * s * (1 - s))).to(x.dtype)
    g_rows = mp.gemm_grouped(gh, up, routed.offsets, trans_b=True)
    g_norm = g_rows[routed.place].sum(1).to(x.dtype)
    gx, gw = mp.rms_norm_backward(g_norm, n.residual, weight, n.rstd, grad_residual=grad_residual)
    return y, Grads(gx, gw, mp.gemm_grouped_wgrad(rows, gh, routed.offsets),
                    mp.gemm_grouped_wgrad(a, gz, routed.offsets))


def main():
    outs, cache = serve(Layer(), [5, 40, 17], 8)
    print(f"served {sum(o[0].shape[0] for o in outs)} tokens; lengths {cache.lens.tolist()}")
    g = torch.Generator(device="cuda").manual_seed(2)
    x, residual, gy, gr = torch.randn(4, 200, WIDTH, generator=g, device="cuda").to(torch.bfloat16)
    up = (torch.randn(EXPERTS, WIDTH, INNER, generator=g, device="cuda") * WIDTH ** -0.5).to(torch.bfloat16)
    down = (torch.randn(EXPERTS, INNER, WIDTH, generator=g, device="cuda") * INNER ** -0.5).to(torch.bfloat16)
    routed = route(torch.randn(200, EXPERTS, generator=g, device="cuda"))
    _, grads = train_step(x, residual, torch.ones(WIDTH, dtype=torch.bfloat16, device="cuda"), up, down, routed, gy, gr)
    print("gradients:", ", ".join(f"{n} {tuple(t.shape)}" for n, t in zip(grads._fields, grads)))


if __name__ == "__main__":
    main()
