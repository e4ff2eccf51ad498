"""The expert layer example end to end: every step of the served layer against its
definition, from what the step before it gave; and the training step's gradients
against autograd's in 64 bits, with the same roundings on the way."""
import os
import sys

import pytest
import torch

from layers_ref import HALF, U, norm_rows, norm_rstd, norm_sum, quantise, rope

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16


def cpu(x):
    if isinstance(x, torch.Tensor):
        return x.cpu()
    return type(x)(*map(cpu, x)) if hasattr(x, "_fields") else tuple(map(cpu, x)) if isinstance(x, tuple) else x


def linear(codes, scales, weight):
    """gemm_w8a8's own steps."""
    w, s = weight
    z = (codes.double() @ w.double().T).float()
    return ((z * scales[:, None]) * s).to(bf16)


def test_served_layer(gpu_ok):
    import expert_layer as ex
    layer = ex.Layer()
    cache = ex.Cache(3)
    g = torch.Generator(device="cuda").manual_seed(1)
    W = {n: cpu(getattr(layer, n)) for n in ("norm1", "norm2", "qkv", "out", "router", "up", "down", "inv_freq")}
    lens = [0, 0, 0]
    keys = [[], [], []]
    for counts in ([5, 40, 17], [1, 1, 1], [0, 3, 1], [1, 1, 1]):
        add = torch.tensor(counts, dtype=torch.int32, device="cuda")
        cu = torch.tensor([0, counts[0], counts[0] + counts[1], sum(counts)], dtype=torch.int32, device="cuda")
        assert int(cache.grow(add)) == 0
        x, res = torch.randn(2, sum(counts), ex.WIDTH, generator=g, device="cuda").to(bf16)
        t = {}
        out, residual = layer(x, res, cache, cu, trace=t)
        t = {n: cpu(v) for n, v in t.items()}
        # norm, in 8 bits, code for code; then the projection bit for bit
        h = norm_sum(cpu(x), cpu(res))
        values, scales = quantise(norm_rows(h, W["norm1"], 1e-6), "int8")
        assert torch.equal(t["n1"].residual, h)
        assert torch.equal(t["n1"].out.float(), values) and torch.equal(t["n1"].scales, scales)
        qkv = linear(t["n1"].out, t["n1"].scales, W["qkv"])
        assert torch.equal(t["qkv"].reshape(qkv.shape), qkv)
        qkv = qkv.view(-1, ex.HEADS + 2 * ex.KV_HEADS, ex.DIM)
        # turned queries and keys; attention over the turned keys that the cache holds
        pos = torch.cat([torch.arange(n, n + c) for n, c in zip(lens, counts)])
        turned, off = rope(qkv[:, :ex.HEADS + ex.KV_HEADS], pos, W["inv_freq"], False)
        err = (t["q"].double() - turned[:, :ex.HEADS]).abs()
        assert (err <= off[:, :ex.HEADS] + HALF[bf16] * turned[:, :ex.HEADS].abs() * 1.02 + 1e-30).all()
        at = 0
        kc, vc, table = cpu(cache.k), cpu(cache.v), cpu(cache.table)
        for b, c in enumerate(counts):
            n = lens[b] + c
            p = torch.arange(n)
            k, v = (z[table[b, p // ex.PAGE].long(), p % ex.PAGE].double() for z in (kc, vc))
            new = slice(at, at + c)
            keys[b].append(turned[new, ex.HEADS:])
            if n:
                want = torch.cat(keys[b])
                assert ((k - want).abs() <= 2.0 ** -8 * want.abs() * 1.02 + 1e-5).all()
            for head in range(ex.HEADS):
                s = t["q"][new, head].double() @ k[:, head // 4].T * ex.DIM ** -0.5
                s = s.masked_fill(p[None] > (lens[b] + torch.arange(c))[:, None], float("-inf"))
                w = s.softmax(-1)
                want = w @ v[:, head // 4]
                # weights and the result rounded to BF16
                assert ((t["att"][new, head].double() - want).abs() <= 2.0 ** -7 * (w @ v[:, head // 4].abs()) + 1e-5).all()
            at += c
            lens[b] = n
        # the experts, from the second norm's codes
        h = norm_sum(t["y"], t["n1"].residual)
        values, scales = quantise(norm_rows(h, W["norm2"], 1e-6), "int8")
        assert torch.equal(cpu(residual), h) and torch.equal(t["n2"].out.float(), values)
        r = t["r"]
        offsets = r.offsets.tolist()
        assert offsets[-1] == ex.TOP * sum(counts) and offsets == sorted(offsets)
        for e in range(ex.EXPERTS):
            rows = slice(offsets[e], offsets[e + 1])
            tok = r.token[rows]
            assert torch.equal(t["h"][rows], linear(t["n2"].out[tok], t["n2"].scales[tok], (W["up"][0][e], W["up"][1][e])))
            assert torch.equal(t["z"][rows], linear(t["a"][0][rows], t["a"][1][rows], (W["down"][0][e], W["down"][1][e])))
        want = (t["z"][r.place].double() * r.gate.double()[..., None]).sum(1)
        mass = (t["z"][r.place].double() * r.gate.double()[..., None]).abs().sum(1)
        assert ((cpu(out).double() - want).abs() <= HALF[bf16] * want.abs() * 1.02 + 4 * U * mass).all()


class Rounded(torch.autograd.Function):
    """To BF16 on the way, and the gradient too where asked."""

    @staticmethod
    def forward(ctx, x, both):
        ctx.both = both
        return x.to(bf16).double()

    @staticmethod
    def backward(ctx, g):
        return (g.to(bf16).double() if ctx.both else g), None


def test_training_step(gpu_ok):
    import expert_layer as ex
    g = torch.Generator(device="cuda").manual_seed(3)
    tokens = 150
    x, res, gy, gr = torch.randn(4, tokens, ex.WIDTH, generator=g, device="cuda").to(bf16)
    weight = (1 + 0.1 * torch.randn(ex.WIDTH, generator=g, device="cuda")).to(bf16)
    up = (torch.randn(ex.EXPERTS, ex.WIDTH, ex.INNER, generator=g, device="cuda") * ex.WIDTH ** -0.5).to(bf16)
    down = (torch.randn(ex.EXPERTS, ex.INNER, ex.WIDTH, generator=g, device="cuda") * ex.INNER ** -0.5).to(bf16)
    routed = ex.route(torch.randn(tokens, ex.EXPERTS, generator=g, device="cuda"))
    y, grads = ex.train_step(x, res, weight, up, down, routed, gy, gr)

    r = cpu(routed)
    h = norm_sum(x.cpu(), res.cpu()).double().requires_grad_()
    w, u, d = (t.cpu().double().requires_grad_() for t in (weight, up, down))
    rstd = norm_rstd(h.detach().to(bf16), 1e-6).double()[:, None]
    normed = h * (h.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
    # (the forward value with the rounded rstd; the gradient is the formula's)
    normed = normed + (h * rstd - normed).detach()
    n = Rounded.apply(normed * w, True)
    off = r.offsets.tolist()
    parts = []
    for e in range(ex.EXPERTS):
        rows = n[r.token[off[e]:off[e + 1]]]
        a = Rounded.apply(torch.nn.functional.silu(Rounded.apply(rows @ u[e], True)), False)
        parts.append(Rounded.apply(a @ d[e], True))
    z = torch.cat(parts)
    out = (z[r.place] * r.gate.double()[..., None]).sum(1)
    ((out * gy.cpu().double()).sum() + (h * gr.cpu().double()).sum()).backward()

    def close(got, want, steps):
        """Within `steps` BF16 roundings of the whole: the roundings of both sides are the same
        but where FP32 and FP64 fall on two sides of a border, a step of a few values each."""
        got, want = got.cpu().double(), want.detach()
        assert (got - want).norm() <= steps * 2.0 ** -8 * want.norm()
        assert ((got - want).abs() <= steps * 2.0 ** -5 * (want.abs() + want.square().mean().sqrt())).all()

    close(y, out, 1)
    close(grads.x, h.grad, 1)
    close(grads.weight, w.grad, 0.5)
    close(grads.up, u.grad, 0.5)
    close(grads.down, d.grad, 0.5)


def test_program(gpu_ok, capsys):
    import expert_layer as ex
    ex.main()
    assert "served 86 tokens; lengths [13, 48, 25]" in capsys.readouterr().out


def test_captured_layer(gpu_ok):
    """A whole step of single tokens in a graph, replayed over a growing cache."""
    import expert_layer as ex
    layer = ex.Layer()
    one, two = ex.Cache(2), ex.Cache(2)
    add = torch.ones(2, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    off = torch.tensor([0] + [2] * ex.EXPERTS, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(4)
    x, res = torch.randn(2, 2, ex.WIDTH, generator=g, device="cuda").to(bf16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        warm = ex.Cache(2)
        warm.grow(add)
        layer(x, res, warm, cu)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one.grow(add)
        n = mp_step(layer, one, x, res, cu, off)
    for _ in range(20):
        x.normal_(generator=g)
        graph.replay()
        torch.cuda.synchronize()
        two.grow(add)
        want = mp_step(layer, two, x, res, cu, off)
        for a, b in zip(n, want):
            assert torch.equal(a, b)
    assert one.lens.tolist() == [20, 20] and torch.equal(one.k, two.k) and torch.equal(one.v, two.v)


def mp_step(layer, cache, x, res, cu, off):
    """The layer up to its experts (the routing's sort stays out of the graph)."""
    import expert_layer as ex
    import mixed_precision_dense_tiled_amd as mp
    n1 = mp.rms_norm(x, layer.norm1, residual=res, quant="int8")
    qkv = mp.gemm_w8a8(n1.out, n1.scales, *layer.qkv).view(-1, ex.HEADS + 2 * ex.KV_HEADS, ex.DIM)
    q, k, v = qkv.split([ex.HEADS, ex.KV_HEADS, ex.KV_HEADS], dim=1)
    where = dict(table=cache.table, cu_q=cu, lens=cache.lens)
    mp.paged_kv_append_rope(q, k, v, cache.k, cache.v, inv_freq=layer.inv_freq, out=q, **where)
    att = mp.paged_attention(q, cache.k, cache.v, **where)
    y = mp.gemm_w8a8(*mp.quantize_i8_rows(att.view(-1, ex.HEADS * ex.DIM)), *layer.out)
    n2 = mp.rms_norm(y, layer.norm2, residual=n1.residual, quant="int8")
    return n2.residual, mp.gemm_grouped_w8a8(n2.out, n2.scales, *layer.up, off)
