"""Definitions of a decoder layer's operators, apart from the package: in 64 bits,
and for outputs of 8 bits step by step as the header defines them."""
import torch

# half a step of each type, relative to the value
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# half a step among the subnormals
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
U = 2.0 ** -24


def norm_sum(x, residual):
    """What is normed: the sum rounded once to the rows' type."""
    return x if residual is None else (x.float() + residual.float()).to(x.dtype)


def norm_rstd(h, eps):
    return (1 / torch.sqrt(h.double().square().sum(-1) / h.shape[1] + eps)).float()


def norm_rows(h, weight, eps):
    """y in FP32, product by product."""
    return (h.float() * norm_rstd(h, eps)[:, None]) * weight.float()


def quantise(y, quant):
    """(codes as the values they stand for, scales) of y in FP32."""
    qmax = 127.0 if quant == "int8" else 448.0
    rows, dim = y.shape
    block = 128 if quant == "fp8_blocks" else dim
    scales = []
    values = torch.empty_like(y)
    for c in range(0, dim, block):
        part = y[:, c:c + block]
        amax = part.abs().amax(-1)
        amax = torch.where(part.isnan().any(-1), torch.full_like(amax, float("nan")), amax)
        s = amax / torch.tensor(qmax)
        s = torch.where(s == 0, torch.ones_like(s), s)
        v = (part / s[:, None]).clamp(-qmax, qmax)      # (NaN stays)
        if quant == "int8":
            v = torch.where(v.isnan(), torch.zeros_like(v), torch.round(v))
        else:
            v = v.to(torch.float8_e4m3fn).float()
        values[:, c:c + block] = v
        scales.append(s)
    return values, torch.stack(scales, 1) if quant == "fp8_blocks" else scales[0]


def norm_backward(grad, h, weight, rstd, grad_residual):
    """(grad_h, grad_weight) in FP64, with what their FP32 steps may be off by: the
    sums are at most `depth` additions deep."""
    g, x, w, r = grad.double(), h.double(), weight.double(), rstd.double()[:, None]
    dim = h.shape[1]
    gw = g * w
    c = (gw * x).sum(-1, keepdim=True) / dim
    dh = r * (gw - x * (r * r * c))
    depth = 8 * 4 + 6 + 16
    off = U * (4 * (r * gw).abs() + (depth + 8) * (r ** 3 * x).abs() * (gw * x).abs().sum(-1, keepdim=True) / dim)
    if grad_residual is not None:
        dh = dh + grad_residual.double()
        off = off + U * dh.abs()
    dw = (g * x * r).sum(0)
    rows = h.shape[0]
    off_w = U * (rows / 512 + 512 / 4 + 8) * (g * x * r).abs().sum(0)
    return dh, off, dw, off_w


def rope(x, pos, inv_freq, interleaved):
    """(turned rows, what their FP32 steps may be off by): x [tokens, heads, dim]."""
    pairs = inv_freq.shape[0]
    angle = pos.double()[:, None] * inv_freq.double()
    cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    x = x.double()
    y, off = x.clone(), torch.zeros_like(x)
    if interleaved:
        first, second = slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)
    else:
        first, second = slice(0, pairs), slice(pairs, 2 * pairs)
    a, b = x[..., first], x[..., second]
    y[..., first], y[..., second] = a * cos - b * sin, b * cos + a * sin
    # cos and sin to four roundings of 1 (and the angle's 53 bits), a product and a sum
    e = (a.abs() + b.abs()) * (6 * U + (angle.abs() * 2.0 ** -51)[:, None])
    off[..., first], off[..., second] = e, e
    return y, off


def groups_of(offsets, rows):
    """[(lo, hi)] of each group: an offset counts as the largest up to it, cut to the rows."""
    out, most = [], 0
    for a, b in zip(offsets, offsets[1:]):
        most = max(most, a)
        lo = min(most, rows)
        most = max(most, b)
        out.append((lo, min(most, rows)))
    return out
