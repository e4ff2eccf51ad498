"""A decoder layer's operators without a GPU: the Python binding refuses wrong
shapes, types and strides before anything native is called, and the C ABI
refuses wrong arguments on the host (or reports that there is no device)."""
import math
import os
import re

import pytest
import torch

import mixed_precision_dense_tiled_amd as mp
from layers_ref import norm_backward, norm_rstd, rope
from mixed_precision_dense_tiled_amd import layers
from test_serving_binding import ALIASING, INVALID, MISALIGNED, NO_DEVICE, SUCCESS, batch, gpu_present

bf16, f16, f32, i32, i8 = torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.int8
P, FAR = 1 << 40, 1 << 36          # addresses that nothing reads, and bytes between them
GROUPS = (2 ** 32 - 1) // 256      # workgroups of 256 threads to a launch
OK = (NO_DEVICE,)                   # all that stops a right call without a GPU


def lib():
    return layers._lib()


def run(call, change, status):
    if status is OK and gpu_present:
        pytest.skip("a right call; its addresses are none")
    s = call(**change)
    assert s in status, (s, lib().mpdt_last_error())


def test_exports_what_the_header_declares():
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "mpdt_layers.h")
    text = re.sub(r"/\*.*?\*/", "", open(header).read(), flags=re.S)
    names = set(re.findall(r"\b([a-z_][a-z0-9_]*)\s*\(", text)) - {"defined"}
    assert len(names) == 7
    for n in names:
        assert hasattr(lib(), n), n
    for n in layers.__all__:
        assert n in mp.__all__ and hasattr(mp, n)


# ---- the binding ------------------------------------------------------------------

def norm(**change):
    a = dict(x=torch.zeros(5, 64, dtype=bf16), weight=torch.zeros(64, dtype=bf16))
    a.update(change)
    return mp.rms_norm(**a)


@pytest.mark.parametrize("change, error, match", [
    (dict(x=torch.zeros(64, dtype=bf16)), ValueError, "x must be 2-D"),
    (dict(x=torch.zeros(5, 64, dtype=torch.float64)), TypeError, "x must be"),
    (dict(x=torch.zeros(5, 64, dtype=torch.uint8)), TypeError, "x must be"),
    (dict(weight=torch.zeros(64, dtype=f16)), TypeError, "weight must be"),
    (dict(weight=torch.zeros(63, dtype=bf16)), ValueError, "weight must have shape"),
    (dict(weight=torch.zeros(128, dtype=bf16)[::2]), ValueError, "contiguous"),
    (dict(quant="fp4"), ValueError, "quant"),
    (dict(residual=torch.zeros(5, 63, dtype=bf16)), ValueError, "residual must have shape"),
    (dict(residual_out=torch.zeros(5, 64, dtype=bf16)), ValueError, "needs a residual"),
    (dict(scales_out=torch.zeros(5)), ValueError, "belongs to"),
    (dict(quant="int8", scales_out=torch.zeros(4)), ValueError, "scales_out must have shape"),
    (dict(quant="fp8_blocks", scales_out=torch.zeros(5)), ValueError, "scales_out must have shape"),
    (dict(out=torch.zeros(5, 65, dtype=bf16)), ValueError, "out must have shape"),
    (dict(), ValueError, "GPU"),
])
def test_norm_refusals(change, error, match):
    with pytest.raises(error, match=match):
        norm(**change)


def backward(**change):
    a = dict(grad=torch.zeros(5, 64, dtype=bf16), h=torch.zeros(5, 64, dtype=bf16),
             weight=torch.zeros(64, dtype=bf16), rstd=torch.zeros(5))
    a.update(change)
    return mp.rms_norm_backward(**a)


@pytest.mark.parametrize("change, error, match", [
    (dict(grad=torch.zeros(4, 64, dtype=bf16)), ValueError, "grad must have shape"),
    (dict(grad_residual=torch.zeros(5, 60, dtype=bf16)), ValueError, "grad_residual must have shape"),
    (dict(out=torch.zeros(5, 60, dtype=bf16)), ValueError, "out must have shape"),
    (dict(weight=torch.zeros(64, dtype=f16)), TypeError, "weight must be"),
    (dict(), ValueError, "GPU"),
])
def test_backward_refusals(change, error, match):
    with pytest.raises(error, match=match):
        backward(**change)


def rotate(**change):
    b = batch()
    a = dict(q=b["q"], k=torch.zeros(5, 2, 64, dtype=bf16), v=torch.zeros(5, 2, 64, dtype=bf16),
             inv_freq=torch.zeros(32), **{n: b[n] for n in ("k_cache", "v_cache", "table", "cu_q", "lens")})
    a.update(change)
    return mp.paged_kv_append_rope(**a)


@pytest.mark.parametrize("change, error, match", [
    (dict(k=torch.zeros(5, 128, dtype=bf16)), ValueError, "k must be"),
    (dict(k=torch.zeros(5, 2, 64, dtype=f16)), TypeError, "do not go into"),
    (dict(k=torch.zeros(5, 2, 48, dtype=bf16)), ValueError, "k must have shape"),
    (dict(v=torch.zeros(4, 2, 64, dtype=bf16)), ValueError, "v must have shape"),
    (dict(q=torch.zeros(4, 8, 64, dtype=bf16)), ValueError, "q must have shape"),
    (dict(q=torch.zeros(5, 8, 64, dtype=f16)), TypeError, "q must be"),
    (dict(q=torch.zeros(5, 0, 64, dtype=bf16)), ValueError, "at least one head"),
    (dict(q=None, out=torch.zeros(5, 8, 64, dtype=bf16)), ValueError, "belongs to q"),
    (dict(inv_freq=torch.zeros(33)), ValueError, "inv_freq"),
    (dict(inv_freq=torch.zeros(0)), ValueError, "inv_freq"),
    (dict(inv_freq=torch.zeros(32, dtype=torch.float64)), TypeError, "inv_freq"),
    (dict(inv_freq=torch.zeros(64)[::2]), ValueError, "contiguous"),
    (dict(k_scale=torch.ones(2)), ValueError, "belong to an FP8 cache"),
    (dict(), ValueError, "GPU"),
])
def test_rotation_refusals(change, error, match):
    with pytest.raises(error, match=match):
        rotate(**change)


OFF = torch.zeros(4, dtype=i32)


def grouped(**change):
    a = dict(A=torch.zeros(5, 16, dtype=bf16), B=torch.zeros(3, 16, 8, dtype=bf16), offsets=OFF)
    a.update(change)
    return mp.gemm_grouped(**a)


@pytest.mark.parametrize("change, error, match", [
    (dict(A=torch.zeros(5, 16)), TypeError, "A must be"),
    (dict(A=torch.zeros(5, 16, dtype=f16)), TypeError, "B must be"),
    (dict(A=torch.zeros(5, 32, dtype=bf16)[:, ::2]), ValueError, "unit stride"),
    (dict(B=torch.zeros(16, 8, dtype=bf16)), ValueError, "B must be 3-D"),
    (dict(B=torch.zeros(2, 16, 8, dtype=bf16)), ValueError, "B must have shape"),
    (dict(B=torch.zeros(3, 8, 16, dtype=bf16)), ValueError, "B must have shape"),
    (dict(B=torch.zeros(3, 16, 8, dtype=bf16), trans_b=True), ValueError, "B must have shape"),
    (dict(B=torch.zeros(3, 8, 16, dtype=bf16).mT), ValueError, "unit stride"),
    (dict(offsets=torch.zeros(4, dtype=torch.int64)), TypeError, "offsets"),
    (dict(offsets=torch.zeros(8, dtype=i32)[::2]), ValueError, "contiguous"),
    (dict(offsets=torch.zeros(0, dtype=i32)), ValueError, "offsets"),
    (dict(out=torch.zeros(5, 9)), ValueError, "out must have shape"),
    (dict(out=torch.zeros(5, 8, dtype=f16)), TypeError, "out must be"),
    (dict(), ValueError, "GPU"),
])
def test_grouped_refusals(change, error, match):
    with pytest.raises(error, match=match):
        grouped(**change)


def wgrad(**change):
    a = dict(A=torch.zeros(5, 16, dtype=bf16), G=torch.zeros(5, 8, dtype=bf16), offsets=OFF)
    a.update(change)
    return mp.gemm_grouped_wgrad(**a)


@pytest.mark.parametrize("change, error, match", [
    (dict(G=torch.zeros(4, 8, dtype=bf16)), ValueError, "same rows"),
    (dict(G=torch.zeros(5, 8, dtype=f16)), TypeError, "G must be"),
    (dict(out=torch.zeros(3, 8, 16)), ValueError, "out must have shape"),
    (dict(), ValueError, "GPU"),
])
def test_wgrad_refusals(change, error, match):
    with pytest.raises(error, match=match):
        wgrad(**change)


def w8a8(**change):
    a = dict(X=torch.zeros(5, 16, dtype=i8), x_scale=torch.ones(5), W=torch.zeros(3, 8, 16, dtype=i8),
             w_scale=torch.ones(3, 8), offsets=OFF)
    a.update(change)
    return mp.gemm_grouped_w8a8(**a)


@pytest.mark.parametrize("change, error, match", [
    (dict(X=torch.zeros(5, 16, dtype=torch.uint8)), TypeError, "X must be"),
    (dict(W=torch.zeros(3, 16, 8, dtype=i8)), ValueError, "W must have shape"),
    (dict(x_scale=torch.ones(4)), ValueError, "x_scale"),
    (dict(w_scale=torch.ones(8)), ValueError, "w_scale"),
    (dict(w_scale=torch.ones(3, 8, dtype=f16)), TypeError, "w_scale"),
    (dict(bias=torch.ones(8)), ValueError, "bias"),
    (dict(out=torch.zeros(5, 9, dtype=bf16)), ValueError, "out must have shape"),
    (dict(), ValueError, "GPU"),
])
def test_w8a8_refusals(change, error, match):
    with pytest.raises(error, match=match):
        w8a8(**change)


# ---- the C ABI ----------------------------------------------------------------------

def c_norm(dtype=0, rows=5, dim=64, x=P, ldx=64, res=P + FAR, ld_res=64, w_dtype=0, w=P + 2 * FAR, eps=1e-6, kind=0,
           out=P + 3 * FAR, ld_out=64, scales=P + 4 * FAR, ld_scales=1, h=P + 5 * FAR, ld_h=64, rstd=P + 6 * FAR):
    return lib().rms_norm(dtype, rows, dim, x, ldx, res, ld_res, w_dtype, w, eps, kind, out, ld_out, scales,
                          ld_scales, h, ld_h, rstd, None)


@pytest.mark.parametrize("change, status", [
    (dict(), OK), (dict(rows=0, x=None), (SUCCESS,)), (dict(dim=0), (INVALID,)),
    (dict(dim=32768, ldx=32768, ld_res=32768, ld_out=32768, ld_h=32768), OK),
    (dict(dim=32769, ldx=40000, ld_res=40000, ld_out=40000, ld_h=40000), (INVALID,)),
    (dict(rows=-1), (INVALID,)), (dict(rows=(2 ** 32 - 1) // 1024 + 1), (INVALID,)), (dict(dtype=3), (INVALID,)),
    (dict(w_dtype=1), (INVALID,)), (dict(w_dtype=2), OK), (dict(eps=-1.0), (INVALID,)),
    (dict(eps=math.inf), (INVALID,)), (dict(eps=math.nan), (INVALID,)), (dict(kind=4), (INVALID,)),
    (dict(kind=-1), (INVALID,)), (dict(x=None), (INVALID,)), (dict(out=None), (INVALID,)), (dict(w=None), (INVALID,)),
    (dict(kind=1, scales=None), (INVALID,)), (dict(kind=3, ld_scales=0), (INVALID,)), (dict(kind=3), OK),
    (dict(kind=3, dim=129, ldx=129, ld_res=129, ld_out=129, ld_h=129), (INVALID,)),
    (dict(ldx=63), (INVALID,)), (dict(ld_res=63), (INVALID,)), (dict(ld_out=63), (INVALID,)),
    (dict(ld_h=63), (INVALID,)), (dict(res=None), (INVALID,)), (dict(res=None, h=None), OK), (dict(h=None), OK),
    (dict(rstd=None), OK), (dict(x=P + 1), (MISALIGNED,)), (dict(x=P + 2), OK), (dict(w=P + 1), (MISALIGNED,)),
    (dict(kind=1, scales=P + 4 * FAR + 2), (MISALIGNED,)), (dict(rstd=P + 2), (MISALIGNED,)),
    (dict(kind=1, out=P + 3 * FAR + 1), OK), (dict(ldx=1 << 50), (INVALID,)),
    # in place
    (dict(out=P), OK), (dict(out=P + FAR), OK), (dict(h=P), OK), (dict(h=P + FAR), OK), (dict(h=P, out=P + FAR), OK),
    (dict(h=P, out=P), (ALIASING,)), (dict(out=P + 2), (ALIASING,)), (dict(out=P, ld_out=65), (ALIASING,)),
    (dict(kind=1, out=P), (ALIASING,)), (dict(h=P + 2), (ALIASING,)), (dict(h=P + FAR, ld_h=70), (ALIASING,)),
    (dict(out=P + 2 * FAR), (ALIASING,)), (dict(rstd=P), (ALIASING,)), (dict(rstd=P + 3 * FAR), (ALIASING,)),
    (dict(kind=1, scales=P + 2 * FAR), (ALIASING,)), (dict(kind=1, scales=P + 6 * FAR), (ALIASING,)),
    (dict(res=P, h=P), OK), (dict(res=P + 2, h=P), (ALIASING,)),
])
def test_norm_abi(change, status):
    run(c_norm, change, status)


def c_back(dtype=0, rows=5, dim=64, g=P, ldg=64, h=P + FAR, ldh=64, w_dtype=0, w=P + 2 * FAR, rstd=P + 3 * FAR,
           r=P + 4 * FAR, ldr=64, o=P + 5 * FAR, ldo=64, gw=P + 6 * FAR, ws=P + 7 * FAR, size=None):
    if size is None:
        size = lib().rms_norm_backward_workspace(rows, dim)
    return lib().rms_norm_backward(dtype, rows, dim, g, ldg, h, ldh, w_dtype, w, rstd, r, ldr, o, ldo, gw, ws, size,
                                   None)


@pytest.mark.parametrize("change, status", [
    (dict(), OK), (dict(rows=0, g=None, h=None), OK), (dict(size=0), (INVALID,)), (dict(ws=None), (INVALID,)),
    (dict(rows=1, ws=None), OK), (dict(gw=None), (INVALID,)), (dict(rstd=None), (INVALID,)), (dict(r=None), OK),
    (dict(o=P), OK), (dict(o=P + 4 * FAR), OK), (dict(o=P + FAR), (ALIASING,)), (dict(o=P + 2), (ALIASING,)),
    (dict(gw=P), (ALIASING,)), (dict(gw=P + 7 * FAR), (ALIASING,)), (dict(ws=P + FAR), (ALIASING,)),
    (dict(gw=P + 5 * FAR), (ALIASING,)), (dict(ws=P + 7 * FAR + 2), (MISALIGNED,)), (dict(ldo=63), (INVALID,)),
    (dict(r=P + 2, o=P), (ALIASING,)), (dict(r=P, o=P), OK), (dict(w_dtype=1), (INVALID,)),
])
def test_backward_abi(change, status):
    run(c_back, change, status)


def test_backward_workspace():
    size = lib().rms_norm_backward_workspace
    assert size(0, 64) == 0 and size(1, 64) == 0 and size(1000, 4096) >= 2 * 4096 * 4
    assert size(-1, 64) == -1 and size(5, 0) == -1 and size(5, 32769) == -1
    assert size(1 << 20, 32768) == size(1 << 21, 32768) > 0


def c_rope(q=P + 6 * FAR, out=P + 7 * FAR, heads=4, pairs=32, interleaved=0, f=P + 8 * FAR, dtype=0, k=P + 4 * FAR,
           v=P + 5 * FAR, k_token=128, q_token=256, o_token=256, q_head=64, o_head=64, cache=None, seq=None):
    kv = layers._PagedKV(P, P + FAR, 2048, 128, 64, 9, 16, 2, 64, 0, None, None)
    for n, x in (cache or {}).items():
        setattr(kv, n, x)
    sq = layers._Sequences(P + 2 * FAR, 3, P + 3 * FAR, P + 3 * FAR + 4096, 2, 3, 5)
    for n, x in (seq or {}).items():
        setattr(sq, n, x)
    return lib().paged_kv_append_rope(kv, sq, dtype, k, k_token, 64, v, 128, 64, f, pairs, interleaved, heads, q,
                                      q_token, q_head, out, o_token, o_head, None)


@pytest.mark.parametrize("change, status", [
    (dict(), OK), (dict(pairs=0), (INVALID,)), (dict(pairs=33), (INVALID,)), (dict(pairs=1), OK),
    (dict(interleaved=2), (INVALID,)), (dict(f=None), (INVALID,)), (dict(f=P + 8 * FAR + 2), (MISALIGNED,)),
    (dict(heads=0), (INVALID,)), (dict(heads=0, q=None, out=None), OK), (dict(q=None), (INVALID,)),
    (dict(out=None), (INVALID,)), (dict(heads=70000), (INVALID,)), (dict(dtype=1), (INVALID,)),
    (dict(q=P + 6 * FAR + 2), (MISALIGNED,)), (dict(out=P + 7 * FAR + 8), (MISALIGNED,)),
    (dict(k=P + 4 * FAR + 2), (MISALIGNED,)), (dict(k_token=132), (MISALIGNED,)), (dict(k=None), (INVALID,)),
    (dict(seq=dict(tokens=0), k=None), (SUCCESS,)), (dict(seq=dict(seqs=0), k=None), (SUCCESS,)),
    (dict(seq=dict(tokens=GROUPS + 1)), (INVALID,)),
    (dict(out=P + 6 * FAR), OK), (dict(out=P + 6 * FAR + 16), (ALIASING,)), (dict(out=P + 6 * FAR, o_token=512), (ALIASING,)),
    (dict(out=P), (ALIASING,)), (dict(q=P), (ALIASING,)), (dict(k=P), (ALIASING,)), (dict(v=P + FAR + 512), (ALIASING,)),
    (dict(out=P + 4 * FAR), (ALIASING,)), (dict(out=P + 8 * FAR), (ALIASING,)), (dict(out=P + 2 * FAR), (ALIASING,)),
    (dict(out=P + 3 * FAR), (ALIASING,)), (dict(o_token=128), (ALIASING,)), (dict(o_head=32), (ALIASING,)),
    (dict(cache=dict(slot_stride=64)), (ALIASING,)), (dict(cache=dict(dim=63)), (INVALID,)),
    # q, k side by side in one wide row
    (dict(q=P + 4 * FAR + 256, out=P + 4 * FAR + 256, k_token=512, q_token=512, o_token=512), OK),
    (dict(q=P + 4 * FAR + 128, out=P + 4 * FAR + 128, k_token=512, q_token=512, o_token=512), (ALIASING,)),
    (dict(q=P + 4 * FAR + 256, out=P + 4 * FAR + 256, k_token=384, q_token=384, o_token=384), OK),
    (dict(q=P + 4 * FAR + 256, out=P + 4 * FAR + 256, k_token=376, q_token=376, o_token=376), (ALIASING,)),
])
def test_rotation_abi(change, status):
    run(c_rope, change, status)


def c_grouped(dtype=0, groups=3, rows=5, N=8, K=16, a=P, lda=16, b=P + FAR, ldb=None, sb=128, trans=0, off=P + 2 * FAR,
              d=P + 3 * FAR, ldd=8, d16=0):
    return lib().gemm_grouped(dtype, groups, rows, N, K, a, lda, b, (K if trans else N) if ldb is None else ldb, sb,
                              trans, off, d, ldd, d16, None)


@pytest.mark.parametrize("change, status", [
    (dict(), OK), (dict(trans=1), OK), (dict(d16=1), OK), (dict(dtype=2), (INVALID,)), (dict(dtype=3), (INVALID,)),
    (dict(trans=2), (INVALID,)), (dict(d16=-1), (INVALID,)), (dict(groups=-1), (INVALID,)),
    (dict(groups=65536), (INVALID,)), (dict(groups=0), (SUCCESS,)), (dict(rows=0), (SUCCESS,)),
    (dict(N=0), (SUCCESS,)), (dict(K=0, a=None, b=None), OK), (dict(K=-1), (INVALID,)),
    (dict(a=None), (INVALID,)), (dict(b=None), (INVALID,)), (dict(d=None), (INVALID,)), (dict(off=None), (INVALID,)),
    (dict(lda=15), (INVALID,)), (dict(ldb=7), (INVALID,)), (dict(trans=1, ldb=15), (INVALID,)), (dict(ldd=7), (INVALID,)),
    (dict(sb=0), OK), (dict(sb=-8), (INVALID,)), (dict(sb=1 << 50), (INVALID,)), (dict(ldb=1 << 50), (INVALID,)),
    (dict(a=P + 1), (MISALIGNED,)), (dict(d=P + 3 * FAR + 2), (MISALIGNED,)), (dict(d=P + 3 * FAR + 2, d16=1), OK),
    (dict(off=P + 2), (MISALIGNED,)), (dict(d=P), (ALIASING,)), (dict(d=P + FAR + 512), (ALIASING,)),
    (dict(d=P + 2 * FAR), (ALIASING,)), (dict(rows=1 << 30, N=1 << 20, ldd=1 << 20, sb=0), (INVALID,)),
])
def test_grouped_abi(change, status):
    run(c_grouped, change, status)


def c_wgrad(dtype=0, groups=3, rows=5, N=8, K=16, a=P, lda=16, g=P + FAR, ldg=8, off=P + 2 * FAR, d=P + 3 * FAR, ldd=8,
            sd=128, d16=0):
    return lib().gemm_grouped_wgrad(dtype, groups, rows, N, K, a, lda, g, ldg, off, d, ldd, sd, d16, None)


@pytest.mark.parametrize("change, status", [
    (dict(), OK), (dict(rows=0, a=None, g=None), OK), (dict(groups=0), (SUCCESS,)), (dict(N=0), (SUCCESS,)),
    (dict(K=0), (SUCCESS,)), (dict(sd=127), (ALIASING,)), (dict(sd=0), (ALIASING,)), (dict(groups=1, sd=0), OK),
    (dict(ldd=24, sd=8), OK), (dict(ldd=16, sd=8), (ALIASING,)), (dict(d=P + FAR), (ALIASING,)),
    (dict(g=None), (INVALID,)), (dict(ldg=7), (INVALID,)), (dict(dtype=2), (INVALID,)), (dict(d=P + 3 * FAR + 2), (MISALIGNED,)),
    (dict(groups=60000, N=1 << 13, K=1 << 13, lda=1 << 13, ldg=1 << 13, ldd=1 << 13, sd=1 << 26), (INVALID,)),
])
def test_wgrad_abi(change, status):
    run(c_wgrad, change, status)


def c_w8a8(groups=3, rows=5, N=8, K=16, x=P, ldx=16, xs=P + FAR, w=P + 2 * FAR, ldw=16, sw=128, ws=P + 3 * FAR, ldws=8,
           b=P + 4 * FAR, ldb=8, off=P + 5 * FAR, y=P + 6 * FAR, ldy=8):
    return lib().gemm_grouped_w8a8(groups, rows, N, K, x, ldx, xs, w, ldw, sw, ws, ldws, b, ldb, off, y, ldy, None)


@pytest.mark.parametrize("change, status", [
    (dict(), OK), (dict(b=None), OK), (dict(x=P + 1, w=P + 2 * FAR + 3), OK), (dict(K=0, x=None, w=None), OK),
    (dict(rows=0), (SUCCESS,)), (dict(xs=None), (INVALID,)), (dict(ws=None), (INVALID,)), (dict(ldws=7), (INVALID,)),
    (dict(ldb=7), (INVALID,)), (dict(ldw=15), (INVALID,)), (dict(ldy=7), (INVALID,)), (dict(xs=P + FAR + 2), (MISALIGNED,)),
    (dict(y=P + 6 * FAR + 1), (MISALIGNED,)), (dict(y=P), (ALIASING,)), (dict(y=P + FAR), (ALIASING,)),
    (dict(y=P + 3 * FAR), (ALIASING,)), (dict(y=P + 4 * FAR), (ALIASING,)), (dict(y=P + 5 * FAR), (ALIASING,)),
])
def test_w8a8_abi(change, status):
    run(c_w8a8, change, status)


# ---- the definitions that the GPU tests hold the kernels against ----------------------

def test_norm_gradient_is_the_gradient():
    """norm_backward against differences in 64 bits."""
    g = torch.Generator().manual_seed(3)
    h, up, res = (torch.randn((4, 24), generator=g) for _ in range(3))
    w = torch.randn(24, generator=g)
    loss = lambda x, v: ((up.double() * x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * v).sum()
                         + (res.double() * x).sum())
    rstd = norm_rstd(h, 1e-6)
    dh, off, dw, off_w = norm_backward(up, h, w, rstd, res)
    step = 2.0 ** -10
    for i in range(0, 24, 5):
        e = torch.zeros(24, dtype=torch.float64)
        e[i] = step
        one = torch.zeros((4, 1), dtype=torch.float64)
        one[2] = 1
        a = (loss(h.double() + one * e, w.double()) - loss(h.double() - one * e, w.double())) / (2 * step)
        b = (loss(h.double(), w.double() + e) - loss(h.double(), w.double() - e)) / (2 * step)
        # (rstd is rounded to FP32, the difference bent by the third derivative)
        assert abs(a - dh[2, i]) < 1e-5 and abs(b - dw[i]) < 1e-5
    assert (off > 0).all() and (off < 1e-4).all() and (off_w < 1e-3).all()


def test_rotation_turns():
    """Lengths stay, angles add up, and both layouts turn the same pairs."""
    g = torch.Generator().manual_seed(4)
    x = torch.randn((6, 2, 16), generator=g).double()
    f = torch.rand(8, generator=g)
    p, q = torch.arange(6), torch.tensor([5, 0, 9, 100, 3, 2])
    y, _ = rope(x, p, f, False)
    assert torch.allclose(y.square().sum(-1), x.square().sum(-1))
    assert torch.allclose(rope(y, q, f, False)[0], rope(x, p + q, f, False)[0])
    mixed = torch.stack([x[..., :8], x[..., 8:]], -1).flatten(-2)
    z, _ = rope(mixed, p, f, True)
    assert torch.allclose(z.unflatten(-1, (8, 2)).transpose(-1, -2).flatten(-2), y)
