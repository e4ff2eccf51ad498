"""The operators of libmpdt.so that a decoder layer has around its linear layers
and its cache (see include/mpdt_layers.h): the root-mean-square norm with the
residual's addition and an output in 8 bits, and its gradient; new keys rotated
on their way into a paged cache with the queries beside them; and products
grouped by expert, with their gradients and in W8A8.

As for the rest of the package, these functions marshal arguments, allocate
outputs and workspaces with torch, and run on torch's current stream (of the
tensors' device) without synchronising.  Numbers that live on the device (page
numbers, lengths, offsets) are not read here; the kernels cut them to the
buffers.  None of them takes part in torch's autograd: results are detached from
inputs that require a gradient, and gradients are calls of their own.
"""
from __future__ import annotations

import ctypes
from collections import namedtuple

import torch

from . import MpdtError, _check, _dims2, _same_device, _shape, _stream, lib
from .serving import _DTYPE, _cache_and_batch, _floats, _ints, _PagedKV, _rows3, _Sequences

__all__ = ["rms_norm", "rms_norm_backward", "RmsNorm", "paged_kv_append_rope", "gemm_grouped",
           "gemm_grouped_wgrad", "gemm_grouped_w8a8"]

_i64, _vp, _int, _f64 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_double

# what rms_norm writes: the C ABI's mpdt_norm_out
_NORM_OUT = {None: 0, "int8": 1, "fp8_rows": 2, "fp8_blocks": 3}

RmsNorm = namedtuple("RmsNorm", "out scales residual rstd")

# rows of a native rms_norm call
_NORM_ROWS = 4194303

_native = None


def _lib():
    """The native library with these entry points' signatures set."""
    global _native
    if _native is None:
        L = lib()
        kv, sq = ctypes.POINTER(_PagedKV), ctypes.POINTER(_Sequences)
        for name, res, args in (
                ("rms_norm", _int, [_int, _i64, _i64, _vp, _i64, _vp, _i64, _int, _vp, _f64, _int, _vp, _i64, _vp,
                                    _i64, _vp, _i64, _vp, _vp]),
                ("rms_norm_backward_workspace", _i64, [_i64, _i64]),
                ("rms_norm_backward", _int, [_int, _i64, _i64, _vp, _i64, _vp, _i64, _int, _vp, _vp, _vp, _i64, _vp,
                                             _i64, _vp, _vp, _i64, _vp]),
                ("paged_kv_append_rope", _int, [kv, sq, _int, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _int,
                                                _i64, _vp, _i64, _i64, _vp, _i64, _i64, _vp]),
                ("gemm_grouped", _int, [_int, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _int, _vp, _vp,
                                        _i64, _int, _vp]),
                ("gemm_grouped_wgrad", _int, [_int, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _i64,
                                              _i64, _int, _vp]),
                ("gemm_grouped_w8a8", _int, [_i64, _i64, _i64, _i64, _vp, _i64, _vp, _vp, _i64, _i64, _vp, _i64,
                                             _vp, _i64, _vp, _vp, _i64, _vp])):
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _native = L
    return _native


def _mat(t, dtype, name):
    """(pointer, leading dimension) of a row-major matrix of exactly this type."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    rows, cols = t.shape
    s0, s1 = t.stride()
    if cols > 1 and s1 != 1:
        raise ValueError(f"{name} must have unit stride along its rows")
    # (a stride over one row says nothing)
    return t.data_ptr(), s0 if rows > 1 else max(cols, 1)


def _stack(t, dtype, name):
    """(pointer, leading dimension, stride between matrices) of [groups, rows, cols]."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be 3-D")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    groups, rows, cols = t.shape
    s0, s1, s2 = t.stride()
    if cols > 1 and s2 != 1:
        raise ValueError(f"{name} must have unit stride along its rows")
    return t.data_ptr(), s1 if rows > 1 else max(cols, 1), s0 if groups > 1 else 0


def _on(ref, name, *ts):
    """All on ref's GPU."""
    _same_device(ref, *ts)
    if not ref.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")


def _call(ref, fn, *args):
    """The native call on ref's device and torch's current stream there."""
    native = getattr(_native or _lib(), fn)
    if ref.get_device() == torch.cuda.current_device():
        status = native(*args, _stream(ref))
    else:
        with torch.cuda.device(ref.device):
            status = native(*args, _stream(ref))
    if status:
        _check(fn, status)


def _norm_operands(x, weight, name):
    rows, dim = _dims2(x, name)
    code = _DTYPE.get(x.dtype)
    if code is None or code == 3:
        raise TypeError(f"{name} must be bfloat16, float16 or float32, got {x.dtype}")
    if weight.dtype not in (x.dtype, torch.float32):
        raise TypeError(f"weight must be {x.dtype} or torch.float32, got {weight.dtype}")
    _shape(weight, (dim,), "weight")
    if not weight.is_contiguous():
        raise ValueError("weight must be contiguous")
    return rows, dim, code, _DTYPE[weight.dtype]


def _apart(*written, rows, read):
    """Raise ValueError where a written operand (pointer, leading dimension, element's
    size, columns) overlaps another, other than exactly."""
    def span(m):
        return m[0], m[0] + ((rows - 1) * m[1] + m[3]) * m[2]

    written = [m for m in written if m[0] is not None]
    for i, a in enumerate(written):
        for b in written[i + 1:] + [m for m in read if m[0] is not None]:
            (lo, hi), (other, end) = span(a), span(b)
            if lo < end and other < hi and a != b:
                raise ValueError("an output overlaps another operand")


def rms_norm(x, weight, eps=1e-6, residual=None, quant=None, return_rstd=False, out=None, scales_out=None,
             residual_out=None):
    """Root-mean-square norm of rows, with the residual's addition before it and
    an output in 8 bits after it.

    x [rows, dim] BF16, FP16 or FP32 (rows may be strided), dim at most 32768;
    weight [dim] in x's type or FP32; residual like x.  (Over 4194303 rows take
    as many launches as they need.)  With h = x + residual, rounded once to x's
    type (x alone without a residual), rstd = 1 / sqrt(mean(h^2) + eps) and y =
    (h * rstd) * weight in FP32.  Returns RmsNorm:
      out       y in x's type, or with quant codes of 8 bits: "int8" for
                gemm_w8a8, "fp8_rows" (E4M3 in uint8) for gemm_fp8_rowscaled,
                "fp8_blocks" (E4M3, 1 x 128 scales) for gemm_fp8_blockscaled
      scales    FP32 [rows], with "fp8_blocks" [rows, ceil(dim / 128)]: the
                largest |y| of the row or block over 127 or 448 (1 where that
                is 0, NaN where the row or block holds one); None without quant
      residual  h with a residual, else None
      rstd      FP32 [rows] with return_rstd, else None.
    residual_out may be x or residual itself, and out too without quant.  There is
    no autograd here: rms_norm_backward gives the gradient."""
    rows, dim, code, w_code = _norm_operands(x, weight, "x")
    if quant not in _NORM_OUT:
        raise ValueError(f"quant must be one of None, 'int8', 'fp8_rows', 'fp8_blocks', got {quant!r}")
    if residual is None and residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if dim == 0:
        raise ValueError("x must have at least one column")
    dtype = x.dtype
    out_type = dtype if quant is None else torch.int8 if quant == "int8" else torch.uint8
    if quant is None and scales_out is not None:
        raise ValueError("scales_out belongs to an output of 8 bits")
    _shape(residual, (rows, dim), "residual")
    _shape(out, (rows, dim), "out")
    _shape(residual_out, (rows, dim), "residual_out")
    blocks = quant == "fp8_blocks"
    grid = (rows, -(-dim // 128)) if blocks else (rows,)
    _shape(scales_out, grid, "scales_out")
    _on(x, "x", ("weight", weight), ("residual", residual), ("out", out), ("scales_out", scales_out),
        ("residual_out", residual_out))
    px, ldx = _mat(x, dtype, "x")
    pr = ph = ps = pd = None
    ldr = ldh = ldo = lds = dim
    # (what is made here is as the call wants it)
    if residual is not None:
        pr, ldr = _mat(residual, dtype, "residual")
        if residual_out is None:
            residual_out = x.new_empty((rows, dim))
            ph = residual_out.data_ptr()
        else:
            ph, ldh = _mat(residual_out, dtype, "residual_out")
    if out is None:
        out = x.new_empty((rows, dim), dtype=out_type)
        po = out.data_ptr()
    else:
        po, ldo = _mat(out, out_type, "out")
    if quant is not None:
        lds = grid[-1] if blocks else 1
        if scales_out is None:
            scales_out = x.new_empty(grid, dtype=torch.float32)
            ps = scales_out.data_ptr()
        elif blocks:
            ps, lds = _mat(scales_out, torch.float32, "scales_out")
        else:
            ps = _floats(scales_out, rows, "scales_out")
    rstd = x.new_empty(rows, dtype=torch.float32) if return_rstd else None
    if rstd is not None:
        pd = rstd.data_ptr()
    if rows <= _NORM_ROWS:
        _call(x, "rms_norm", code, rows, dim, px, ldx, pr, ldr, w_code, weight.data_ptr(), eps, _NORM_OUT[quant], po,
              ldo, ps, lds, ph, ldh, pd)
    else:
        es, os = dtype.itemsize, out_type.itemsize
        # (each part's operands are checked against each other, so here all parts' at once)
        _apart((po, ldo, os, dim), (ph, ldh, es, dim), (ps, lds, 4, grid[-1] if blocks else 1), (pd, 1, 4, 1),
               rows=rows, read=((px, ldx, es, dim), (pr, ldr, es, dim), (weight.data_ptr(), 0, 1, dim * weight.itemsize)))
        at = lambda p, ld, size, lo: None if p is None else p + lo * ld * size
        for lo in range(0, rows, _NORM_ROWS):
            _call(x, "rms_norm", code, min(_NORM_ROWS, rows - lo), dim, at(px, ldx, es, lo), ldx, at(pr, ldr, es, lo),
                  ldr, w_code, weight.data_ptr(), eps, _NORM_OUT[quant], at(po, ldo, os, lo), ldo, at(ps, lds, 4, lo),
                  lds, at(ph, ldh, es, lo), ldh, at(pd, 1, 4, lo))
    return RmsNorm(out, scales_out, residual_out, rstd)


def rms_norm_backward(grad, h, weight, rstd, grad_residual=None, out=None):
    """Gradient of rms_norm (without quant) in its normed rows and its weight.

    grad [rows, dim]: the gradient in rms_norm's out; h: what was normed (its
    residual field, or x without a residual); rstd FP32 [rows] as it gave it;
    grad_residual, the gradient in the residual field, is added where given.
    Returns (grad_h in h's type, which is the gradient in x and in residual
    alike, and grad_weight FP32 [dim]).  out may be grad or grad_residual."""
    rows, dim, code, w_code = _norm_operands(h, weight, "h")
    for t, name in ((grad, "grad"), (grad_residual, "grad_residual"), (out, "out")):
        _shape(t, (rows, dim), name)
    _on(h, "h", ("grad", grad), ("weight", weight), ("rstd", rstd), ("grad_residual", grad_residual),
                ("out", out))
    if dim == 0:
        raise ValueError("h must have at least one column")
    pg, ldg = _mat(grad, h.dtype, "grad")
    ph, ldh = _mat(h, h.dtype, "h")
    pr, ldr = (None, dim) if grad_residual is None else _mat(grad_residual, h.dtype, "grad_residual")
    pd = _floats(rstd, rows, "rstd")
    if out is None:
        out = h.new_empty((rows, dim))
    po, ldo = _mat(out, h.dtype, "out")
    grad_weight = h.new_empty(dim, dtype=torch.float32)
    L = _lib()
    size = L.rms_norm_backward_workspace(rows, dim)
    if size < 0:
        raise MpdtError("rms_norm_backward", 1, L.mpdt_last_error().decode())
    ws = h.new_empty(size, dtype=torch.uint8) if size else None
    _call(h, "rms_norm_backward", code, rows, dim, pg, ldg, ph, ldh, w_code, weight.data_ptr(), pd, pr, ldr, po, ldo,
          grad_weight.data_ptr(), None if ws is None else ws.data_ptr(), size)
    return out, grad_weight


def paged_kv_append_rope(q, k, v, k_cache, v_cache, table, cu_q, lens, inv_freq, interleaved=False, k_scale=None,
                         v_scale=None, out=None):
    """paged_kv_append with the keys rotated by their positions on the way, and
    the queries beside them.

    k, v, the cache, table, cu_q and lens as in paged_kv_append; inv_freq FP32
    [pairs], 2 * pairs <= dim: pair i of a row at position p is turned by p *
    inv_freq[i] (formed in FP64, so far positions keep their angle).  Pair i is
    the elements (i, i + pairs), or with interleaved (2 i, 2 i + 1); elements
    from 2 * pairs on stay.  The position of new token t of a sequence with n
    tokens, nq of them new, is n - nq + t.  q [tokens, heads, dim] in k's type, or
    None.  Returns the turned q (in out, which may be q itself; None without q):
    rows that belong to no sequence are not written."""
    if k.dim() != 3:
        raise ValueError("k must be [tokens, kv_heads, dim]")
    tokens = k.shape[0]
    kv, sq = _cache_and_batch(k_cache, v_cache, table, cu_q, lens, tokens, k_scale, v_scale)
    dtype = k.dtype
    if dtype not in (torch.bfloat16, torch.float16) or (kv.dtype != 3 and dtype != k_cache.dtype):
        raise TypeError(f"new keys of {dtype} do not go into a cache of {k_cache.dtype}")
    shape = (tokens, kv.kv_heads, kv.dim)
    pk, kt, kh = _rows3(k, shape, dtype, "k")
    pv, vt, vh = _rows3(v, shape, dtype, "v")
    if inv_freq.dim() != 1 or not 1 <= inv_freq.shape[0] <= kv.dim // 2:
        raise ValueError(f"inv_freq must be 1-D with 1 to {kv.dim // 2} values")
    pf = _floats(inv_freq, inv_freq.shape[0], "inv_freq")
    heads, pq, qt, qh, po, ot, oh = 0, None, 0, 0, None, 0, 0
    if q is None:
        if out is not None:
            raise ValueError("out belongs to q")
    else:
        if q.dim() != 3 or q.shape[1] == 0:
            raise ValueError("q must be [tokens, heads, dim] with at least one head")
        heads = q.shape[1]
        pq, qt, qh = _rows3(q, (tokens, heads, kv.dim), dtype, "q")
    _on(k, "k", ("q", q), ("v", v), ("k_cache", k_cache), ("v_cache", v_cache), ("table", table),
                ("cu_q", cu_q), ("lens", lens), ("inv_freq", inv_freq), ("k_scale", k_scale), ("v_scale", v_scale),
                ("out", out))
    if q is not None:
        if out is None:
            out = q.new_empty((tokens, heads, kv.dim))
            po, ot, oh = out.data_ptr(), heads * kv.dim, kv.dim
        else:
            po, ot, oh = _rows3(out, (tokens, heads, kv.dim), dtype, "out")
    if tokens == 0:
        return out      # (an empty tensor has no address)
    _call(k, "paged_kv_append_rope", kv, sq, _DTYPE[dtype], pk, kt, kh, pv, vt, vh, pf, inv_freq.shape[0],
          int(bool(interleaved)), heads, pq, qt, qh, po, ot, oh)
    return out


def _offsets(offsets):
    """(pointer, groups) of the groups' borders."""
    if offsets.dim() != 1 or offsets.shape[0] < 1:
        raise ValueError("offsets must be 1-D with groups + 1 values")
    groups = offsets.shape[0] - 1
    return _ints(offsets, (groups + 1,), "offsets"), groups


def _half(t, name):
    if t.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"{name} must be bfloat16 or float16, got {t.dtype}")
    return _DTYPE[t.dtype]


def _out_type(out, dtype, d16):
    """An output's type: the given buffer's, or by d16."""
    kind = out.dtype if out is not None else dtype if d16 else torch.float32
    if kind not in (dtype, torch.float32):
        raise TypeError(f"out must be {dtype} or torch.float32, got {kind}")
    return kind


def gemm_grouped(A, B, offsets, trans_b=False, out=None, d16=False):
    """Products grouped by expert: D[i] = A[i] . B[e] for the rows i of group e.

    A [rows, K] BF16 or FP16, sorted by group: group e has the rows offsets[e] to
    offsets[e + 1] (INT32 [groups + 1], ascending; empty groups are fine).  B
    [groups, K, N] in A's type, or with trans_b [groups, N, K]; the matrices may
    be strided.  Returns D [rows, N]: FP32, or A's type with d16 (or an out of
    that type); sums are FP32 and rounded once.  Rows that belong to no group are
    not written.

    The gradient in A from the one in D, G, is gemm_grouped(G, B, offsets,
    trans_b=not trans_b); the one in B is gemm_grouped_wgrad's."""
    rows, K = _dims2(A, "A")
    code = _half(A, "A")
    poff, groups = _offsets(offsets)
    pb, ldb, sb = _stack(B, A.dtype, "B")
    N = B.shape[1 if trans_b else 2]
    _shape(B, (groups, N, K) if trans_b else (groups, K, N), "B")
    _shape(out, (rows, N), "out")
    kind = _out_type(out, A.dtype, d16)
    pa, lda = _mat(A, A.dtype, "A")
    _on(A, "A", ("B", B), ("offsets", offsets), ("out", out))
    if out is None:
        out = A.new_empty((rows, N), dtype=kind)
        pd, ldd = out.data_ptr(), max(N, 1)
    else:
        pd, ldd = _mat(out, kind, "out")
    _call(A, "gemm_grouped", code, groups, rows, N, K, pa, lda, pb, ldb, sb, int(bool(trans_b)), poff, pd, ldd,
          int(kind != torch.float32))
    return out


def gemm_grouped_wgrad(A, G, offsets, out=None, d16=False):
    """The gradient of gemm_grouped in its matrices: D[e] = A_e^T . G_e over the
    rows of group e.

    A [rows, K], G [rows, N], the gradient in gemm_grouped's D; offsets as there.
    Returns D [groups, K, N], FP32 or A's type with d16 (or an out of that type);
    0 for a group without rows.  For matrices kept as [groups, N, K] (trans_b)
    the gradient is gemm_grouped_wgrad(G, A, offsets)."""
    rows, K = _dims2(A, "A")
    code = _half(A, "A")
    rows_g, N = _dims2(G, "G")
    if rows_g != rows:
        raise ValueError("A and G must have the same rows")
    poff, groups = _offsets(offsets)
    _shape(out, (groups, K, N), "out")
    kind = _out_type(out, A.dtype, d16)
    pa, lda = _mat(A, A.dtype, "A")
    pg, ldg = _mat(G, A.dtype, "G")
    _on(A, "A", ("G", G), ("offsets", offsets), ("out", out))
    if out is None:
        out = A.new_empty((groups, K, N), dtype=kind)
    pd, ldd, sd = _stack(out, kind, "out")
    _call(A, "gemm_grouped_wgrad", code, groups, rows, N, K, pa, lda, pg, ldg, poff, pd, ldd, sd,
          int(kind != torch.float32))
    return out


def gemm_grouped_w8a8(X, x_scale, W, w_scale, offsets, bias=None, out=None):
    """The W8A8 layer of gemm_w8a8 by groups of rows.

    X INT8 [rows, K] with x_scale FP32 [rows] (as rms_norm or quantize_i8_rows
    give them), sorted by group as in gemm_grouped; W INT8 [groups, N, K] (one
    output channel per row) with w_scale FP32 [groups, N]; bias FP32 [groups, N] or
    None.  Returns Y BF16 [rows, N], each value bit for bit gemm_w8a8's."""
    rows, K = _dims2(X, "X")
    poff, groups = _offsets(offsets)
    pw, ldw, sw = _stack(W, torch.int8, "W")
    N = W.shape[1]
    _shape(W, (groups, N, K), "W")
    _shape(w_scale, (groups, N), "w_scale")
    _shape(bias, (groups, N), "bias")
    _shape(out, (rows, N), "out")
    px, ldx = _mat(X, torch.int8, "X")
    psx = _floats(x_scale, rows, "x_scale")
    psw, ldsw = _mat(w_scale, torch.float32, "w_scale")
    pb, ldb = (None, N) if bias is None else _mat(bias, torch.float32, "bias")
    _on(X, "X", ("x_scale", x_scale), ("W", W), ("w_scale", w_scale), ("offsets", offsets), ("bias", bias),
                ("out", out))
    if out is None:
        out = X.new_empty((rows, N), dtype=torch.bfloat16)
        py, ldy = out.data_ptr(), max(N, 1)
    else:
        py, ldy = _mat(out, torch.bfloat16, "out")
    _call(X, "gemm_grouped_w8a8", groups, rows, N, K, px, ldx, psx, pw, ldw, sw, psw, ldsw, pb, ldb, poff, py, ldy)
    return out
