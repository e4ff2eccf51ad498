"""The serving operators of libmpdt.so (see include/mpdt_serving.h): a paged
key/value cache, attention of new tokens over it, the bookkeeping of its
pages, and log probabilities of given tokens with their gradient.

As for the rest of the package, these functions marshal arguments, allocate
outputs and workspaces with torch, and run on torch's current stream without
synchronising.  Numbers that live on the device (page numbers, lengths,
offsets) are not read here; the kernels cut them to the buffers.  None of them
takes part in torch's autograd: results are detached from logits, q or caches that
require a gradient, and token_logprobs_backward is a call of its own.
"""
from __future__ import annotations

import ctypes
from collections import namedtuple

import torch

from . import MpdtError, _check, _same_device, _shape, _stream, lib

__all__ = ["paged_kv_append", "paged_attention", "cache_fork", "cache_extend", "cache_free",
           "cache_compact", "token_logprobs", "token_logprobs_backward", "TokenLogprobs"]

_i64, _vp, _int, _f32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float

# the C ABI's mpdt_dtype
_DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, torch.float8_e4m3fn: 3, torch.uint8: 3}


class _PagedKV(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("page_stride", _i64), ("slot_stride", _i64), ("head_stride", _i64),
                ("pages", _i64), ("page_size", _i64), ("kv_heads", _i64), ("dim", _i64), ("dtype", _int),
                ("k_scale", _vp), ("v_scale", _vp)]


class _Sequences(ctypes.Structure):
    _fields_ = [("table", _vp), ("ld_table", _i64), ("cu_q", _vp), ("lens", _vp), ("seqs", _i64),
                ("width", _i64), ("tokens", _i64)]


class _Pages(ctypes.Structure):
    _fields_ = [("kv", _vp), ("plane_stride", _i64), ("page_stride", _i64), ("page_bytes", _i64),
                ("planes", _i64), ("pages", _i64), ("page_size", _i64), ("refs", _vp), ("table", _vp),
                ("ld_table", _i64), ("lens", _vp), ("rows", _i64), ("width", _i64)]


TokenLogprobs = namedtuple("TokenLogprobs", "logprob lse entropy top_logprobs top_indices")

_native = None


def _lib():
    """The native library with the serving entry points' signatures set."""
    global _native
    if _native is None:
        L = lib()
        kv, sq, pg = (ctypes.POINTER(t) for t in (_PagedKV, _Sequences, _Pages))
        for name, res, args in (
                ("paged_kv_append", _int, [kv, sq, _int, _vp, _i64, _i64, _vp, _i64, _i64, _vp]),
                ("paged_attention_workspace", _i64, [kv, sq, _i64]),
                ("paged_attention", _int, [kv, sq, _i64, _int, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64,
                                           _f32, _f32, _i64, _vp, _i64, _vp]),
                ("cache_pages_workspace", _i64, [_i64, _i64]),
                ("cache_fork", _int, [pg, _vp, _vp, _vp, _i64, _vp]),
                ("cache_extend", _int, [pg, _vp, _vp, _vp, _i64, _vp]),
                ("cache_free", _int, [pg, _vp, _vp]),
                ("cache_compact", _int, [pg, _vp, _i64, _vp]),
                ("token_logprobs_workspace", _i64, [_int, _i64, _i64, _i64]),
                ("token_logprobs", _int, [_int, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp,
                                          _i64, _vp]),
                ("token_logprobs_backward", _int, [_int, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp,
                                                   _i64, _vp])):
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _native = L
    return _native


def _ints(t, shape, name, dtype=torch.int32):
    """Pointer of a contiguous whole-number tensor of exactly this shape."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _floats(t, n, name):
    """Pointer of a contiguous FP32 vector of n values."""
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be torch.float32, got {t.dtype}")
    if tuple(t.shape) != (n,):
        raise ValueError(f"{name} must have shape {(n,)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows3(t, shape, dtype, name):
    """(pointer, token stride, head stride) of a [tokens, heads, dim] tensor."""
    if t.dim() != 3 or tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    s0, s1, s2 = t.stride()
    if s2 != 1:
        raise ValueError(f"{name} must have unit stride along dim")
    # (a stride over one element says nothing)
    return t.data_ptr(), s0 if shape[0] > 1 else 0, s1 if shape[1] > 1 else 0


def _table(table, name="table"):
    if table.dtype != torch.int32:
        raise TypeError(f"{name} must be torch.int32, got {table.dtype}")
    if table.dim() != 2 or table.shape[1] < 1:
        raise ValueError(f"{name} must be 2-D with at least one column")
    rows, width = table.shape
    s0, s1 = table.stride()
    if width > 1 and s1 != 1:
        raise ValueError(f"{name} must have unit stride along its rows")
    return rows, width, (s0 if rows > 1 else width)


def _on_gpu(ref, name, *ts):
    _same_device(ref, *ts)
    if not ref.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")


def _cache_and_batch(k_cache, v_cache, table, cu_q, lens, tokens, k_scale, v_scale):
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [pages, page_size, kv_heads, dim]")
    shape, strides, dtype = k_cache.shape, k_cache.stride(), k_cache.dtype
    if v_cache.shape != shape or v_cache.stride() != strides or v_cache.dtype != dtype:
        raise ValueError("k_cache and v_cache must have the same shape, strides and type")
    code = _DTYPE.get(dtype)
    if code is None or code == 2:
        raise TypeError(f"a cache must be bfloat16, float16, float8_e4m3fn or uint8, got {dtype}")
    if strides[3] != 1:
        raise ValueError("the cache must have unit stride along dim")
    pages, page, heads, dim = shape
    ks = vs = None
    if code == 3:
        if k_scale is None or v_scale is None:
            raise ValueError("an FP8 cache needs k_scale and v_scale")
        ks, vs = _floats(k_scale, heads, "k_scale"), _floats(v_scale, heads, "v_scale")
    elif k_scale is not None or v_scale is not None:
        raise ValueError("k_scale and v_scale belong to an FP8 cache")
    seqs, width, ld = _table(table)
    # (a stride over one element says nothing)
    kv = _PagedKV(k_cache.data_ptr(), v_cache.data_ptr(), strides[0] if pages > 1 else 0,
                  strides[1] if page > 1 else 0, strides[2] if heads > 1 else 0, pages, page, heads, dim, code,
                  ks, vs)
    sq = _Sequences(table.data_ptr(), ld, _ints(cu_q, (seqs + 1,), "cu_q"), _ints(lens, (seqs,), "lens"), seqs,
                    width, tokens)
    return kv, sq


def paged_kv_append(k, v, k_cache, v_cache, table, cu_q, lens, k_scale=None, v_scale=None):
    """Write the keys and values of new tokens into a paged cache, in place.

    k, v [tokens, kv_heads, dim] BF16 or FP16: the new tokens of all sequences
    one after the other; sequence b has rows cu_q[b] to cu_q[b + 1] (INT32
    [seqs + 1]), the last of its lens[b] tokens (INT32 [seqs], new ones
    included).  k_cache, v_cache [pages, page_size, kv_heads, dim] with any
    page, slot and head strides (the same for both): k's type, or E4M3 with a
    scale per head (k_scale, v_scale FP32 [kv_heads]), where x is stored as
    e4m3(clamp(x / scale, -448, 448)).  table INT32 [seqs, width]: the page of
    each page_size tokens; its rows may be strided.  dim is a multiple of 16
    up to 128.  Tokens without a place (no page in the table) are dropped."""
    if k.dim() != 3:
        raise ValueError("k must be [tokens, kv_heads, dim]")
    kv, sq = _cache_and_batch(k_cache, v_cache, table, cu_q, lens, k.shape[0], k_scale, v_scale)
    dtype = k.dtype
    if dtype not in (torch.bfloat16, torch.float16) or (kv.dtype != 3 and dtype != k_cache.dtype):
        raise TypeError(f"new keys of {dtype} do not go into a cache of {k_cache.dtype}")
    shape = (k.shape[0], kv.kv_heads, kv.dim)
    pk, kt, kh = _rows3(k, shape, dtype, "k")
    pv, vt, vh = _rows3(v, shape, dtype, "v")
    _on_gpu(k, "k", ("v", v), ("k_cache", k_cache), ("v_cache", v_cache), ("table", table), ("cu_q", cu_q),
            ("lens", lens), ("k_scale", k_scale), ("v_scale", v_scale))
    _check("paged_kv_append", _lib().paged_kv_append(kv, sq, _DTYPE[dtype], pk, kt, kh, pv, vt, vh, _stream(k)))


def paged_attention(q, k_cache, v_cache, table, cu_q, lens, scale=None, softcap=0.0, window=0, k_scale=None,
                    v_scale=None, out=None, lse=None, return_lse=False):
    """Causal attention of new tokens over a paged cache that holds their own
    keys and values already (paged_kv_append).

    q [tokens, heads, dim] BF16 or FP16, heads a multiple of the cache's
    kv_heads; the cache, table, cu_q and lens as in paged_kv_append.  The new
    token t of a sequence with n tokens, nq of them new, stands at position
    p = n - nq + t and sees the keys j <= p, with window > 0 only j > p -
    window.  Scores are scale * (q . k) (scale: dim ** -0.5 by default), with
    softcap > 0 softcap * tanh(score / softcap).  Returns out [tokens, heads,
    dim] in q's type, with return_lse (or an lse buffer) also the FP32
    [tokens, heads] log of the sum of exp(scores).  A token that sees no key
    gets 0 and -inf; rows of q that belong to no sequence are not written.  There
    is no gradient: the outputs are detached from q and the cache."""
    if q.dim() != 3:
        raise ValueError("q must be [tokens, heads, dim]")
    tokens, heads, dim = q.shape
    dtype = q.dtype
    kv, sq = _cache_and_batch(k_cache, v_cache, table, cu_q, lens, tokens, k_scale, v_scale)
    if dtype not in (torch.bfloat16, torch.float16) or (kv.dtype != 3 and dtype != k_cache.dtype):
        raise TypeError(f"q of {dtype} does not go with a cache of {k_cache.dtype}")
    if dim != kv.dim:
        raise ValueError(f"q must have the cache's dim {kv.dim}, got {dim}")
    if heads == 0 or heads % kv.kv_heads:
        raise ValueError(f"heads ({heads}) must be a multiple of kv_heads ({kv.kv_heads})")
    pq, qt, qh = _rows3(q, (tokens, heads, dim), dtype, "q")
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    po, ot, oh = _rows3(out, (tokens, heads, dim), dtype, "out")
    if lse is None and return_lse:
        lse = torch.empty((tokens, heads), dtype=torch.float32, device=q.device)
    pl, lt = None, heads
    if lse is not None:
        _shape(lse, (tokens, heads), "lse")
        if lse.dtype != torch.float32 or (heads > 1 and lse.stride(1) != 1):
            raise ValueError("lse must be FP32 with unit stride along heads")
        pl, lt = lse.data_ptr(), lse.stride(0) if tokens > 1 else heads
    _on_gpu(q, "q", ("k_cache", k_cache), ("v_cache", v_cache), ("table", table), ("cu_q", cu_q), ("lens", lens),
            ("k_scale", k_scale), ("v_scale", v_scale), ("out", out), ("lse", lse))
    L = _lib()
    size = L.paged_attention_workspace(kv, sq, heads)
    if size < 0:
        raise MpdtError("paged_attention", 1, L.mpdt_last_error().decode())
    ws = torch.empty(size, dtype=torch.uint8, device=q.device) if size else None
    _check("paged_attention",
           L.paged_attention(kv, sq, heads, _DTYPE[dtype], pq, qt, qh, po, ot, oh, pl, lt,
                             dim ** -0.5 if scale is None else scale, softcap, window,
                             None if ws is None else ws.data_ptr(), size, _stream(q)))
    return out if lse is None else (out, lse)


def _pages(kv, refs, table, lens, page_size):
    """The C ABI's view of a cache's pages; kv may be None."""
    if refs.dim() != 1:
        raise ValueError("refs must be 1-D")
    pages = refs.shape[0]
    rows, width, ld = _table(table)
    c = _Pages(None, 0, 0, 0, 0, pages, page_size, _ints(refs, (pages,), "refs"), table.data_ptr(), ld,
               _ints(lens, (rows,), "lens"), rows, width)
    if kv is not None:
        if kv.dim() < 3 or kv.shape[1] != pages or kv.shape[2] != page_size:
            raise ValueError(f"kv must be [planes, {pages}, {page_size}, ...], got {tuple(kv.shape)}")
        es, inner = kv.element_size(), 1
        for n, s in zip(reversed(kv.shape[2:]), reversed(kv.stride()[2:])):
            if n > 1 and s != inner:
                raise ValueError("a page of kv must be contiguous")
            inner *= n
        c.kv, c.planes, c.page_bytes = kv.data_ptr(), kv.shape[0], inner * es
        s0, s1 = kv.stride()[:2]
        # (a stride over one element says nothing)
        c.page_stride = s1 * es if pages > 1 else inner * es
        c.plane_stride = s0 * es if kv.shape[0] > 1 else 0
    return c


def _pages_call(name, kv, refs, table, lens, which, which_name, page_size, shortfall, workspace=True):
    c = _pages(kv, refs, table, lens, page_size)
    pw = None if which is None else _ints(which, (c.rows,), which_name)
    _on_gpu(refs, "refs", ("kv", kv), ("table", table), ("lens", lens), (which_name, which))
    L = _lib()
    args = [] if which is None else [pw]
    short = None
    if shortfall:
        short = torch.zeros(1, dtype=torch.int32, device=refs.device) if c.rows == 0 else \
            torch.empty(1, dtype=torch.int32, device=refs.device)
        args.append(short.data_ptr())
    if workspace:
        size = L.cache_pages_workspace(c.pages, c.rows)
        ws = torch.empty(max(size, 4), dtype=torch.uint8, device=refs.device)
        args += [ws.data_ptr(), size]
    _check(name, getattr(L, name)(c, *args, _stream(refs)))
    return short


def cache_fork(kv, refs, table, lens, parent, page_size):
    """Make rows of a paged cache copies of others, in place.

    kv [planes, pages, page_size, ...]: every plane (layer; K and V) of the
    cache, any type, each page contiguous; refs INT32 [pages]: how many rows
    hold a page (0: free); table INT32 [rows, width]; lens INT32 [rows].  Row r
    becomes a copy of row parent[r] (INT32 [rows]; itself or no row: it stays): whole
    pages are shared and their refs raised, a part-filled last page is copied
    to a free page of its own, the lowest free pages going to the rows in
    ascending order.  What row r held before is forgotten (cache_free it
    first); a row that names another one in this call is no parent.

    Returns an INT32 tensor of one number: pages that were missing.  Where it
    is not 0, nothing was changed."""
    return _pages_call("cache_fork", kv, refs, table, lens, parent, "parent", page_size, True)


def cache_extend(refs, table, lens, add, page_size):
    """Make room for add[r] (INT32 [rows], >= 0) more tokens in every row, in
    place: lens grows, and the pages that the new lengths need are the lowest
    free ones in ascending order of rows.  refs, table, lens as in cache_fork.

    Returns an INT32 tensor of one number: pages that were missing, or where a
    row of the table is full all that were asked for.  Where it is not 0, nothing
    was changed."""
    return _pages_call("cache_extend", None, refs, table, lens, add, "add", page_size, True)


def cache_free(refs, table, lens, drop, page_size):
    """Empty the rows with drop[r] != 0 (INT32 [rows]), in place: the refs of
    their pages fall by one, their lens become 0 and their table entries -1."""
    _pages_call("cache_free", None, refs, table, lens, drop, "drop", page_size, False, workspace=False)


def cache_compact(kv, refs, table, lens, page_size):
    """Bring the pages in use to the lowest numbers, in place: with n pages in
    use, the i-th free page below n takes the contents, refs and table entries
    of the i-th used page from n on.  kv, refs, table, lens as in cache_fork."""
    _pages_call("cache_compact", kv, refs, table, lens, None, "", page_size, False)


def _logits(logits, targets):
    if logits.dim() != 2:
        raise ValueError("logits must be 2-D")
    rows, vocab = logits.shape
    code = _DTYPE.get(logits.dtype)
    if code is None or code == 3:
        raise TypeError(f"logits must be bfloat16, float16 or float32, got {logits.dtype}")
    if vocab == 0:
        raise ValueError("logits must have at least one column")
    s0, s1 = logits.stride()
    if vocab > 1 and s1 != 1:
        raise ValueError("logits must have unit stride along its rows")
    return rows, vocab, code, (s0 if rows > 1 else vocab), _ints(targets, (rows,), "targets", torch.int64)


def token_logprobs(logits, targets, top_k=0):
    """Log probabilities of given tokens, with entropy and the most likely ones.

    logits [rows, vocab] BF16, FP16 or FP32 (rows may be strided), targets
    INT64 [rows].  Returns TokenLogprobs: logprob [rows] = x[t] - lse (0 where
    the target lies outside [0, vocab)), lse [rows] = log sum exp(x), entropy
    [rows] = -sum p log p, all FP32, and with top_k (at most 64 and vocab)
    top_logprobs FP32 and top_indices INT64 [rows, top_k], largest first, ties
    to the lower index (None otherwise).  -inf logits have p = 0; a row of
    nothing else has lse = -inf, entropy 0 and log probabilities -inf.  Results
    are detached from logits that require a gradient: token_logprobs_backward
    gives it."""
    rows, vocab, code, ld, pt = _logits(logits, targets)
    if not 0 <= top_k <= min(64, vocab):
        raise ValueError("top_k must be at most 64 and at most the vocabulary")
    _on_gpu(logits, "logits", ("targets", targets))
    L, dev = _lib(), logits.device
    stats = torch.empty((3, rows), dtype=torch.float32, device=dev)
    logprob, lse, entropy = stats.unbind(0)
    top_v = top_i = None
    if top_k:
        top_v = torch.empty((rows, top_k), dtype=torch.float32, device=dev)
        top_i = torch.empty((rows, top_k), dtype=torch.int64, device=dev)
    size = L.token_logprobs_workspace(code, rows, vocab, top_k)
    ws = torch.empty(size, dtype=torch.uint8, device=dev) if size > 0 else None
    p = stats.data_ptr()
    _check("token_logprobs",
           L.token_logprobs(code, rows, vocab, logits.data_ptr(), ld, pt, top_k, p, p + 4 * rows, p + 8 * rows,
                            top_v.data_ptr() if top_k else None, top_i.data_ptr() if top_k else None,
                            None if ws is None else ws.data_ptr(), size, _stream(logits)))
    return TokenLogprobs(logprob, lse, entropy, top_v, top_i)


def token_logprobs_backward(logits, targets, lse, entropy, g_logprob=None, g_entropy=None, out=None):
    """Gradient of token_logprobs in the logits: with p = exp(x - lse),
    g_logprob * ([j = t] - p) - g_entropy * p * (log p + entropy), in the
    logits' type.  lse and entropy FP32 [rows] as token_logprobs gave them;
    either gradient (FP32 [rows]) may be None.  Rows without a target have no
    first term."""
    rows, vocab, code, ld, pt = _logits(logits, targets)
    pl, pe = _floats(lse, rows, "lse"), _floats(entropy, rows, "entropy")
    gl = None if g_logprob is None else _floats(g_logprob, rows, "g_logprob")
    ge = None if g_entropy is None else _floats(g_entropy, rows, "g_entropy")
    if out is None:
        out = torch.empty((rows, vocab), dtype=logits.dtype, device=logits.device)
    _shape(out, (rows, vocab), "out")
    if out.dtype != logits.dtype or (vocab > 1 and out.stride(1) != 1):
        raise ValueError("out must have the logits' type and unit stride along its rows")
    _on_gpu(logits, "logits", ("targets", targets), ("lse", lse), ("entropy", entropy), ("g_logprob", g_logprob),
            ("g_entropy", g_entropy), ("out", out))
    _check("token_logprobs_backward",
           _lib().token_logprobs_backward(code, rows, vocab, logits.data_ptr(), ld, pt, pl, pe, gl, ge,
                                          out.data_ptr(), out.stride(0) if rows > 1 else vocab, _stream(logits)))
    return out
