"""The serving operators without a GPU: the Python binding refuses wrong
shapes, types and strides before anything native is called, and the C ABI
refuses wrong arguments on the host (or reports that there is no device)."""
import ctypes
import os
import re

import pytest
import torch

import mixed_precision_dense_tiled_amd as mp
from mixed_precision_dense_tiled_amd import serving

bf16, f16, f32, i32, i64 = torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.int64
SUCCESS, INVALID, MISALIGNED, ALIASING, NO_DEVICE = range(5)
gpu_present = torch.cuda.is_available()


def batch(tokens=5, heads=8, kv_heads=2, dim=64, pages=9, page=16, seqs=2, width=3, dtype=bf16, cache=None):
    c = torch.zeros(pages, page, kv_heads, dim, dtype=cache or dtype)
    return dict(q=torch.zeros(tokens, heads, dim, dtype=dtype), k_cache=c, v_cache=c.clone(),
                table=torch.zeros(seqs, width, dtype=i32), cu_q=torch.zeros(seqs + 1, dtype=i32),
                lens=torch.zeros(seqs, dtype=i32))


def attn(**change):
    a = batch()
    a.update(change)
    return mp.paged_attention(**a)


@pytest.mark.parametrize("change, error, match", [
    (dict(q=torch.zeros(5, 8, dtype=bf16)), ValueError, "tokens, heads, dim"),
    (dict(q=torch.zeros(5, 8, 64)), TypeError, "does not go with"),
    (dict(q=torch.zeros(5, 8, 64, dtype=f16)), TypeError, "does not go with"),
    (dict(q=torch.zeros(5, 8, 48, dtype=bf16)), ValueError, "dim 64"),
    (dict(q=torch.zeros(5, 7, 64, dtype=bf16)), ValueError, "multiple of kv_heads"),
    (dict(q=torch.zeros(5, 0, 64, dtype=bf16)), ValueError, "multiple of kv_heads"),
    (dict(q=torch.zeros(5, 8, 128, dtype=bf16)[..., ::2]), ValueError, "unit stride"),
    (dict(k_cache=torch.zeros(9, 16, 128, dtype=bf16)), ValueError, "k_cache must be"),
    (dict(v_cache=torch.zeros(9, 16, 2, 48, dtype=bf16)), ValueError, "same shape"),
    (dict(v_cache=torch.zeros(9, 2, 16, 64, dtype=bf16).transpose(1, 2)), ValueError, "strides"),
    (dict(k_cache=torch.zeros(9, 16, 2, 64), v_cache=torch.zeros(9, 16, 2, 64)), TypeError, "a cache must be"),
    (dict(table=torch.zeros(2, 3, dtype=i64)), TypeError, "table must be"),
    (dict(table=torch.zeros(2, 6, dtype=i32)[:, ::2]), ValueError, "unit stride"),
    (dict(table=torch.zeros(2, 0, dtype=i32)), ValueError, "at least one column"),
    (dict(cu_q=torch.zeros(2, dtype=i32)), ValueError, "cu_q must have shape"),
    (dict(cu_q=torch.zeros(3, dtype=i64)), TypeError, "cu_q"),
    (dict(lens=torch.zeros(3, dtype=i32)), ValueError, "lens must have shape"),
    (dict(out=torch.zeros(5, 8, 48, dtype=bf16)), ValueError, "out must have shape"),
    (dict(out=torch.zeros(5, 8, 64)), TypeError, "out must be"),
    (dict(lse=torch.zeros(5, 7)), ValueError, "lse must have shape"),
    (dict(lse=torch.zeros(5, 8, dtype=bf16)), ValueError, "lse must be FP32"),
    (dict(k_scale=torch.ones(2)), ValueError, "belong to an FP8 cache"),
    (dict(), ValueError, "GPU"),
])
def test_attention_refusals(change, error, match):
    with pytest.raises(error, match=match):
        attn(**change)


def test_fp8_cache_needs_scales():
    a = batch(cache=torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="needs k_scale"):
        mp.paged_attention(**a)
    with pytest.raises(ValueError, match="k_scale must have shape"):
        mp.paged_attention(**a, k_scale=torch.ones(3), v_scale=torch.ones(2))
    with pytest.raises(TypeError, match="v_scale"):
        mp.paged_attention(**a, k_scale=torch.ones(2), v_scale=torch.ones(2, dtype=bf16))


@pytest.mark.parametrize("k, v, error", [
    (torch.zeros(5, 3, 64, dtype=bf16), None, ValueError),
    (torch.zeros(5, 2, 64, dtype=bf16), torch.zeros(4, 2, 64, dtype=bf16), ValueError),
    (torch.zeros(5, 2, 64, dtype=bf16), torch.zeros(5, 2, 64, dtype=f16), TypeError),
    (torch.zeros(5, 2, 64, dtype=f16), None, TypeError),
    (torch.zeros(5, 2, 64), None, TypeError),
    (torch.zeros(10, 64, dtype=bf16), None, ValueError),
])
def test_append_refusals(k, v, error):
    a = batch()
    del a["q"]
    with pytest.raises(error):
        mp.paged_kv_append(k, k.clone() if v is None else v, **a)


def pages(planes=2, n=8, page=16, rows=3, width=4):
    return dict(kv=torch.zeros(planes, n, page, 2, 16, dtype=bf16), refs=torch.zeros(n, dtype=i32),
                table=torch.zeros(rows, width, dtype=i32), lens=torch.zeros(rows, dtype=i32))


def test_page_refusals():
    p = pages()
    who = torch.zeros(3, dtype=i32)
    with pytest.raises(ValueError, match="kv must be"):
        mp.cache_fork(**{**p, "kv": p["kv"][:, :7]}, parent=who, page_size=16)
    with pytest.raises(ValueError, match="kv must be"):
        mp.cache_fork(**p, parent=who, page_size=8)
    with pytest.raises(ValueError, match="contiguous"):
        mp.cache_fork(**{**p, "kv": p["kv"].transpose(3, 4)}, parent=who, page_size=16)
    with pytest.raises(ValueError, match="parent must have shape"):
        mp.cache_fork(**p, parent=who[:2], page_size=16)
    with pytest.raises(TypeError, match="parent"):
        mp.cache_fork(**p, parent=who.long(), page_size=16)
    with pytest.raises(TypeError, match="refs"):
        mp.cache_compact(**{**p, "refs": p["refs"].long()}, page_size=16)
    del p["kv"]
    with pytest.raises(ValueError, match="add must have shape"):
        mp.cache_extend(**p, add=who[:1], page_size=16)
    with pytest.raises(ValueError, match="lens must have shape"):
        mp.cache_free(**{**p, "lens": who[:2]}, drop=who, page_size=16)
    with pytest.raises(ValueError, match="GPU"):
        mp.cache_free(**p, drop=who, page_size=16)


def test_logprob_refusals():
    x, t = torch.zeros(4, 100), torch.zeros(4, dtype=i64)
    row = torch.zeros(4)
    for args, error in (((x[0], t), ValueError), ((x.double(), t), TypeError), ((x, t[:3]), ValueError),
                        ((x, t.int()), TypeError), ((x, t, 65), ValueError), ((x[:, :10], t, 11), ValueError),
                        ((x, t, -1), ValueError), ((x.t().contiguous().t(), t), ValueError), ((x, t), ValueError)):
        with pytest.raises(error):
            mp.token_logprobs(*args)
    for args, error in (((x, t, row[:3], row), ValueError), ((x, t, row, row.double()), TypeError),
                        ((x, t, row, row, row[:1]), ValueError), ((x, t, row, row, None, row, x[:3]), ValueError),
                        ((x, t, row, row, None, row, x.to(bf16)), ValueError), ((x, t, row, row), ValueError)):
        with pytest.raises(error):
            mp.token_logprobs_backward(*args)


# ---- the C ABI: fake addresses, never read on the host ---------------------------

P = 1 << 40
GB = 1 << 30


def kv(**k):
    a = dict(k=P, v=P + GB, page_stride=2048, slot_stride=128, head_stride=64, pages=10, page_size=16, kv_heads=2,
             dim=64, dtype=0, k_scale=None, v_scale=None)
    a.update(k)
    return serving._PagedKV(*a.values())


def seqs(**k):
    a = dict(table=P + 2 * GB, ld_table=4, cu_q=P + 3 * GB, lens=P + 4 * GB, seqs=2, width=4, tokens=5)
    a.update(k)
    return serving._Sequences(*a.values())


def c_attn(kvs=None, sq=None, heads=8, dtype=0, q=P + 5 * GB, qt=512, qh=64, out=P + 6 * GB, ot=512, oh=64,
           lse=P + 7 * GB, lt=8, scale=1.0, cap=0.0, window=0, ws=P + 8 * GB, size=None):
    L = serving._lib()
    kvs, sq = kvs or kv(), sq or seqs()
    need = L.paged_attention_workspace(kvs, sq, heads)
    return L.paged_attention(kvs, sq, heads, dtype, q, qt, qh, out, ot, oh, lse, lt, scale, cap, window, ws,
                             max(need, 0) if size is None else size, None)


def test_attention_abi():
    for k in (dict(dim=8), dict(dim=72), dict(dim=144), dict(pages=0), dict(page_size=0), dict(kv_heads=0),
              dict(dtype=2), dict(dtype=7), dict(k=None), dict(page_stride=-2048), dict(dtype=3),
              dict(page_stride=1 << 50), dict(slot_stride=1 << 26), dict(pages=(1 << 30) + 1)):
        assert c_attn(kv(**k)) == INVALID, k
    for k in (dict(k=P + 2), dict(slot_stride=129), dict(head_stride=60)):
        assert c_attn(kv(**k)) == MISALIGNED, k
    for k in (dict(width=0), dict(ld_table=3), dict(table=None), dict(cu_q=None), dict(lens=None), dict(tokens=-1),
              dict(width=1 << 27, ld_table=1 << 27), dict(seqs=-1)):
        assert c_attn(sq=seqs(**k)) == INVALID, k
    assert c_attn(sq=seqs(lens=P + 2)) == MISALIGNED
    for k in (dict(heads=7), dict(heads=0), dict(dtype=1), dict(dtype=2), dict(q=None), dict(out=None), dict(lt=7),
              dict(scale=float("nan")), dict(scale=float("inf")), dict(cap=-1.0), dict(window=-1), dict(qt=-512)):
        assert c_attn(**k) == INVALID, k
    for k in (dict(q=P + 5 * GB + 8), dict(oh=60), dict(lse=P + 7 * GB + 2)):
        assert c_attn(**k) == MISALIGNED, k
    for k in (dict(out=P + 5 * GB + 16), dict(out=P + 1024), dict(lse=P + 6 * GB)):
        assert c_attn(**k) == ALIASING, k
    # long tables need a workspace; nothing to do needs none
    long = seqs(width=4096, ld_table=4096)
    assert c_attn(sq=long, size=0) == INVALID
    assert c_attn(sq=long, ws=P + 8 * GB + 16) == MISALIGNED
    assert c_attn(sq=seqs(tokens=0)) == SUCCESS
    if not gpu_present:
        assert c_attn() == NO_DEVICE and c_attn(sq=long) == NO_DEVICE
        scales = dict(k_scale=P + 9 * GB, v_scale=P + 9 * GB)
        assert c_attn(kv(dtype=3, page_stride=2048, **scales)) == NO_DEVICE


def test_append_abi():
    L = serving._lib()

    def call(kvs=None, sq=None, dtype=0, k=P + 5 * GB, kt=128, kh=64, v=P + 6 * GB, vt=128, vh=64):
        return L.paged_kv_append(kvs or kv(), sq or seqs(), dtype, k, kt, kh, v, vt, vh, None)

    assert call(dtype=1) == INVALID and call(dtype=3) == INVALID and call(k=None) == INVALID
    assert call(kt=-8) == INVALID and call(kvs=kv(dtype=3)) == INVALID
    assert call(v=P + 6 * GB + 4) == MISALIGNED and call(kh=63) == MISALIGNED
    assert call(k=P) == ALIASING
    assert call(sq=seqs(tokens=0)) == SUCCESS
    if not gpu_present:
        assert call() == NO_DEVICE


def test_pages_abi():
    L = serving._lib()

    def view(**k):
        a = dict(kv=P, plane_stride=1 << 20, page_stride=4096, page_bytes=4096, planes=2, pages=8, page_size=16,
                 refs=P + GB, table=P + 2 * GB, ld_table=4, lens=P + 3 * GB, rows=3, width=4)
        a.update(k)
        return serving._Pages(*a.values())

    size = L.cache_pages_workspace(8, 3)
    assert size > 0 and L.cache_pages_workspace(-1, 3) == -1

    def fork(c, who=P + 4 * GB, short=P + 5 * GB, ws=P + 6 * GB, n=size):
        return L.cache_fork(c, who, short, ws, n, None)

    for k in (dict(kv=None), dict(page_bytes=8192), dict(planes=-1), dict(page_size=0), dict(width=0),
              dict(ld_table=3), dict(refs=None), dict(table=None), dict(lens=None), dict(plane_stride=-1),
              dict(plane_stride=100), dict(rows=1 << 30)):
        assert fork(view(**k)) == INVALID, k
    assert fork(view(), who=None) == INVALID and fork(view(), ws=None) == INVALID and fork(view(), n=size - 1) == INVALID
    assert fork(view(refs=P + GB + 2)) == MISALIGNED
    assert fork(view(table=P + GB)) == ALIASING and fork(view(), who=P + 3 * GB) == ALIASING
    assert fork(view(lens=P + 64)) == ALIASING
    assert fork(view(rows=0)) == SUCCESS
    assert L.cache_extend(view(), None, None, P + 6 * GB, size, None) == INVALID
    assert L.cache_free(view(), None, None) == INVALID
    assert L.cache_compact(view(), P + 6 * GB, 0, None) == INVALID
    if not gpu_present:
        page_major = view(plane_stride=4096, page_stride=8192)
        assert fork(view()) == NO_DEVICE and fork(page_major) == NO_DEVICE
        assert fork(view(), short=None) == NO_DEVICE
        assert L.cache_extend(view(kv=None), P + 4 * GB, None, P + 6 * GB, size, None) == NO_DEVICE
        assert L.cache_free(view(kv=None), P + 4 * GB, None) == NO_DEVICE
        assert L.cache_compact(view(), P + 6 * GB, size, None) == NO_DEVICE


def test_logprobs_abi():
    L = serving._lib()
    big = 1 << 30

    def call(dtype=2, rows=4, vocab=100, x=P, ld=100, t=P + GB, top=5, lp=P + 2 * GB, lse=P + 3 * GB,
             ent=P + 4 * GB, tv=P + 5 * GB, ti=P + 6 * GB, ws=P + 7 * GB, n=big):
        return L.token_logprobs(dtype, rows, vocab, x, ld, t, top, lp, lse, ent, tv, ti, ws, n, None)

    for k in (dict(dtype=3), dict(rows=-1), dict(vocab=0), dict(x=None), dict(t=None), dict(ld=99), dict(top=65),
              dict(top=-1), dict(lp=None), dict(lse=None), dict(ent=None), dict(tv=None), dict(ti=None),
              dict(ws=None, vocab=9000, ld=9000), dict(n=1, vocab=9000, ld=9000), dict(vocab=10, top=11), dict(rows=1 << 30, vocab=1 << 30, ld=1 << 30)):
        assert call(**k) == INVALID, k
    for k in (dict(x=P + 2), dict(t=P + GB + 4), dict(ti=P + 6 * GB + 4), dict(ws=P + 7 * GB + 8)):
        assert call(**k) == MISALIGNED, k
    assert call(lp=P + 64) == ALIASING and call(lse=P + 2 * GB) == ALIASING and call(ws=P + 6 * GB, vocab=9000, ld=9000) == ALIASING
    assert call(rows=0) == SUCCESS
    assert L.token_logprobs_workspace(2, 4, 100, 65) == -1

    def back(dtype=2, rows=4, vocab=100, x=P, ld=100, t=P + GB, lse=P + 3 * GB, ent=P + 4 * GB, gl=P + 5 * GB,
             ge=None, grad=P + 6 * GB, ldg=100):
        return L.token_logprobs_backward(dtype, rows, vocab, x, ld, t, lse, ent, gl, ge, grad, ldg, None)

    for k in (dict(lse=None), dict(ent=None), dict(grad=None), dict(ldg=99), dict(dtype=5)):
        assert back(**k) == INVALID, k
    assert back(grad=P + 6 * GB + 1) == MISALIGNED and back(gl=P + 5 * GB + 2) == MISALIGNED
    assert back(grad=P) == ALIASING and back(grad=P + 3 * GB) == ALIASING
    if not gpu_present:
        assert call() == NO_DEVICE and call(top=0, tv=None, ti=None) == NO_DEVICE
        assert back() == NO_DEVICE and back(gl=None) == NO_DEVICE


def test_every_declared_entry_point_is_exported():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "mpdt_serving.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b([a-z_][a-z0-9_]*)\s*\(", text))
    assert len(names) == 11
    for n in names:
        assert isinstance(getattr(mp.lib(), n), ctypes._CFuncPtr), n
