"""paged_attention and paged_kv_append on the GPU against their FP64
definitions: every type, head sharing, page size and row length, single tokens
and chunks, masks that leave a row empty, strides, and places that do not
exist."""
import math

import pytest
import torch

import mixed_precision_dense_tiled_amd as mp
from serving_ref import Batch, close, e4m3

pytestmark = pytest.mark.gpu
bf16, f16 = torch.bfloat16, torch.float16


def check(b, what="", hidden=None, **k):
    out, lse = mp.paged_attention(**b.gpu(), return_lse=True, **k)
    o, z, tol, tol_z = b.attention(hidden=hidden, **k)
    close(lse, z, tol_z, what + " lse")
    close(out, o, tol, what + " out")
    return out, lse


SINGLES = [(1, 1), (1, 2), (1, 31), (1, 33), (1, 517), (1, 0), (1, 64), (1, 1200)]
CHUNKS = [(40, 40), (1, 300), (130, 700), (0, 21), (9, 4), (3, 0), (65, 64), (257, 1000)]


@pytest.mark.parametrize("dim", [16, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("dtype, fp8", [(bf16, False), (f16, False), (bf16, True), (f16, True)])
@pytest.mark.parametrize("seqs", [SINGLES, CHUNKS], ids=["singles", "chunks"])
def test_types_and_dims(gpu_ok, dim, dtype, fp8, seqs):
    check(Batch(seqs, 4, 2, dim, 16, dtype, fp8, seed=dim), f"dim {dim}")


@pytest.mark.parametrize("page", [1, 3, 16, 24, 128, 1024])
@pytest.mark.parametrize("seqs", [[(1, 1300), (1, 7), (1, 1)], [(70, 1300), (33, 50), (2, 1100)]],
                         ids=["singles", "chunks"])
def test_page_sizes(gpu_ok, page, seqs):
    # pages of one token run past the page numbers that a workgroup keeps at a time
    check(Batch(seqs, 4, 1, 64, page, seed=page), f"page {page}")


@pytest.mark.parametrize("heads, kv_heads", [(1, 1), (8, 8), (6, 2), (7, 1), (16, 2), (20, 1), (48, 1)])
@pytest.mark.parametrize("seqs", [[(1, 200), (1, 90)], [(2, 200), (5, 90)], [(50, 200), (100, 190)]],
                         ids=["singles", "few", "chunks"])
def test_head_sharing(gpu_ok, heads, kv_heads, seqs):
    check(Batch(seqs, heads, kv_heads, 64, 16, seed=heads), f"{heads}/{kv_heads}")


@pytest.mark.parametrize("softcap, window", [(5.0, 0), (0.0, 1), (0.0, 40), (0.0, 5000), (30.0, 200)])
@pytest.mark.parametrize("seqs", [SINGLES, CHUNKS], ids=["singles", "chunks"])
@pytest.mark.parametrize("dtype, fp8", [(bf16, False), (f16, True)])
def test_cap_and_window(gpu_ok, softcap, window, seqs, dtype, fp8):
    check(Batch(seqs, 4, 2, 64, 16, dtype, fp8, seed=window), softcap=softcap, window=window)


@pytest.mark.parametrize("seqs", [SINGLES, CHUNKS], ids=["singles", "chunks"])
def test_large_and_negative_scores(gpu_ok, seqs):
    # scores in the hundreds: the reference moves often, most weights vanish
    check(Batch(seqs, 4, 2, 64, 16, f16, seed=4), scale=20.0)
    check(Batch(seqs, 4, 2, 64, 16, bf16, seed=5), scale=-3.0)
    b = Batch(seqs, 4, 2, 64, 16, bf16, seed=6)
    b.q.zero_()       # all weights equal
    check(b)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seqs", [SINGLES, CHUNKS], ids=["singles", "chunks"])
@pytest.mark.parametrize("window", [0, 50])
def test_places_beyond_a_sequence_are_not_read(gpu_ok, seqs, fp8, window):
    out, lse = check(Batch(seqs, 4, 2, 80, 16, bf16, fp8, seed=8, junk=True), window=window)
    assert not out.isnan().any() and not lse.isnan().any()


@pytest.mark.parametrize("seqs", [[(1, 300), (1, 600), (1, 40)], [(60, 300), (100, 600), (30, 40)]],
                         ids=["singles", "chunks"])
def test_pages_that_do_not_exist_hold_no_keys(gpu_ok, seqs):
    b = Batch(seqs, 4, 2, 64, 16, seed=9)
    b.table[0, 3], b.table[0, 7], b.table[1, 0], b.table[2, :3] = -1, b.pages, 2 ** 31 - 1, -7
    gone = {0: [3, 7], 1: [0], 2: [0, 1, 2]}

    def hidden(i):
        m = torch.zeros(b.seqs[i][1], dtype=torch.bool)
        for p in gone[i]:
            m[16 * p:16 * p + 16] = True
        return m

    real = b.table.clone()
    o = mp.paged_attention(**b.gpu(), return_lse=True)
    b.table = torch.where((real < 0) | (real >= b.pages), 0, real)     # for the definition's own reads
    out, lse, tol, tol_z = b.attention(hidden=hidden)
    close(o[1], lse, tol_z, "lse")
    close(o[0], out, tol, "out")
    assert (o[0][b.cu[2]:] == 0).all() and (o[1][b.cu[2]:] == -math.inf).all()


def test_numbers_that_leave_the_batch_are_cut(gpu_ok):
    b = Batch([(4, 40), (5, 30)], 4, 2, 64, 16, seed=10)
    g = b.gpu()
    g["lens"] = torch.tensor([-5, 10 ** 9], dtype=torch.int32, device="cuda")
    g["cu_q"] = torch.tensor([-3, 4, 10 ** 9], dtype=torch.int32, device="cuda")
    out, lse = mp.paged_attention(**g, return_lse=True)
    assert (out[:4] == 0).all() and (lse[:4] == -math.inf).all()
    assert torch.isfinite(out[4:].float()).all()
    g["cu_q"] = torch.tensor([7, 2, 1], dtype=torch.int32, device="cuda")     # nothing new anywhere
    mp.paged_attention(**g)
    torch.cuda.synchronize()


@pytest.mark.parametrize("seqs", [[(1, 100), (1, 2000)], [(90, 100), (3, 500)]], ids=["singles", "chunks"])
def test_strides(gpu_ok, seqs):
    b = Batch(seqs, 6, 2, 64, 16, seed=11, heads_first=True)
    g = b.gpu()
    assert g["k_cache"].stride(1) < g["k_cache"].stride(2)
    o, z, tol, tol_z = b.attention()
    fused = torch.randn(b.tokens, 10, 64, device="cuda").to(bf16)
    fused[:, 2:8] = g["q"]
    wide = torch.full((len(seqs), 500), 3, dtype=torch.int32, device="cuda")
    wide[:, 5:5 + b.table.shape[1]] = g["table"]
    out = torch.full((b.tokens, 8, 80), 7.0, dtype=bf16, device="cuda")
    lse = torch.full((b.tokens, 9), 7.0, device="cuda")
    g["q"], g["table"] = fused[:, 2:8], wide[:, 5:5 + b.table.shape[1]]
    mp.paged_attention(**g, out=out[:, 1:7, :64], lse=lse[:, :6])
    close(out[:, 1:7, :64], o, tol, "out")
    close(lse[:, :6], z, tol_z, "lse")
    assert (out[:, 0] == 7).all() and (out[:, 7] == 7).all() and (out[..., 64:] == 7).all() and (lse[:, 6:] == 7).all()


@pytest.mark.parametrize("seqs", [[(1, 500)] * 3 + [(1, 3000)], [(700, 2000), (1, 900)]], ids=["singles", "chunks"])
def test_same_bits_again_and_on_another_stream(gpu_ok, seqs):
    g = Batch(seqs, 8, 2, 128, 16, seed=12).gpu()
    first = mp.paged_attention(**g, return_lse=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = mp.paged_attention(**g, return_lse=True)
    side.synchronize()
    for a, c in zip(first, other):
        assert torch.equal(a.view(torch.uint8), c.view(torch.uint8))


def test_captured_into_a_graph(gpu_ok):
    b = Batch([(1, 500), (1, 2000), (1, 17)], 8, 2, 64, 16, seed=13)
    g = b.gpu()
    knew, vnew = (torch.randn(3, 2, 64, device="cuda").to(bf16) for _ in range(2))

    def step():
        mp.paged_kv_append(knew, vnew, g["k_cache"], g["v_cache"], g["table"], g["cu_q"], g["lens"])
        return mp.paged_attention(**g, return_lse=True)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step()
    for i in range(3):
        g["q"].copy_(torch.randn(b.q.shape, device="cuda"))
        g["lens"].sub_(1)
        knew.copy_(torch.randn(knew.shape, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        want = mp.paged_attention(**g, return_lse=True)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), i


def test_cache_past_four_gib(gpu_ok):
    """Pages whose bytes start beyond 2^32, read and written."""
    pages, page, hk, dim = 9000, 64, 8, 64                  # 65536 bytes a page: 590 MB
    shape = (pages, page, hk, dim * 10)                      # rows 10 times as far apart: 5.9 GB
    k, v = (torch.empty(shape, dtype=bf16, device="cuda")[..., :dim] for _ in range(2))
    assert k.stride(0) * 2 * (pages - 1) > 2 ** 32
    b = Batch([(1, 150), (1, 64)], 16, hk, dim, page, seed=14)
    last = pages - b.pages
    g = b.gpu()
    k[last:], v[last:] = g["k_cache"], g["v_cache"]
    table = torch.where(g["table"] >= 0, g["table"] + last, g["table"])
    g.update(k_cache=k, v_cache=v, table=table)
    knew = torch.randn(2, hk, dim, device="cuda").to(bf16)
    mp.paged_kv_append(knew, -knew, k, v, table, g["cu_q"], g["lens"])
    b.caches = [k[last:].cpu(), v[last:].cpu()]
    for s, (_, n) in enumerate(b.seqs):
        pg = b.table[s, (n - 1) // page].long()
        assert torch.equal(b.caches[0][pg, (n - 1) % page], knew[s].cpu())
        assert torch.equal(b.caches[1][pg, (n - 1) % page], -knew[s].cpu())
    out, lse = mp.paged_attention(**g, return_lse=True)
    o, z, tol, tol_z = b.attention()
    close(out, o, tol, "out")
    close(lse, z, tol_z, "lse")


@pytest.mark.parametrize("kind", ["short", "long", "chunks"])
def test_many_sequences(gpu_ok, kind):
    """More sequences than a wave, a workgroup and a planning pass hold."""
    if kind == "short":          # one launch
        seqs, heads = [(1, i % 50) for i in range(1500)], 2
    elif kind == "long":         # shared out over the card
        seqs, heads = [(i % 2, i % 40) for i in range(1500)] + [(1, 3000), (1, 5)], 2
    else:                        # 40 rows a sequence
        seqs, heads = [(1, i % 40) for i in range(1100)] + [(9, 100)], 40
    check(Batch(seqs, heads, 1, 16, 16, bf16, seed=31), kind)


@pytest.mark.parametrize("n", [63, 64, 65, 255, 256, 257])
def test_batches_around_the_plan_sizes(gpu_ok, n):
    check(Batch([(1, 1 + 37 * i % 90) for i in range(n - 1)] + [(1, 2000)], 2, 1, 16, 16, f16, seed=n))
    check(Batch([(3, 1 + 37 * i % 90) for i in range(n - 1)] + [(40, 700)], 16, 1, 16, 16, bf16, seed=n))


def test_empty_batches(gpu_ok):
    b = Batch([(0, 5), (0, 0)], 4, 2, 64, 16)
    out, lse = mp.paged_attention(**b.gpu(), return_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    g = b.gpu()
    del g["q"]
    e = torch.empty(0, 2, 64, dtype=bf16, device="cuda")
    mp.paged_kv_append(e, e, **g)


# ---- append ---------------------------------------------------------------------


@pytest.mark.parametrize("dtype, fp8", [(bf16, False), (f16, False), (bf16, True), (f16, True)])
@pytest.mark.parametrize("page, dim, hk", [(16, 64, 2), (3, 80, 1), (128, 128, 8)])
def test_append(gpu_ok, dtype, fp8, page, dim, hk):
    seqs = [(1, 1), (0, 9), (40, 40), (33, 150), (7, 3), (2, 0), (1, 77)]
    b = Batch(seqs, hk, hk, dim, page, dtype, fp8, seed=page)
    g = b.gpu()
    fused = (torch.randn(b.tokens, 3 * hk, dim, device="cuda") * 4).to(dtype)
    fused.view(torch.int16)[:: 5, :, 3] = fused.view(torch.int16)[:: 5, :, 3] & -32768      # zeros of both signs
    fused[:: 7, :, 5] = math.inf
    k, v = fused[:, hk:2 * hk], fused[:, 2 * hk:]
    want = [c.clone() for c in b.caches]
    for i, new in enumerate((k.cpu(), v.cpu())):
        x = new.double() if not fp8 else (new.float() / b.scales[i][:, None]).double()
        for s, (nq, n) in enumerate(seqs):
            for t in range(nq):
                pos = n - nq + t
                if pos >= 0:
                    pg = b.table[s, pos // page].long()
                    row = x[int(b.cu[s]) + t]
                    if fp8:
                        want[i][pg, pos % page] = e4m3(row).float().to(torch.float8_e4m3fn)
                    else:
                        want[i][pg, pos % page] = new[int(b.cu[s]) + t]
    mp.paged_kv_append(k, v, g["k_cache"], g["v_cache"], g["table"], g["cu_q"], g["lens"], g["k_scale"], g["v_scale"])
    for got, w in zip((g["k_cache"], g["v_cache"]), want):
        assert int((got.cpu().float() != w.float()).sum()) == 0


def test_append_drops_tokens_without_a_place(gpu_ok):
    b = Batch([(20, 40), (3, 9)], 2, 2, 64, 16, seed=3)
    g = b.gpu()
    g["table"][0, 1], g["table"][0, 2] = -1, b.pages
    g["lens"][1] = 10 ** 9
    before = g["k_cache"].clone(), g["v_cache"].clone()
    k = torch.randn(23, 2, 64, device="cuda").to(bf16)
    mp.paged_kv_append(k, k, g["k_cache"], g["v_cache"], g["table"], g["cu_q"], g["lens"])
    assert torch.equal(before[0], g["k_cache"]) and torch.equal(before[1], g["v_cache"])


def test_append_then_attend(gpu_ok):
    """A prompt taken in by chunks and then token by token gives what one
    attention over the whole gives."""
    hk, heads, dim, page, n = 2, 8, 64, 16, 150
    b = Batch([(n, n)], heads, hk, dim, page, seed=21)
    g = b.gpu()
    k = torch.stack([g["k_cache"][g["table"][0, t // page], t % page] for t in range(n)])
    v = torch.stack([g["v_cache"][g["table"][0, t // page], t % page] for t in range(n)])
    kc, vc = torch.full_like(g["k_cache"], math.nan), torch.full_like(g["v_cache"], math.nan)
    outs = []
    at = 0
    for step in (100, 40, 1, 1, 8):
        cu = torch.tensor([0, step], dtype=torch.int32, device="cuda")
        lens = torch.tensor([at + step], dtype=torch.int32, device="cuda")
        mp.paged_kv_append(k[at:at + step], v[at:at + step], kc, vc, g["table"], cu, lens)
        outs.append(mp.paged_attention(g["q"][at:at + step], kc, vc, g["table"], cu, lens))
        at += step
    o, _, tol, _ = b.attention()
    close(torch.cat(outs), o, tol, "by steps")
