"""token_logprobs and its gradient on the GPU against FP64: types, odd
vocabularies and row strides, ties, rows with nothing left, NaN, and the
gradient against differences."""
import math

import pytest
import torch

import mixed_precision_dense_tiled_amd as mp
from serving_ref import EPS, close, logprobs, logprobs_grad

pytestmark = pytest.mark.gpu
bf16, f16, f32 = torch.bfloat16, torch.float16, torch.float32
U = EPS[f32]


def logits(rows, vocab, dtype, seed=0, scale=2.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, vocab, generator=g) * scale).to(dtype).cuda()


def bounds(x):
    """How far FP32 may be off: an exponent's rounding (its size times 2^-24),
    sums over the vocabulary, joined from pieces whose length is under 2^14."""
    x = x.double().cpu()
    fine = x.masked_fill(~torch.isfinite(x), 0.0)
    size = fine.abs().amax(-1)
    rel = (4 * (size + fine.amax(-1) - fine.amin(-1)) + 256) * U        # of a p, and of their sum
    lse = torch.logsumexp(x, -1)
    base = rel + 4 * U * lse.masked_fill(~torch.isfinite(lse), 0.0).abs()
    return base, rel


def check(x, t, top=0, r=None):
    r = mp.token_logprobs(x, t, top_k=top) if r is None else r
    lp, lse, ent, tv, ti = logprobs(x, t, top)
    base, rel = bounds(x)
    close(r.lse, lse, base, "lse")
    close(r.logprob, lp, base + 4 * U * lp.masked_fill(~torch.isfinite(lp), 0).abs(), "logprob")
    close(r.entropy, ent, 2 * base + 2 * rel * (ent + 1), "entropy")
    if top:
        assert r.top_indices.dtype == torch.int64
        assert torch.equal(r.top_indices.cpu(), ti)
        close(r.top_logprobs, tv, (base[:, None] + 4 * U * tv.masked_fill(~torch.isfinite(tv), 0).abs()), "top")
    else:
        assert r.top_logprobs is None and r.top_indices is None
    return r


def check_grad(x, t, r, gl, ge, out=None, got=None):
    got = mp.token_logprobs_backward(x, t, r.lse, r.entropy, gl, ge, out=out) if got is None else got
    zero = torch.zeros(x.shape[0], device="cuda")
    gl, ge = zero if gl is None else gl, zero if ge is None else ge
    want = logprobs_grad(x, t, gl, ge)
    base, rel = bounds(x)
    _, lse, ent, _, _ = logprobs(x, t)
    p = torch.exp(x.double().cpu() - lse.masked_fill(lse == -math.inf, 0.0)[:, None])
    lp = torch.where(p > 0, p.log(), torch.zeros_like(p))
    a = gl.double().cpu().abs()[:, None], ge.double().cpu().abs()[:, None]
    # p is off by its exponent's rounding and lse's error; the factor by the entropy's
    tol = p * (a[0] + a[1] * (lp.abs() + ent[:, None] + 1)) * (4 * (base + rel)[:, None] + 8 * U) + 4 * U * a[0]
    tol = tol + EPS[x.dtype] * want.abs() * 1.01 + (2.0 ** -25 if x.dtype == f16 else 1e-30)
    close(got, want, tol, "grad")
    return got


@pytest.mark.parametrize("dtype", [bf16, f16, f32])
@pytest.mark.parametrize("rows, vocab", [(1, 1), (3, 2), (5, 7), (2, 64), (4, 255), (3, 1024), (2, 1025), (3, 4099),
                                         (2, 50021), (1, 131072), (257, 5003), (600, 8192)])
def test_sizes(gpu_ok, dtype, rows, vocab):
    x = logits(rows, vocab, dtype, seed=vocab)
    t = torch.randint(-1, vocab, (rows,), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    gl, ge = torch.randn(rows, device="cuda"), torch.randn(rows, device="cuda") * 0.1
    for top in {0, 1, min(5, vocab), min(20, vocab), min(64, vocab)}:
        r = check(x, t, top)
    check_grad(x, t, r, gl, ge)
    check_grad(x, t, r, gl, None)
    check_grad(x, t, r, None, ge)
    assert not check_grad(x, t, r, None, None).any()


@pytest.mark.parametrize("dtype", [bf16, f16, f32])
@pytest.mark.parametrize("rows, vocab", [(4, 3001), (1100, 9001)], ids=["small", "large"])
@pytest.mark.parametrize("shift, grad_shift", [(0, 0), (1, 1), (3, 0), (0, 2)])
def test_rows_off_16_bytes(gpu_ok, dtype, rows, vocab, shift, grad_shift):
    wide = torch.full((rows, vocab + 9), math.nan, dtype=dtype, device="cuda")
    x = wide[:, shift:shift + vocab]
    x.copy_(logits(rows, vocab, dtype, seed=3))
    t = torch.arange(rows, device="cuda") % vocab
    r = check(x, t, 5)
    out = torch.full((rows, vocab + 9), 5.0, dtype=dtype, device="cuda")
    check_grad(x, t, r, torch.randn(rows, device="cuda"), torch.randn(rows, device="cuda"),
               out=out[:, grad_shift:grad_shift + vocab])
    assert (out[:, :grad_shift] == 5).all() and (out[:, grad_shift + vocab:] == 5).all()


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("vocab", [300, 20000])
def test_ties_go_to_the_lower_index(gpu_ok, dtype, vocab):
    rows = 6
    x = torch.zeros(rows, vocab, dtype=dtype)
    x[1] = torch.arange(vocab) % 3
    x[2, vocab // 2:] = 1
    x[3] = -0.0
    x[3, ::2] = 0.0                    # zeros of both signs are equal
    x[4] = -torch.arange(vocab).div(100, rounding_mode="floor").float()
    x[5] = torch.arange(vocab).div(100, rounding_mode="floor").float()
    x = x.cuda()
    t = torch.zeros(rows, dtype=torch.int64, device="cuda")
    for top in (1, 20, 64):
        check(x, t, top)


@pytest.mark.parametrize("dtype", [bf16, f16, f32])
@pytest.mark.parametrize("vocab", [100, 20000])
def test_masked_logits(gpu_ok, dtype, vocab):
    """-inf among the logits, a row of nothing else, and rows of the type's
    lowest value."""
    x = logits(6, vocab, dtype, seed=5)
    low = torch.finfo(dtype).min
    x[0] = -math.inf
    x[1, 7:] = -math.inf
    x[2, :] = -math.inf
    x[2, vocab - 2] = 3.0
    x[3] = low if dtype != f32 else -1e30
    x[4, ::2] = low if dtype != f32 else -1e30
    x[5, 3:90] = -math.inf
    t = torch.tensor([5, 50, vocab - 2, 0, 1, 50], device="cuda")
    r = check(x, t, 20)
    assert r.lse[0] == -math.inf and r.entropy[0] == 0 and r.logprob[0] == -math.inf
    g = check_grad(x, t, r, torch.ones(6, device="cuda"), torch.ones(6, device="cuda"))
    assert not g[0].any() and torch.isfinite(g).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("vocab", [100, 20000])
def test_no_numbers(gpu_ok, bad, vocab):
    x = logits(3, vocab, f32, seed=6)
    x[1, 60] = bad
    t = torch.tensor([1, 2, 3], device="cuda")
    r = mp.token_logprobs(x, t, top_k=5)
    for v in (r.logprob, r.lse, r.entropy, r.top_logprobs):
        assert v[1].isnan().all() and torch.isfinite(v[0]).all() and torch.isfinite(v[2]).all()
    assert r.top_indices[1, 0] == 60 and int(r.top_indices.max()) < vocab and int(r.top_indices.min()) >= 0
    assert len(set(r.top_indices[1].tolist())) == 5
    g = mp.token_logprobs_backward(x, t, r.lse, r.entropy, r.lse, r.lse)
    assert g[1].isnan().all() and torch.isfinite(g[0]).all() and torch.isfinite(g[2]).all()


def test_targets_out_of_range(gpu_ok):
    x = logits(4, 1000, f32, seed=7)
    t = torch.tensor([-100, 1000, 2 ** 40, 3], device="cuda")
    r = check(x, t)
    assert r.logprob[:3].tolist() == [0, 0, 0]
    g = check_grad(x, t, r, torch.ones(4, device="cuda"), None)
    assert not g[:3].any() and g[3].any()


def test_gradient_against_differences(gpu_ok):
    rows, vocab = 3, 40
    x = logits(rows, vocab, f32, seed=8).double().cpu()
    t = torch.tensor([3, 39, -100])
    gl, ge = torch.tensor([1.5, -0.7, 2.0]), torch.tensor([0.3, -1.1, 0.8])

    def loss(x):
        lp, _, ent, _, _ = logprobs(x, t)
        return (gl.double() * lp + ge.double() * ent).sum()

    h = 1e-5
    want = torch.zeros_like(x)
    for i in range(rows):
        for j in range(vocab):
            d = torch.zeros_like(x)
            d[i, j] = h
            want[i, j] = (loss(x + d) - loss(x - d)) / (2 * h)
    xf = x.float().cuda()
    r = mp.token_logprobs(xf, t.cuda())
    got = mp.token_logprobs_backward(xf, t.cuda(), r.lse, r.entropy, gl.cuda(), ge.cuda())
    # differences: h^2 times a third derivative of order 1, and 1e-16 / h; the kernel: FP32
    assert (got.cpu().double() - want).abs().max() < 1e-8 + 2e-6


def test_more_logits_than_the_cache_holds(gpu_ok):
    """Over 256 MB the gradient reads and writes past the caches."""
    rows, vocab = 2200, 65001
    g = torch.Generator("cuda").manual_seed(12)
    x = (torch.randn(rows, vocab, device="cuda", generator=g) * 2.5).to(bf16)
    t = torch.arange(rows, device="cuda") * 29 - 5
    gl, ge = torch.randn(rows, device="cuda", generator=g), torch.randn(rows, device="cuda", generator=g)
    r = mp.token_logprobs(x, t, top_k=5)
    got = mp.token_logprobs_backward(x, t, r.lse, r.entropy, gl, ge)
    some = [0, 1, 1000, rows - 2, rows - 1]
    check(x[some], t[some], 5, mp.TokenLogprobs(*(v[some] for v in r)))
    check_grad(x[some], t[some], r, gl[some], ge[some], got=got[some])


def test_same_bits_again_and_on_another_stream(gpu_ok):
    x = logits(700, 30011, bf16, seed=9)
    t = torch.arange(700, device="cuda")
    w = torch.randn(700, device="cuda")

    def both():
        r = mp.token_logprobs(x, t, top_k=20)
        return [*r, mp.token_logprobs_backward(x, t, r.lse, r.entropy, w, w)]

    first = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = both()
    side.synchronize()
    for a, b in zip(first, other):
        assert torch.equal(a, b)


def test_captured_into_a_graph(gpu_ok):
    x = logits(64, 30011, f32, seed=10)
    t = torch.arange(64, device="cuda")
    w = torch.randn(64, device="cuda")

    def both():
        r = mp.token_logprobs(x, t, top_k=3)
        return [*r, mp.token_logprobs_backward(x, t, r.lse, r.entropy, w, w)]

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for i in range(3):
        x.copy_(logits(64, 30011, f32, seed=11 + i))
        graph.replay()
        torch.cuda.synchronize()
        want = both()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), i


def test_no_rows(gpu_ok):
    x, t = torch.empty(0, 50, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    r = mp.token_logprobs(x, t, top_k=3)
    assert r.logprob.shape == (0,) and r.top_indices.shape == (0, 3)
    assert mp.token_logprobs_backward(x, t, r.lse, r.entropy, r.lse).shape == (0, 50)
