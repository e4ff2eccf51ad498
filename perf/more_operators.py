"""The operators of a decoder layer around its products and its cache, as measured calls.

The root-mean-square norm with the residual's addition and an 8-bit output
(with its gradient), new keys rotated on their way into the paged cache with
the queries beside them, and products grouped by expert: forward, both
gradients, and the W8A8 form.

``run`` computes each in plain torch operations, or, where ``own`` is true,
through this package's entry points.  ``exact`` is the definition in 64 bits.
Lengths and group sizes are a function of the case alone; the seed orders them
and draws every value and every page number.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4, "fp8": 1}


# ---- cases ------------------------------------------------------------------

def _norm(name, **k):
    c = dict(name=name, kind="norm", dtype="bf16", rows=1, dim=4096, residual=True, quant="fp8_blocks",
             train=False)
    c.update(k)
    return c


def _rope(name, **k):
    c = dict(name=name, kind="rope", dtype="bf16", cache="bf16", seqs=1, q_min=1, q_max=1, past_min=0,
             past_max=0, heads=32, kv_heads=8, dim=128, rot=128, interleaved=False, page=16)
    c.update(k)
    return c


def _experts(name, **k):
    c = dict(name=name, kind="experts", dtype="bf16", rows=8, groups=8, skew=0.5, empty=0, k=4096,
             n=14336, trans_b=False, train=False)
    c.update(k)
    return c


def listed():
    return [
        # one token of one user before an FP8 layer: nothing but latency
        _norm("norm_one"),
        # a large prompt batch before a block-scaled FP8 layer
        _norm("norm_fp8", rows=8192, dim=7168),
        # a training step in fp16 over an odd number of tokens, gradients of activations and weight
        _norm("norm_train", dtype="f16", rows=3001, dim=5120, quant="", train=True),
        # a serving batch of single tokens: q rotated, keys and values to their pages
        _rope("rope_decode", seqs=64, past_min=700, past_max=8000),
        # the same for prompt chunks
        _rope("rope_chunk", seqs=16, q_min=100, q_max=1000, past_min=0, past_max=4000),
        # a cache of 8 bits, neighbouring pairs, part of the head rotated
        _rope("rope_fp8", dtype="f16", cache="fp8", seqs=24, q_min=1, q_max=400, past_min=0, past_max=100,
              heads=16, kv_heads=4, dim=80, rot=32, interleaved=True, page=64),
        # one token through its eight of many small experts: latency and eight matrices
        _experts("experts_one", rows=8, groups=64, skew=0.0, k=2048, n=1408),
        # a serving batch, two experts of eight to each of 64 tokens: the weights have to be read
        _experts("experts_decode", rows=128),
        # the same in 8 bits, more tokens
        _experts("experts_w8a8", kind="experts_w8a8", rows=1536, groups=16, k=4096, n=4096, trans_b=True),
        # prompts of 8192 tokens, two experts each
        _experts("experts_prompt", rows=16384, skew=0.25),
        # a training step over many small experts: product, gradients of inputs and weights, idle experts among them
        _experts("experts_train", dtype="f16", rows=12288, groups=32, skew=0.5, empty=3, k=2048, n=1408, train=True),
        # widths that no tile or vector fits
        _experts("experts_odd", dtype="f16", rows=3001, groups=12, empty=1, k=1003, n=1501),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "norm", "rope", "rope", "experts", "experts", "experts_train", "experts_w8a8"])
    if kind == "norm":
        dim = _log(rng, 64, 16384)
        if rng.random() < 0.7:
            dim = (dim + 63) // 64 * 64
        train = rng.random() < 0.4
        return _norm("", dtype=rng.choice(["bf16", "f16", "f32"]), rows=_log(rng, 1, min(16384, 58000000 // dim)),
                     dim=dim, residual=rng.choice([True, False]), train=train,
                     quant="" if train else rng.choice(["", "int8", "fp8_blocks", "fp8_rows"]))
    if kind == "rope":
        dtype = rng.choice(["bf16", "f16"])
        seqs = _log(rng, 1, 64)
        q = _log(rng, 1, 8000 // seqs)
        past = _log(rng, 1, 2000)
        kv_heads = rng.choice([1, 2, 4, 8])
        dim = rng.choice([64, 80, 128])
        return _rope("", dtype=dtype, cache=rng.choice([dtype, dtype, "fp8"]), seqs=seqs,
                     q_min=rng.randint(1, q), q_max=q, past_min=rng.randint(0, past), past_max=past,
                     heads=kv_heads * rng.choice([1, 2, 4]), kv_heads=kv_heads, dim=dim,
                     rot=rng.choice([dim, dim, 32, 64]), interleaved=rng.choice([True, False]),
                     page=rng.choice([16, 32, 64]))
    groups = _log(rng, 1, 64)
    k, n = _log(rng, 128, 8192), _log(rng, 128, 8192)
    if rng.random() < 0.75:
        k, n = (k + 63) // 64 * 64, (n + 63) // 64 * 64
    while groups * k * n > 400000000:
        groups = (groups + 1) // 2
    rows = _log(rng, 1, min(16384, 300000000000 // (k * n)))
    return _experts("", kind="experts_w8a8" if kind == "experts_w8a8" else "experts",
                    dtype=rng.choice(["bf16", "f16"]), rows=rows, groups=groups, skew=rng.choice([0.0, 0.5, 1.0]),
                    empty=rng.randint(0, groups // 4), k=k, n=n,
                    trans_b=kind == "experts_w8a8" or rng.choice([True, False]), train=kind == "experts_train")


# ---- shapes that a case stands for -------------------------------------------

def _spread(lo, hi, n, i):
    """The i-th of n lengths spread between lo and hi."""
    return hi if n == 1 else lo + (hi - lo) * i // (n - 1)


def _lengths(case):
    """(new tokens, all tokens) of each sequence."""
    n = case["seqs"]
    out = []
    for i in range(n):
        q = _spread(case["q_min"], case["q_max"], n, i * 7 % n if n % 7 else i)
        out.append((q, q + _spread(case["past_min"], case["past_max"], n, i)))
    return out


def _held(n, page):
    return (n + page - 1) // page


def _group_rows(case):
    """Rows of each group: the busiest has (groups)^skew times the idlest's, `empty` have none."""
    n = case["groups"] - case["empty"]
    w = [(i + 1) ** -case["skew"] for i in range(n)]
    cut = [int(case["rows"] * sum(w[:i]) / sum(w) + 0.5) for i in range(n)] + [case["rows"]]
    return [b - a for a, b in zip(cut, cut[1:])] + [0] * case["empty"]


def work(case):
    kind = case["kind"]
    if kind == "norm":
        n, es = case["rows"] * case["dim"], _SIZE[case["dtype"]]
        moved = es * (1 + 2 * case["residual"])                       # x; residual read and written
        moved += es if not case["quant"] else 1
        if case["train"]:
            moved += es * (3 + case["residual"])                      # gradient and h in, gradient out
        return {"bytes": n * moved, "flops": n * (14 if case["train"] else 6)}
    if kind == "rope":
        tokens = sum(q for q, _ in _lengths(case))
        es, d = _SIZE[case["dtype"]], case["dim"]
        return {"bytes": tokens * d * (case["heads"] * 2 * es + 2 * case["kv_heads"] * (es + _SIZE[case["cache"]])),
                "flops": tokens * (case["heads"] + case["kv_heads"]) * case["rot"] * 3}
    busy = sum(r > 0 for r in _group_rows(case))
    t, k, n, g = case["rows"], case["k"], case["n"], case["groups"]
    es = 1 if kind == "experts_w8a8" else 2
    once = {"bytes": es * (t * k + busy * k * n) + 2 * t * n, "flops": 2 * t * k * n}
    if not case["train"]:
        return once
    # the inputs' gradient reads the weights and the gradient, the weights' reads both sides' rows
    return {"bytes": 2 * once["bytes"] + 2 * (t * k + t * n + g * k * n), "flops": 3 * once["flops"]}


# ---- inputs -------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    kind = case["kind"]
    st = {"case": case}

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if kind == "norm":
        dt, shape = _DT[case["dtype"]], (case["rows"], case["dim"])
        st["x"] = randn(*shape).to(dt)
        st["residual"] = (randn(*shape) * 3).to(dt) if case["residual"] else None
        st["weight"] = (1 + 0.2 * randn(case["dim"])).to(dt)
        if case["train"]:
            st["grad"] = randn(*shape).to(dt)
            st["grad_residual"] = randn(*shape).to(dt) if case["residual"] else None
        return st
    if kind == "rope":
        seqs = _lengths(case)
        seqs = [seqs[i] for i in torch.randperm(len(seqs), generator=cpu).tolist()]
        page, hk, d = case["page"], case["kv_heads"], case["dim"]
        need = [_held(n, page) for _, n in seqs]
        total = sum(need) + 5
        order = torch.randperm(total, generator=cpu).to(torch.int32)
        table = torch.full((len(seqs), max(max(need), 1)), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        cu = [0]
        for q, _ in seqs:
            cu.append(cu[-1] + q)
        st["table"] = table.cuda()
        st["lens"] = torch.tensor([n for _, n in seqs], dtype=torch.int32).cuda()
        st["cu_q"] = torch.tensor(cu, dtype=torch.int32).cuda()
        st["seqs"] = seqs
        st["inv_freq"] = (10000.0 ** (-torch.arange(0, case["rot"], 2) / case["rot"])).float().cuda()
        dt, fp8 = _DT[case["dtype"]], case["cache"] == "fp8"
        for x in ("k", "v"):
            t = randn(total, page, hk, d)
            st[x + "_cache"] = (t * 32).to(torch.float8_e4m3fn) if fp8 else t.to(dt)
            st[x + "_scale"] = (0.8 + 0.4 * torch.rand(hk, generator=g, device="cuda")) / 32 if fp8 else None
            st[x] = randn(cu[-1], hk, d).to(dt)
        st["q"] = randn(cu[-1], case["heads"], d).to(dt)
        return st
    rows = _group_rows(case)
    st["rows"] = rows = [rows[i] for i in torch.randperm(len(rows), generator=cpu).tolist()]
    cu = [0]
    for r in rows:
        cu.append(cu[-1] + r)
    st["offsets"] = torch.tensor(cu, dtype=torch.int32).cuda()
    t, k, n, e = case["rows"], case["k"], case["n"], case["groups"]
    shape = (e, n, k) if case["trans_b"] else (e, k, n)
    if kind == "experts_w8a8":
        st["x"] = torch.randint(-127, 128, (t, k), generator=g, device="cuda", dtype=torch.int8)
        st["x_scale"] = 0.01 + 0.02 * torch.rand(t, generator=g, device="cuda")
        st["w"] = torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)
        st["w_scale"] = (0.5 + torch.rand((e, n), generator=g, device="cuda")) * k ** -0.5 / 73
        return st
    dt = _DT[case["dtype"]]
    st["a"] = randn(t, k).to(dt)
    st["b"] = torch.empty(shape, dtype=dt, device="cuda")
    for i in range(e):
        st["b"][i] = randn(*shape[1:]) * k ** -0.5
    if case["train"]:
        st["g"] = randn(t, n).to(dt)
    return st


# ---- the plain forms ------------------------------------------------------------

def _blocks(y):
    """[rows, ceil(dim / 128), 128] of y [rows, dim], zeros behind its end."""
    pad = -y.shape[1] % 128
    if pad:
        y = torch.cat([y, y.new_zeros((y.shape[0], pad))], -1)
    return y.view(y.shape[0], -1, 128)


def _plain_norm(st):
    case, x = st["case"], st["x"]
    out = {}
    if case["residual"]:
        out["h"] = x = (x.float() + st["residual"].float()).to(x.dtype)
    # (the sum in 64 bits: codes next to a border go by its last bits)
    mean = x.double().square().sum(-1, keepdim=True) / case["dim"]
    rstd = (1 / torch.sqrt(mean + 1e-6)).float()
    w = st["weight"].float()
    y = x.float() * rstd * w
    if case["quant"] == "int8":
        s = y.abs().amax(-1, keepdim=True) / 127
        codes = torch.round(y / s).clamp(-127, 127).to(torch.int8)
        out["y"], out["scale"] = (codes * s).to(torch.bfloat16), s.squeeze(-1)
    elif case["quant"] == "fp8_rows":
        s = y.abs().amax(-1, keepdim=True) / 448
        out["y"], out["scale"] = (y / s).to(torch.float8_e4m3fn), s.squeeze(-1)
    elif case["quant"]:
        b = _blocks(y)
        s = b.abs().amax(-1, keepdim=True) / 448
        out["y"] = (b / s).view(y.shape[0], -1)[:, :y.shape[1]].to(torch.float8_e4m3fn)
        out["scale"] = s.squeeze(-1)
    else:
        out["y"] = y.to(x.dtype)
    if case["train"]:
        h, g = x.float(), st["grad"].float()
        gw = g * w
        c = (gw * h).sum(-1, keepdim=True) / case["dim"]
        dh = rstd * (gw - h * (rstd * rstd * c))
        if case["residual"]:
            dh = dh + st["grad_residual"].float()
        out["dh"] = dh.to(x.dtype)
        out["dw"] = (g * (h * rstd)).sum(0)
    return out


def _turned(x, cos, sin, interleaved):
    """Rows [tokens, heads, dim] in 32 bits with their first pairs turned."""
    x = x.float()
    r = 2 * cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2], y[..., r // 2:r] = a * cos - b * sin, b * cos + a * sin
    return y


def _places(st):
    """Each new token's position and its slot in the cache."""
    page = st["case"]["page"]
    cu, lens = st["cu_q"].long(), st["lens"].long()
    t = torch.arange(st["q"].shape[0], device=cu.device)
    seq = (t[:, None] >= cu[None, 1:]).sum(-1)
    pos = lens[seq] - (cu[seq + 1] - t)
    return pos, st["table"].long()[seq, pos // page] * page + pos % page


def _plain_rope(st):
    case = st["case"]
    pos, slot = _places(st)
    angle = pos.double()[:, None] * st["inv_freq"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    for x in ("k", "v"):
        new = _turned(st["k"], cos, sin, case["interleaved"]) if x == "k" else st["v"].float()
        cache = st[x + "_cache"]
        flat = cache.view(-1, *cache.shape[2:])
        if st[x + "_scale"] is not None:
            new = (new / st[x + "_scale"][:, None]).clamp(-448, 448)
            flat.view(torch.uint8)[slot] = new.to(cache.dtype).view(torch.uint8)
        else:
            flat[slot] = new.to(cache.dtype)
    return {"q": _turned(st["q"], cos, sin, case["interleaved"]).to(st["q"].dtype), "k": st["k_cache"],
            "v": st["v_cache"]}


def _by_group(st, rows, product):
    """product(group, its rows of `rows`) of every group, one after the other."""
    at, out = 0, []
    for e, n in enumerate(st["rows"]):
        out.append(product(e, rows[at:at + n]))
        at += n
    return out


def _plain_experts(st):
    case, dt = st["case"], st["a"].dtype
    a, b = st["a"].float(), st["b"]
    bt = (lambda e: b[e].float().t()) if case["trans_b"] else (lambda e: b[e].float())
    out = {"d": torch.cat(_by_group(st, a, lambda e, x: x @ bt(e))).to(dt)}
    if case["train"]:
        g = st["g"].float()
        out["da"] = torch.cat(_by_group(st, g, lambda e, x: x @ bt(e).t())).to(dt)
        both = torch.cat([a, g], -1)
        k = case["k"]
        if case["trans_b"]:
            out["db"] = torch.stack(_by_group(st, both, lambda e, x: x[:, k:].t() @ x[:, :k])).to(dt)
        else:
            out["db"] = torch.stack(_by_group(st, both, lambda e, x: x[:, :k].t() @ x[:, k:])).to(dt)
    return out


def _plain_experts_w8a8(st):
    # (sums of whole numbers up to k * 127^2 need more than the 24 bits of FP32)
    x = st["x"].double()
    z = torch.cat(_by_group(st, x, lambda e, r: r @ st["w"][e].double().t())).float()
    per_row = torch.cat(_by_group(st, x, lambda e, r: st["w_scale"][e].expand(r.shape[0], -1)))
    return {"y": (z * st["x_scale"][:, None] * per_row).to(torch.bfloat16)}


# ---- the framework's calls ------------------------------------------------------

def _own_norm(st):
    import mixed_precision_dense_tiled_amd as mp
    case = st["case"]
    r = mp.rms_norm(st["x"], st["weight"], eps=1e-6, residual=st["residual"], quant=case["quant"] or None,
                    return_rstd=case["train"])
    out = {"y": r.out}
    if case["residual"]:
        out["h"] = r.residual
    if case["quant"]:
        out["scale"] = r.scales
        out["y"] = (r.out * r.scales[:, None]).to(torch.bfloat16) if case["quant"] == "int8" else \
            r.out.view(torch.float8_e4m3fn)
    if case["train"]:
        out["dh"], out["dw"] = mp.rms_norm_backward(st["grad"], r.residual if case["residual"] else st["x"],
                                                    st["weight"], r.rstd, grad_residual=st["grad_residual"])
    return out


def _own_rope(st):
    import mixed_precision_dense_tiled_amd as mp
    q = mp.paged_kv_append_rope(st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"], st["table"], st["cu_q"],
                                st["lens"], st["inv_freq"], interleaved=st["case"]["interleaved"],
                                k_scale=st["k_scale"], v_scale=st["v_scale"])
    return {"q": q, "k": st["k_cache"], "v": st["v_cache"]}


def _own_experts(st):
    import mixed_precision_dense_tiled_amd as mp
    case = st["case"]
    out = {"d": mp.gemm_grouped(st["a"], st["b"], st["offsets"], trans_b=case["trans_b"], d16=True)}
    if case["train"]:
        out["da"] = mp.gemm_grouped(st["g"], st["b"], st["offsets"], trans_b=not case["trans_b"], d16=True)
        x, y = (st["g"], st["a"]) if case["trans_b"] else (st["a"], st["g"])
        out["db"] = mp.gemm_grouped_wgrad(x, y, st["offsets"], d16=True)
    return out


def _own_experts_w8a8(st):
    import mixed_precision_dense_tiled_amd as mp
    return {"y": mp.gemm_grouped_w8a8(st["x"], st["x_scale"], st["w"], st["w_scale"], st["offsets"])}


def run(state):
    kind = state["case"]["kind"]
    return globals()[("_own_" if own else "_plain_") + kind](state)


# ---- the definitions in 64 bits --------------------------------------------------

def _e4m3(x):
    """Nearest value of E4M3 (ties to even), at most 448 in size."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_norm(st):
    case = st["case"]
    x = st["x"].double()
    out = {}
    if case["residual"]:
        # what the residual stream holds is its sum rounded to its type
        x = x + st["residual"].double()
        out["h"] = x
        x = x.to(_DT[case["dtype"]]).double()
    r = torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + 1e-6)
    w = st["weight"].double()
    y = x * r * w
    if case["quant"] == "int8":
        s = y.abs().amax(-1) / 127
        out["y"], out["scale"] = torch.round(y / s[:, None]) * s[:, None], s
    elif case["quant"] == "fp8_rows":
        s = y.abs().amax(-1) / 448
        out["y"], out["scale"] = _e4m3(y / s[:, None]), s
    elif case["quant"]:
        cols = torch.arange(case["dim"], device=y.device) // 128
        s = torch.zeros((case["rows"], (case["dim"] + 127) // 128), dtype=torch.float64, device=y.device)
        s = s.scatter_reduce(1, cols.expand(case["rows"], -1), y.abs(), "amax") / 448
        out["y"], out["scale"] = _e4m3(y / s[:, cols]), s
    else:
        out["y"] = y
    if case["train"]:
        g = st["grad"].double()
        u = x * r
        gu = g * w
        out["dh"] = r * (gu - u * (gu * u).mean(-1, keepdim=True))
        if case["residual"]:
            out["dh"] = out["dh"] + st["grad_residual"].double()
        out["dw"] = (g * u).sum(0)
    return out


def _exact_rope(st):
    case = st["case"]
    page = case["page"]
    cu = st["cu_q"].tolist()
    pairs = case["rot"] // 2
    first = torch.arange(pairs, device="cuda") * (2 if case["interleaved"] else 1)
    second = first + (1 if case["interleaved"] else pairs)

    def turn(x, pos):
        z = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                        pos.double()[:, None] * st["inv_freq"].double())[:, None]
        w = torch.complex(x[..., first].double(), x[..., second].double()) * z
        y = x.double()
        y[..., first], y[..., second] = w.real, w.imag
        return y

    out = {"q": st["q"].double(), "k": st["k_cache"].double(), "v": st["v_cache"].double()}
    for b, (nq, n) in enumerate(st["seqs"]):
        rows = slice(cu[b], cu[b + 1])
        at = torch.arange(n - nq, n, device="cuda")
        out["q"][rows] = turn(st["q"][rows], at)
        where = st["table"][b].long()[at // page], at % page
        for x, new in (("k", turn(st["k"][rows], at)), ("v", st["v"][rows].double())):
            if st[x + "_scale"] is not None:
                new = _e4m3(new / st[x + "_scale"].double()[:, None])
            out[x][where] = new
    return out


def _exact_experts(st):
    case = st["case"]
    out = {"d": [], "da": [], "db": []}
    lo = 0
    for e, n in enumerate(st["rows"]):
        a = st["a"][lo:lo + n].double()
        b = st["b"][e].double()
        b = b.mT.contiguous() if case["trans_b"] else b
        out["d"].append(torch.mm(a, b))
        if case["train"]:
            g = st["g"][lo:lo + n].double()
            out["da"].append(torch.mm(g, b.mT))
            grad = torch.mm(a.mT, g)
            out["db"].append(grad.mT if case["trans_b"] else grad)
        lo += n
    r = {"d": torch.cat(out["d"])}
    if case["train"]:
        r["da"], r["db"] = torch.cat(out["da"]), torch.stack(out["db"])
    return r


def _exact_experts_w8a8(st):
    lo, parts = 0, []
    for e, n in enumerate(st["rows"]):
        x = st["x"][lo:lo + n].double() * st["x_scale"][lo:lo + n].double()[:, None]
        parts.append(torch.mm(x, (st["w"][e].double() * st["w_scale"][e].double()[:, None]).mT))
        lo += n
    return {"y": torch.cat(parts)}


def exact(case, seed):
    return globals()["_exact_" + case["kind"]](prepare(case, seed))
