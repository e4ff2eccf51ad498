"""The serving operators around the W8A8 / FP8 linear layers, as measured calls.

Four operators that share one paged cache and what the model answers from it:
writing new keys and values into the cache, attention of new tokens over it,
the page bookkeeping that forks, extends, frees and compacts sequences, and
the log probabilities of given tokens (with their gradient) at the end.

``run`` computes each in plain torch operations in 32 bits, or, where ``own``
is true, through this package's entry points.  ``exact`` is the definition in
64 bits.  Sequence lengths are a function of the case alone; the seed orders
them and draws every value and every page number.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4, "fp8": 1}


# ---- cases ------------------------------------------------------------------

def _attn(name, **k):
    c = dict(name=name, kind="attn", dtype="bf16", cache="bf16", seqs=1, q_min=1, q_max=1,
             past_min=0, past_max=0, heads=32, kv_heads=8, dim=128, page=16, softcap=0.0,
             window=0, empty=False)
    c.update(k)
    return c


def _append(name, **k):
    c = dict(name=name, kind="append", dtype="bf16", cache="bf16", seqs=1, q_min=1, q_max=1,
             past_min=0, past_max=0, kv_heads=8, dim=128, page=16)
    c.update(k)
    return c


def _pages(name, kind, **k):
    c = dict(name=name, kind=kind, planes=2, pages=1024, page=16, kv_heads=8, dim=128, seqs=8,
             len_min=100, len_max=1000)
    c.update(k)
    return c


def _logp(name, **k):
    c = dict(name=name, kind="logprobs", dtype="f32", rows=1, vocab=32768, top=0, train=False)
    c.update(k)
    return c


def listed():
    return [
        # one user, one new token, a short conversation: nothing but latency
        _attn("decode_one", past_min=516, past_max=516),
        # a serving batch of single tokens over contexts of very different lengths
        _attn("decode_batch", seqs=64, past_min=700, past_max=8000),
        # few long documents, cache held in 8 bits
        _attn("decode_fp8_long", cache="fp8", seqs=8, past_min=9000, past_max=65000, page=64),
        # two prompts taken in by chunks of 4096 tokens, the last chunk of each
        _attn("chunk_large", seqs=2, q_min=4096, q_max=4096, past_min=12288, past_max=12288, page=64),
        # chunks and single tokens in one batch, fp16, small heads without sharing,
        # capped scores, a sliding window, a sequence without keys and one shorter than its queries
        _attn("mixed_ragged", dtype="f16", cache="f16", seqs=14, q_min=1, q_max=700, past_min=3,
              past_max=5000, heads=16, kv_heads=16, dim=64, page=32, softcap=30.0, window=1500,
              empty=True),
        # the keys and values of prompt chunks written to their pages
        _append("append_chunk", seqs=16, q_min=100, q_max=1000, past_min=0, past_max=4000),
        # the same into a cache of 8 bits
        _append("append_fp8", cache="fp8", seqs=24, q_min=1, q_max=400, past_min=0, past_max=100, page=64),
        # beams: sequences forked, extended by a token, dropped again
        _pages("fork_beams", "fork", planes=8, pages=4096, seqs=32, len_min=20, len_max=1500),
        # a fragmented cache of many layers brought together
        _pages("compact_large", "compact", planes=32, pages=8192, seqs=96, len_min=50, len_max=1200),
        # answers of a small batch, with the most likely alternatives
        _logp("logprobs_serve", rows=4, vocab=131072, top=20),
        # a training step on a policy: log probabilities, entropy, and their gradient
        _logp("logprobs_train", dtype="bf16", rows=2048, vocab=131072, top=5, train=True),
        # the same over an odd vocabulary in 32 bits, tokens without a target among them
        _logp("logprobs_train_odd", rows=777, vocab=50021, top=1, train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "chunk", "chunk", "append", "fork", "compact",
                       "logprobs", "logprobs"])
    page = rng.choice([16, 32, 64, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 7, 8])
    dim = rng.choice([64, 80, 128])
    if kind == "decode":
        dtype = rng.choice(["bf16", "f16"])
        seqs = _log(rng, 1, 64)
        past = _log(rng, 1, min(65000, 300000 // seqs))
        return _attn("", dtype=dtype, cache=rng.choice([dtype, dtype, "fp8"]), seqs=seqs,
                     past_min=rng.randint(0, past), past_max=past, heads=kv_heads * group,
                     kv_heads=kv_heads, dim=dim, page=page,
                     softcap=rng.choice([0.0, 0.0, 30.0]), window=rng.choice([0, 0, 777]))
    if kind == "chunk":
        dtype = rng.choice(["bf16", "f16"])
        seqs = _log(rng, 1, 16)
        q = _log(rng, 2, 4096 // seqs)
        past = _log(rng, 1, 12000)
        return _attn("", dtype=dtype, cache=rng.choice([dtype, dtype, "fp8"]), seqs=seqs,
                     q_min=rng.randint(1, q), q_max=q, past_min=rng.randint(0, past), past_max=past,
                     heads=kv_heads * min(group, 4), kv_heads=kv_heads, dim=dim, page=page,
                     softcap=rng.choice([0.0, 0.0, 30.0]), window=rng.choice([0, 0, 777]),
                     empty=rng.choice([True, False]))
    if kind == "append":
        dtype = rng.choice(["bf16", "f16"])
        seqs = _log(rng, 1, 64)
        q = _log(rng, 1, 8000 // seqs)
        past = _log(rng, 1, 2000)
        return _append("", dtype=dtype, cache=rng.choice([dtype, dtype, "fp8"]), seqs=seqs,
                       q_min=rng.randint(1, q), q_max=q, past_min=rng.randint(0, past), past_max=past,
                       kv_heads=kv_heads, dim=dim, page=page)
    if kind in ("fork", "compact"):
        seqs = _log(rng, 1, 64)
        length = _log(rng, 16, 60000 // seqs)
        planes = 2 * rng.randint(1, 8)
        pages = 2 * seqs * (length // page + 3) + rng.randint(0, 999)
        return _pages("", kind, planes=planes, pages=pages, page=page, kv_heads=kv_heads, dim=dim,
                      seqs=seqs, len_min=rng.randint(1, length), len_max=length)
    rows = _log(rng, 1, 1500)
    return _logp("", dtype=rng.choice(["bf16", "f16", "f32"]), rows=rows,
                 vocab=min(_log(rng, 300, 150000), 120000000 // rows), top=rng.choice([0, 1, 5, 20]),
                 train=rng.choice([True, False]))


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
    if case.get("empty"):
        out += [(3, 0), (9, 4), (0, 21)]
    return out


def _pairs(case):
    """Pairs of a query and a key that it sees, and keys that any query sees."""
    pairs = keys = 0
    for q, n in _lengths(case):
        w = case["window"] or n + 1
        lo, hi = max(n - q, 0), n          # positions of the queries that see a key
        # sum of min(p + 1, w) over p in [lo, hi)
        a = min(max(w - 1, lo), hi)
        pairs += (a * (a + 1) - lo * (lo + 1)) // 2 + (hi - a) * w
        if q and n:
            keys += n - max(lo + 1 - w, 0)
    return pairs, keys


def _seq_lengths(case):
    return [_spread(case["len_min"], case["len_max"], case["seqs"], i) for i in range(case["seqs"])]


def _held(n, page):
    return (n + page - 1) // page


def work(case):
    kind = case["kind"]
    if kind == "attn":
        pairs, keys = _pairs(case)
        tokens = sum(q for q, _ in _lengths(case))
        h, d = case["heads"], case["dim"]
        return {"bytes": 2 * keys * case["kv_heads"] * d * _SIZE[case["cache"]]
                + tokens * h * (2 * d * _SIZE[case["dtype"]] + 4),
                "flops": 4 * pairs * h * d}
    if kind == "append":
        values = 2 * sum(q for q, _ in _lengths(case)) * case["kv_heads"] * case["dim"]
        return {"bytes": values * (_SIZE[case["dtype"]] + _SIZE[case["cache"]]), "flops": values}
    page_bytes = case["planes"] * case["page"] * case["kv_heads"] * case["dim"] * 2 if "planes" in case else 0
    if kind == "fork":
        lens = _seq_lengths(case)
        part = sum(1 for n in lens if n % case["page"])
        table = sum(_held(n, case["page"]) for n in lens)
        return {"bytes": 2 * part * page_bytes + 12 * table + 8 * case["pages"], "flops": table}
    if kind == "compact":
        live = sum(_held(n, case["page"]) for n in _seq_lengths(case))
        moved = live * (case["pages"] - live) // case["pages"]
        return {"bytes": 2 * moved * page_bytes + 12 * live + 8 * case["pages"], "flops": live}
    n = case["rows"] * case["vocab"]
    return {"bytes": n * _SIZE[case["dtype"]] * (2 if case["train"] else 1) + case["rows"] * (28 + 12 * case["top"]),
            "flops": n * (8 if case["train"] else 5)}


# ---- inputs -------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    kind = case["kind"]
    st = {"case": case}
    if kind in ("attn", "append"):
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
        st["table"] = table.cuda()
        st["lens"] = torch.tensor([n for _, n in seqs], dtype=torch.int32).cuda()
        cu = [0]
        for q, _ in seqs:
            cu.append(cu[-1] + q)
        st["cu_q"] = torch.tensor(cu, dtype=torch.int32).cuda()
        st["seqs"] = seqs
        dt = _DT[case["dtype"]]
        fp8 = case["cache"] == "fp8"
        for x in ("k", "v"):
            t = torch.randn((total, page, hk, d), generator=g, device="cuda", dtype=torch.bfloat16)
            st[x + "_cache"] = (t * 32).to(torch.float8_e4m3fn) if fp8 else t.to(dt)
            st[x + "_scale"] = (0.8 + 0.4 * torch.rand(hk, generator=g, device="cuda")) / 32 if fp8 else None
        if kind == "attn":
            st["q"] = torch.randn((cu[-1], case["heads"], d), generator=g, device="cuda").to(dt)
            st["scale"] = d ** -0.5
        else:
            for x in ("k", "v"):
                st[x + "_new"] = torch.randn((cu[-1], hk, d), generator=g, device="cuda").to(dt)
        return st
    if kind in ("fork", "compact"):
        lens = _seq_lengths(case)
        lens = [lens[i] for i in torch.randperm(len(lens), generator=cpu).tolist()]
        page, n_pages, n = case["page"], case["pages"], len(lens)
        need = [_held(x, page) for x in lens]
        order = torch.randperm(n_pages, generator=cpu).to(torch.int32)
        rows = 2 * n if kind == "fork" else n
        table = torch.full((rows, max(need) + 1), -1, dtype=torch.int32)
        refs = torch.zeros(n_pages, dtype=torch.int32)
        at = 0
        for b, k in enumerate(need):
            table[b, :k] = order[at:at + k]
            refs[order[at:at + k].long()] = 1
            at += k
        st["table"], st["refs"] = table.cuda(), refs.cuda()
        st["lens"] = torch.tensor(lens + [0] * (rows - n), dtype=torch.int32).cuda()
        shape = (case["planes"], n_pages, page, case["kv_heads"], case["dim"])
        st["kv"] = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
        if kind == "fork":
            parent = torch.full((rows,), -1, dtype=torch.int32)
            parent[n:] = torch.randperm(n, generator=cpu).to(torch.int32)
            st["parent"] = parent.cuda()
            st["drop"] = (parent >= 0).to(torch.int32).cuda()
            st["add"] = (parent >= 0).to(torch.int32).cuda()
        return st
    rows, vocab = case["rows"], case["vocab"]
    x = torch.randn((rows, vocab), generator=g, device="cuda") * 2.5
    st["logits"] = x.to(_DT[case["dtype"]])
    targets = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    if case["train"]:
        targets[torch.rand(rows, generator=g, device="cuda") < 0.1] = -100
        st["g_logprob"] = torch.randn(rows, generator=g, device="cuda")
        st["g_entropy"] = torch.randn(rows, generator=g, device="cuda") * 0.1
    st["targets"] = targets
    return st


# ---- the plain forms ------------------------------------------------------------

def _plain_attn(st):
    case = st["case"]
    q = st["q"]
    heads, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    group = heads // hk
    out = torch.zeros_like(q)
    lse = torch.full((q.shape[0], heads), -math.inf, dtype=torch.float32, device=q.device)
    at = 0
    for b, (nq, n) in enumerate(st["seqs"]):
        rows = slice(at, at + nq)
        at += nq
        if nq == 0 or n == 0:
            continue
        first = max(n - nq + 1 - case["window"], 0) if case["window"] else 0
        first = first // page * page
        pages = st["table"][b, first // page:_held(n, page)].long()
        pos = torch.arange(first, n, device=q.device)
        qpos = torch.arange(n - nq, n, device=q.device)[:, None]
        hidden = pos[None, :] > qpos
        if case["window"]:
            hidden = hidden | (pos[None, :] <= qpos - case["window"])
        for h in range(hk):
            k = st["k_cache"][pages, :, h].reshape(-1, d)[:n - first].float()
            v = st["v_cache"][pages, :, h].reshape(-1, d)[:n - first].float()
            if st["k_scale"] is not None:
                k, v = k * st["k_scale"][h], v * st["v_scale"][h]
            hs = slice(h * group, (h + 1) * group)
            qh = q[rows, hs].float().transpose(0, 1).reshape(group * nq, d)
            s = (qh @ k.t()).view(group, nq, -1) * st["scale"]
            if case["softcap"]:
                s = case["softcap"] * torch.tanh(s / case["softcap"])
            s = s.masked_fill(hidden, -math.inf)
            m = s.amax(-1, keepdim=True).clamp_min(-3e38)
            p = torch.exp(s - m)
            den = p.sum(-1, keepdim=True)
            o = (p.view(group * nq, -1) @ v).view(group, nq, d) / den.clamp_min(1e-30)
            out[rows, hs] = o.transpose(0, 1).to(out.dtype)
            lse[rows, hs] = (m + torch.log(den)).squeeze(-1).t().masked_fill(hidden.all(-1)[:, None], -math.inf)
    return {"out": out, "lse": lse}


def _values(st, x):
    """What a cache of 8 bits stands for; a wider one as it is."""
    c = st[x + "_cache"]
    return c if st[x + "_scale"] is None else c.float() * st[x + "_scale"][:, None]


def _plain_append(st):
    page = st["case"]["page"]
    cu, lens = st["cu_q"].long(), st["lens"].long()
    t = torch.arange(st["k_new"].shape[0], device=cu.device)
    seq = (t[:, None] >= cu[None, 1:]).sum(-1)
    pos = lens[seq] - (cu[seq + 1] - t)
    keep = pos >= 0
    slot = st["table"].long()[seq, (pos // page).clamp_min(0)] * page + pos % page
    slot, src = slot[keep], t[keep]
    for x in ("k", "v"):
        new = st[x + "_new"][src].float()
        if st[x + "_scale"] is not None:
            new = (new / st[x + "_scale"][:, None]).clamp(-448, 448)
        cache = st[x + "_cache"]
        flat = cache.view(-1, *cache.shape[2:])
        if st[x + "_scale"] is not None:
            flat.view(torch.uint8)[slot] = new.to(cache.dtype).view(torch.uint8)
        else:
            flat[slot] = new.to(cache.dtype)
    return {"k": _values(st, "k"), "v": _values(st, "v")}


def _plain_fork(st):
    case, page = st["case"], st["case"]["page"]
    refs, table, lens, kv = st["refs"].clone(), st["table"].clone(), st["lens"].clone(), st["kv"]
    # fork: whole pages shared, a part-filled one copied to the lowest free page
    child = (st["parent"] >= 0).nonzero().squeeze(-1)
    par = st["parent"][child].long()
    length = lens[par]
    lens[child] = length
    table[child] = table[par]
    full = length // page
    cols = torch.arange(table.shape[1], device=table.device)
    shared = table[child][cols[None, :] < full[:, None]].long()
    refs.index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    part = (length % page > 0).nonzero().squeeze(-1)
    free = (refs == 0).nonzero().squeeze(-1)[:part.numel()]
    kv[:, free] = kv[:, table[par[part], full[part].long()].long()]
    table[child[part], full[part].long()] = free.to(torch.int32)
    refs[free] = 1
    forked = (table.clone(), lens.clone(), refs.clone())
    # extend by the new tokens
    more = (lens + st["add"] + page - 1) // page - (lens + page - 1) // page
    rows = (more > 0).nonzero().squeeze(-1)
    free = (refs == 0).nonzero().squeeze(-1)[:rows.numel()]
    table[rows, ((lens[rows] + page - 1) // page).long()] = free.to(torch.int32)
    refs[free] = 1
    lens += st["add"]
    extended = (table.clone(), lens.clone(), refs.clone())
    # drop
    gone = st["drop"] != 0
    held = (cols[None, :] < ((lens + page - 1) // page)[:, None]) & gone[:, None]
    back = table[held].long()
    refs.index_add_(0, back, -torch.ones_like(back, dtype=torch.int32))
    table[gone] = -1
    lens[gone] = 0
    return {"kv": kv, "forked": forked, "extended": extended, "dropped": (table, lens, refs)}


def _plain_compact(st):
    refs, table, lens, kv = st["refs"].clone(), st["table"].clone(), st["lens"].clone(), st["kv"]
    live = refs > 0
    n = int(live.sum())
    hole = (~live[:n]).nonzero().squeeze(-1)
    mover = live[n:].nonzero().squeeze(-1) + n
    kv[:, hole] = kv[:, mover]
    to = torch.arange(refs.shape[0], dtype=torch.int32, device=refs.device)
    to[mover] = hole.to(torch.int32)
    table = torch.where(table >= 0, to[table.clamp_min(0).long()], table)
    refs[hole] = refs[mover]
    refs[mover] = 0
    return {"kv": kv, "table": table, "lens": lens, "refs": refs}


def _plain_logprobs(st):
    case = st["case"]
    x = st["logits"].float()
    rows = torch.arange(x.shape[0], device=x.device)
    has = st["targets"] >= 0
    at = st["targets"].clamp_min(0)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    den = e.sum(-1, keepdim=True)
    lse = m + torch.log(den)
    entropy = (torch.log(den) - (e * (x - m)).sum(-1, keepdim=True) / den).squeeze(-1)
    out = {"logprob": torch.where(has, x[rows, at] - lse.squeeze(-1), torch.zeros_like(entropy)),
           "lse": lse.squeeze(-1), "entropy": entropy}
    if case["top"]:
        rest = x.clone()
        vals, idx = [], []
        for _ in range(case["top"]):
            i = rest.argmax(-1)
            vals.append(rest[rows, i])
            idx.append(i)
            rest[rows, i] = -math.inf
        out["top_logprobs"] = torch.stack(vals, -1) - lse
        out["top_indices"] = torch.stack(idx, -1)
    if case["train"]:
        logp = x - lse
        p = torch.exp(logp)
        gl = torch.where(has, st["g_logprob"], torch.zeros_like(entropy))[:, None]
        grad = -gl * p - st["g_entropy"][:, None] * p * (logp + entropy[:, None])
        grad[rows, at] += gl.squeeze(-1)
        out["grad"] = grad.to(st["logits"].dtype)
    return out


# ---- the framework's calls ------------------------------------------------------

def _own_attn(st):
    import mixed_precision_dense_tiled_amd as mp
    case = st["case"]
    out, lse = mp.paged_attention(st["q"], st["k_cache"], st["v_cache"], st["table"], st["cu_q"],
                                  st["lens"], scale=st["scale"], softcap=case["softcap"],
                                  window=case["window"], k_scale=st["k_scale"], v_scale=st["v_scale"],
                                  return_lse=True)
    return {"out": out, "lse": lse}


def _own_append(st):
    import mixed_precision_dense_tiled_amd as mp
    mp.paged_kv_append(st["k_new"], st["v_new"], st["k_cache"], st["v_cache"], st["table"],
                       st["cu_q"], st["lens"], k_scale=st["k_scale"], v_scale=st["v_scale"])
    return {"k": _values(st, "k"), "v": _values(st, "v")}


def _own_fork(st):
    import mixed_precision_dense_tiled_amd as mp
    page = st["case"]["page"]
    refs, table, lens, kv = st["refs"].clone(), st["table"].clone(), st["lens"].clone(), st["kv"]
    mp.cache_fork(kv, refs, table, lens, st["parent"], page)
    forked = (table.clone(), lens.clone(), refs.clone())
    mp.cache_extend(refs, table, lens, st["add"], page)
    extended = (table.clone(), lens.clone(), refs.clone())
    mp.cache_free(refs, table, lens, st["drop"], page)
    return {"kv": kv, "forked": forked, "extended": extended, "dropped": (table, lens, refs)}


def _own_compact(st):
    import mixed_precision_dense_tiled_amd as mp
    refs, table, lens, kv = st["refs"].clone(), st["table"].clone(), st["lens"].clone(), st["kv"]
    mp.cache_compact(kv, refs, table, lens, st["case"]["page"])
    return {"kv": kv, "table": table, "lens": lens, "refs": refs}


def _own_logprobs(st):
    import mixed_precision_dense_tiled_amd as mp
    case = st["case"]
    r = mp.token_logprobs(st["logits"], st["targets"], top_k=case["top"])
    out = {"logprob": r.logprob, "lse": r.lse, "entropy": r.entropy}
    if case["top"]:
        out["top_logprobs"], out["top_indices"] = r.top_logprobs, r.top_indices
    if case["train"]:
        out["grad"] = mp.token_logprobs_backward(st["logits"], st["targets"], r.lse, r.entropy,
                                                 st["g_logprob"], st["g_entropy"])
    return out


def run(state):
    kind = state["case"]["kind"]
    return globals()[("_own_" if own else "_plain_") + kind](state)


# ---- the definitions in 64 bits --------------------------------------------------

def _exact_attn(st):
    case = st["case"]
    heads, d, page, cap, w = case["heads"], case["dim"], case["page"], case["softcap"], case["window"]
    share = heads // case["kv_heads"]
    q = st["q"].double()
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    start = 0
    for b, (nq, n) in enumerate(st["seqs"]):
        if n:
            tok = torch.arange(n, device=q.device)
            where = st["table"][b].long()[tok // page]
            for lo in range(0, nq, 1024):
                hi = min(lo + 1024, nq)
                p = n - nq + torch.arange(lo, hi, device=q.device)
                see = tok <= p[:, None]
                if w:
                    see &= tok > p[:, None] - w
                for h in range(heads):
                    k = st["k_cache"][where, tok % page, h // share].double()
                    v = st["v_cache"][where, tok % page, h // share].double()
                    if st["k_scale"] is not None:
                        k = k * st["k_scale"][h // share].double()
                        v = v * st["v_scale"][h // share].double()
                    s = st["scale"] * (q[start + lo:start + hi, h] @ k.t())
                    if cap:
                        s = cap * torch.tanh(s / cap)
                    s[~see] = -math.inf
                    z = torch.logsumexp(s, -1)
                    a = torch.where(see, torch.exp(s - z[:, None]), torch.zeros_like(s))
                    out[start + lo:start + hi, h] = a @ v
                    lse[start + lo:start + hi, h] = z
        start += nq
    return {"out": out, "lse": lse}


def _exact_logprobs(st):
    case = st["case"]
    parts = []
    for lo in range(0, case["rows"], 128):
        x = st["logits"][lo:lo + 128].double()
        t = st["targets"][lo:lo + 128]
        lp = torch.log_softmax(x, -1)
        p = lp.exp()
        ent = -(p * lp).sum(-1)
        has = t >= 0
        pick = lp.gather(1, t.clamp_min(0)[:, None])[:, 0]
        o = {"logprob": torch.where(has, pick, torch.zeros_like(pick)), "lse": torch.logsumexp(x, -1), "entropy": ent}
        if case["top"]:
            order = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :case["top"]]
            o["top_logprobs"], o["top_indices"] = lp.gather(1, order), order
        if case["train"]:
            gl = torch.where(has, st["g_logprob"][lo:lo + 128].double(), torch.zeros_like(pick))
            hot = torch.zeros_like(x).scatter_(1, t.clamp_min(0)[:, None], 1.0)
            o["grad"] = gl[:, None] * (hot - p) - st["g_entropy"][lo:lo + 128].double()[:, None] * p * (lp + ent[:, None])
        parts.append(o)
    return {k: torch.cat([o[k] for o in parts]) for k in parts[0]}


def exact(case, seed):
    if case["kind"] == "attn":
        if work(case)["flops"] > 4e12:
            return None
        return _exact_attn(prepare(case, seed))
    if case["kind"] == "logprobs":
        return _exact_logprobs(prepare(case, seed))
    if case["kind"] == "append":
        # where each token belongs, in whole numbers; its value in the cache's own steps
        st = prepare(case, seed)
        out = {}
        cu = st["cu_q"].tolist()
        for x in ("k", "v"):
            cache = _values(st, x).double()
            new = st[x + "_new"].double()
            if st[x + "_scale"] is not None:
                scale = st[x + "_scale"].double()[:, None]
                cache = st[x + "_cache"].double() * scale
                new = _e4m3(new / scale) * scale
            for b, (nq, n) in enumerate(st["seqs"]):
                at = torch.arange(n - nq, n, device=cache.device)
                cache[st["table"][b].long()[at // case["page"]], at % case["page"]] = new[cu[b]:cu[b + 1]]
            out[x] = cache
        return out
    return None      # pages are moved, not computed


def _e4m3(x):
    """Nearest value of E4M3 (ties to even), at most 448 in size."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)
