"""Plain FP64 definitions of the serving operators, on the CPU, and batches to
hold the kernels against."""
import math

import torch

EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}   # half a step


def e4m3(x):
    """Nearest E4M3 value (ties to even) of x, at most 448 in size."""
    x = x.clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(x / step) * step


class Batch:
    """Sequences (new tokens, all tokens) over a cache with shuffled pages;
    everything on the CPU until gpu() copies it."""

    def __init__(self, seqs, heads, kv_heads, dim, page, dtype=torch.bfloat16, fp8=False, seed=0, spare=3,
                 heads_first=False, junk=False):
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.heads, self.kv_heads, self.dim, self.page, self.dtype = seqs, heads, kv_heads, dim, page, dtype
        need = [-(-n // page) for _, n in seqs]
        self.pages = sum(need) + spare
        order = torch.randperm(self.pages, generator=g).to(torch.int32)
        self.table = torch.full((len(seqs), max(max(need), 1) + 1), -1, dtype=torch.int32)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = order[at:at + k]
            at += k
        self.lens = torch.tensor([n for _, n in seqs], dtype=torch.int32)
        self.cu = torch.tensor([0] + [q for q, _ in seqs]).cumsum(0).to(torch.int32)
        self.tokens = int(self.cu[-1])
        shape = (self.pages, kv_heads, page, dim) if heads_first else (self.pages, page, kv_heads, dim)
        self.scales = [None, None]
        self.caches = []
        for i in range(2):
            c = torch.randn(shape, generator=g)
            if fp8:
                c = (c * 32).to(torch.float8_e4m3fn)
                self.scales[i] = (0.8 + 0.4 * torch.rand(kv_heads, generator=g)) / 32
            else:
                c = c.to(dtype)
            if heads_first:
                c = c.transpose(1, 2)
            self.caches.append(c)
        self.q = torch.randn((self.tokens, heads, dim), generator=g).to(dtype)
        if junk:       # what lies past a sequence's end, and in pages of nobody, is never looked at
            used = torch.zeros(self.pages, page, dtype=torch.bool)
            for b, (_, n) in enumerate(seqs):
                for t in range(n):
                    used[self.table[b, t // page].long(), t % page] = True
            bad = [math.nan, math.inf, -math.inf]
            for c in self.caches:
                if fp8:
                    c.view(torch.uint8)[~used] = 0x7f
                else:
                    c[~used] = torch.tensor([bad[i % 3] for i in range(dim)], dtype=dtype)

    def keys(self, b, h, which, n=None):
        n = self.seqs[b][1] if n is None else n
        t = torch.arange(n)
        c = self.caches[which]
        x = (c.float() if c.dtype == torch.float8_e4m3fn else c)[self.table[b].long()[t // self.page], t % self.page, h]
        x = x.double()
        return x if self.scales[which] is None else x * self.scales[which][h].double()

    def attention(self, scale=None, softcap=0.0, window=0, hidden=None):
        """out, lse, and bounds on how far a kernel may be off in each: the
        weights are rounded once to 16 bits (half a step of FP16 for an FP8
        cache), scores and sums run in FP32.  hidden(b): keys that count as
        absent."""
        scale = self.dim ** -0.5 if scale is None else scale
        out = torch.zeros(self.q.shape, dtype=torch.float64)
        lse = torch.full(self.q.shape[:2], -math.inf, dtype=torch.float64)
        tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
        u = EPS[torch.float32]
        ep = EPS[torch.float16] if self.scales[0] is not None else EPS[self.dtype]
        for b, (nq, n) in enumerate(self.seqs):
            if not nq or not n:
                continue
            rows = slice(int(self.cu[b]), int(self.cu[b + 1]))
            pos, tok = torch.arange(n - nq, n)[:, None], torch.arange(n)
            see = tok <= pos
            if window:
                see &= tok > pos - window
            if hidden is not None:
                see &= ~hidden(b)
            for h in range(self.heads):
                kvh = h // (self.heads // self.kv_heads)
                k, v = self.keys(b, kvh, 0), self.keys(b, kvh, 1)
                v = torch.where(see.any(0)[:, None], v, torch.zeros_like(v))
                k = torch.where(see.any(0)[:, None], k, torch.zeros_like(k))
                q = self.q[rows, h].double()
                s = scale * (q @ k.T)
                # FP32: a dot of `dim` products, the factor, the exponent's rounding (and the cap's terms)
                ds = (self.dim + 4) * u * abs(scale) * (q.abs() @ k.abs().T) + 4 * u * s.abs()
                if softcap:
                    s = softcap * torch.tanh(s / softcap)
                    ds = ds + 8 * u * softcap
                s = s.masked_fill(~see, -math.inf)
                z = torch.logsumexp(s, -1)
                some = see.any(-1)
                p = torch.where(see, torch.exp(s - z.masked_fill(~some, 0.0)[:, None]), torch.zeros_like(s))
                o = p @ v
                d_s = torch.where(see, ds, torch.zeros_like(ds)).amax(-1)
                rel = 2 * d_s + (2 * n + 16) * u                # weights and their sum
                out[rows, h] = o
                tol[rows, h] = (p @ v.abs()) * (ep + rel)[:, None] * 1.01 + EPS[self.dtype] * o.abs() * 1.01 + 1e-7
                lse[rows, h] = z
                tol_lse[rows, h] = d_s + (n + 16) * u + 4 * u * z.masked_fill(~some, 0.0).abs()
        return out, lse, tol, tol_lse

    def gpu(self, device="cuda:0"):
        def put(t):
            return None if t is None else t.to(device)
        k, v = (put(c) for c in self.caches)
        return dict(q=put(self.q), k_cache=k, v_cache=v, table=put(self.table), cu_q=put(self.cu),
                    lens=put(self.lens), k_scale=put(self.scales[0]), v_scale=put(self.scales[1]))


def close(got, want, tol, what=""):
    """Element by element; infinities and NaN in the same places."""
    got, want = got.detach().cpu().double(), want.double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fine), f"{what}: infinities or NaN in other places"
    assert torch.equal(got[~fine & ~want.isnan()], want[~fine & ~want.isnan()]), what
    off = (got - want).abs()[fine] - tol.expand_as(want)[fine]
    assert off.numel() == 0 or off.max() <= 0, \
        f"{what}: {int((off > 0).sum())} of {off.numel()} over the bound, worst by {float(off.max()):.3g}"


class Pages:
    """The page bookkeeping in plain Python: lists and counters."""

    def __init__(self, refs, table, lens, page):
        self.refs, self.table, self.lens, self.page = refs.tolist(), table.tolist(), lens.tolist(), page
        self.copies = []

    def free(self, n):
        got = [p for p, r in enumerate(self.refs) if r == 0][:n]
        return got, n - len(got)

    def fork(self, parent):
        rows, width = range(len(self.lens)), len(self.table[0])
        child = [r for r in rows if 0 <= parent[r] < len(self.lens) and parent[r] != r and parent[parent[r]] < 0]
        part = [r for r in child if self.lens[parent[r]] % self.page and self.lens[parent[r]] // self.page < width]
        got, short = self.free(len(part))
        if short:
            return short
        new = dict(zip(part, got))
        for r in child:
            p = parent[r]
            full = self.lens[p] // self.page
            for pg in self.table[p][:full]:
                self.refs[pg] += 1
            self.table[r], self.lens[r] = list(self.table[p]), self.lens[p]
            if r in new:
                self.copies.append((self.table[p][full], new[r]))
                self.table[r][full] = new[r]
                self.refs[new[r]] = 1
        return 0

    def extend(self, add):
        width, page = len(self.table[0]), self.page
        have = [-(-n // page) for n in self.lens]
        want = [-(-(n + a) // page) for n, a in zip(self.lens, add)]
        past = sum(max(w - width, 0) for w in want)
        need = sum(min(w, width) - h for w, h in zip(want, have))
        if past:
            return need + past
        got, short = self.free(need)
        if short:
            return short
        for r, a in enumerate(add):
            for i in range(have[r], want[r]):
                self.table[r][i] = got.pop(0)
                self.refs[self.table[r][i]] = 1
            self.lens[r] += a
        return 0

    def drop(self, marks):
        for r, m in enumerate(marks):
            if m:
                for pg in self.table[r][:-(-self.lens[r] // self.page)]:
                    self.refs[pg] -= 1
                self.table[r], self.lens[r] = [-1] * len(self.table[r]), 0

    def compact(self):
        n = sum(r > 0 for r in self.refs)
        holes = [p for p in range(n) if self.refs[p] <= 0]
        movers = [p for p in range(n, len(self.refs)) if self.refs[p] > 0]
        to = dict(zip(movers, holes))
        for m, h in to.items():
            self.copies.append((m, h))
            self.refs[h], self.refs[m] = self.refs[m], 0
        self.table = [[to.get(pg, pg) for pg in row] for row in self.table]


def logprobs(x, targets, top=0):
    """(logprob, lse, entropy, top values, top indices) in FP64."""
    x = x.double().cpu()
    targets = targets.cpu()
    lse = torch.logsumexp(x, -1)
    none = lse == -math.inf
    lp = x - lse.masked_fill(none, 0.0)[:, None]
    p = lp.exp()
    entropy = -(p * lp.masked_fill(p == 0, 0.0)).sum(-1)
    has = (targets >= 0) & (targets < x.shape[1])
    pick = lp.gather(1, targets.masked_fill(~has, 0)[:, None])[:, 0]
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :top]
    return pick.masked_fill(~has, 0.0), lse, entropy, lp.gather(1, order), order


def logprobs_grad(x, targets, gl, ge):
    x, targets = x.double().cpu(), targets.cpu()
    _, lse, h, _, _ = logprobs(x, targets)
    none = lse == -math.inf
    lp = x - lse.masked_fill(none, 0.0)[:, None]
    p = lp.exp()
    has = (targets >= 0) & (targets < x.shape[1])
    g = gl.double().cpu().masked_fill(~has, 0.0)[:, None]
    hot = torch.zeros_like(x).scatter_(1, targets.masked_fill(~has, 0)[:, None], 1.0)
    ent = p * (lp.masked_fill(p == 0, 0.0) + h[:, None])
    return (g * (hot - p) - ge.double().cpu()[:, None] * ent).masked_fill(none[:, None], 0.0)
