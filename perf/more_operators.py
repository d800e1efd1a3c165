"""What is measured of attention with a sliding window and of the paged key-value cache: the
operators with which a model that is trained and prompted on long sequences over W virtual ranks
forgets what lies far back, and answers token by token.

Four operators, each over W ranks in one call:

* ``window``: causal attention in which the query at position p sees the keys j <= p with
  j > p - window or j < sinks (the first tokens stay visible), over shared key heads, ragged key
  counts and rows that continue a cache.
* ``window_backward``: dq, dk and dv from the forward's output and log-sum-exp.
* ``paged``: the last few tokens of each sequence (one, mostly) against a cache that is held in
  pages of a pool, found through a table; with or without a window.
* ``append``: new tokens' keys and values written to their places in the pages.

``own`` selects the library's calls; otherwise ``run`` computes the same in plain torch, in 32 bits.
"""
import math
import random

import torch

own = False


# ---- cases --------------------------------------------------------------------------------------

def listed():
    def window(name, op="window", **kw):
        return dict(dict(name=name, op=op, W=8, b=1, q_tokens=1, kv_tokens=1, heads=8, kv_heads=8,
                         d=128, dtype="bfloat16", window=1, sinks=0, ragged=False, lens_seed=0), **kw)

    def paged(name, **kw):
        return dict(dict(name=name, op="paged", W=8, b=1, q_tokens=1, keys_lo=1, keys_hi=1, heads=8,
                         kv_heads=8, d=128, dtype="bfloat16", page=16, window=0, sinks=0,
                         lens_seed=0), **kw)

    def append(name, **kw):
        return dict(dict(name=name, op="append", W=8, b=1, tokens=1, keys_lo=0, keys_hi=0, kv_heads=8,
                         d=128, dtype="bfloat16", page=16, ragged=False, lens_seed=0), **kw)

    return [
        # a causal video model over the whole clip of the benchmark (21 frames of 45 x 80 tokens):
        # the last three frames and the first one stay visible
        window("window video 75600 tokens", q_tokens=75600, kv_tokens=75600, window=10800, sinks=3600),
        # a prompt with shared key heads and an odd length
        window("window prompt", W=4, b=2, q_tokens=4095, kv_tokens=4095, heads=32, kv_heads=8,
               window=1024, sinks=4),
        # a short padded batch in fp16, a head dimension that is no power of two: latency
        window("window short", W=2, b=2, q_tokens=333, kv_tokens=333, heads=4, kv_heads=4, d=80,
               dtype="float16", window=64, sinks=1, ragged=True, lens_seed=1),
        # training on a long sequence, the first tokens kept
        window("window backward long", "window_backward", q_tokens=16380, kv_tokens=16380,
               window=2048, sinks=4),
        # training: shared key heads, a padded batch, fp16, no first tokens
        window("window backward padded", "window_backward", W=2, b=3, q_tokens=2047, kv_tokens=2047,
               heads=24, kv_heads=8, d=64, dtype="float16", window=512, ragged=True, lens_seed=3),
        # one new token per sequence, long caches of different lengths
        paged("paged one token, long caches", W=2, b=16, keys_lo=12000, keys_hi=32768, heads=32,
              kv_heads=4, page=64, lens_seed=2),
        # many sequences of ordinary lengths, small pages
        paged("paged one token, many sequences", b=256, keys_lo=100, keys_hi=2000, heads=64, kv_heads=8,
              page=16, lens_seed=4),
        # one short sequence: latency
        paged("paged one token, short cache", W=1, keys_lo=1000, keys_hi=1000, d=64),
        # a window over long sequences, whose pages between the first and the last are given back
        paged("paged window, long sequences", W=4, b=32, keys_lo=20000, keys_hi=60000, heads=40,
              kv_heads=8, dtype="float16", page=128, window=4096, sinks=4, lens_seed=5),
        # four drafted tokens each, looked at in one call
        paged("paged four tokens", W=4, b=8, q_tokens=4, keys_lo=3000, keys_hi=9000, heads=32,
              kv_heads=8, page=32, lens_seed=6),
        # each step's new keys and values, one token a sequence
        append("append one token", b=256, keys_lo=100, keys_hi=2000, lens_seed=7),
        # a prompt's, behind a shared beginning
        append("append prompt", W=4, b=4, tokens=16380, keys_lo=0, keys_hi=500, page=64, ragged=True,
               lens_seed=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["window", "window", "window_backward", "paged", "paged", "append"])
    W = rng.choice([1, 2, 3, 4, 8])
    d = rng.choice([64, 64, 72, 80, 96, 120, 128, 128, 128])
    kv_heads = W * rng.choice([1, 1, 2, 3])
    group = rng.choice([1, 1, 2, 3, 4, 8])
    c = dict(op=op, W=W, kv_heads=kv_heads, d=d, dtype=rng.choice(["bfloat16", "bfloat16", "float16"]),
             lens_seed=rng.randint(0, 10 ** 6))
    if op.startswith("window"):
        kv = _log(rng, 60, 32768)
        q = rng.choice([kv, kv, kv, rng.randint(1, min(kv, 40))]) if op == "window" else kv
        c.update(b=rng.choice([1, 1, 2, 3]), q_tokens=q, kv_tokens=kv, heads=kv_heads * group,
                 window=_log(rng, 1, 16384), sinks=rng.choice([0, 1, 4, 16, _log(rng, 1, 1000)]),
                 ragged=rng.random() < 0.4)
        while float(c["q_tokens"]) * min(c["kv_tokens"], c["window"] + c["sinks"] + 128) * \
                c["heads"] * d * c["b"] * 4 > 1.5e12:
            if c["b"] > 1:
                c["b"] = 1
            else:
                same = c["q_tokens"] == c["kv_tokens"]
                c["kv_tokens"] = c["kv_tokens"] // 2 + 1
                c["q_tokens"] = c["kv_tokens"] if same else min(c["q_tokens"], c["kv_tokens"])
        return c
    page = rng.choice([8, 16, 16, 32, 64, 128, 48, 256])
    if op == "append":
        tokens = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 10, 16384)])
        b = _log(rng, 1, 256)
        while b > 1 and float(b) * tokens * kv_heads * d > 2 ** 26:
            b //= 2
        hi = _log(rng, 1, 4000)
        c.update(b=b, tokens=tokens, keys_lo=hi // 3, keys_hi=hi, page=page, ragged=rng.random() < 0.4)
        return c
    hi = _log(rng, 1, 32768)
    b = _log(rng, 1, 256)
    while b > 1 and float(b) * hi * kv_heads * d > 2 ** 28:
        b //= 2
    q = rng.choice([1, 1, 1, rng.randint(2, 64 // group)])
    window = rng.choice([0, 0, _log(rng, 1, 8192)])
    c.update(b=b, q_tokens=q, keys_lo=max(1, hi // 3), keys_hi=hi, heads=kv_heads * group, page=page,
             window=window, sinks=rng.choice([0, 4, _log(rng, 1, 300)]) if window else 0)
    return c


# ---- geometry of a case -------------------------------------------------------------------------

def _share(total, W):
    return [total // W + (1 if r < total % W else 0) for r in range(W)]


def _lens(c):
    """Keys of each batch element: those of a window case's tensors that count, those that a
    sequence's pages hold (before the append, in an append case)."""
    rng = random.Random(c["lens_seed"])
    if c["op"].startswith("window"):
        if not c["ragged"]:
            return [c["kv_tokens"]] * c["b"]
        return [rng.randint(max(1, c["kv_tokens"] // 3), c["kv_tokens"]) for _ in range(c["b"])]
    return [rng.randint(c["keys_lo"], c["keys_hi"]) for _ in range(c["b"])]


def _starts(c):
    """Position of each batch element's first query."""
    if c["op"] == "paged":  # the last tokens are the new ones
        return [n - c["q_tokens"] for n in _lens(c)]
    if c["q_tokens"] == c["kv_tokens"]:
        return [0] * c["b"]
    return [n - c["q_tokens"] for n in _lens(c)]


def _counts(c):
    """Tokens that an append case writes for each sequence."""
    rng = random.Random(c["lens_seed"] + 1)
    return [rng.randint(0, c["tokens"]) if c["ragged"] else c["tokens"] for _ in range(c["b"])]


def _window(c):
    return c["window"] if c["window"] else 2 ** 30


def _pairs_and_keys(c):
    """Visible (query, key) pairs of one head and keys that any query sees, over the batch."""
    pairs = keys = 0
    for n, s in zip(_lens(c), _starts(c)):
        p = torch.arange(max(0, s), s + c["q_tokens"], dtype=torch.int64)  # (before 0: no key)
        hi = (p + 1).clamp(max=n)
        lo = (p + 1 - _window(c)).clamp(min=0)
        first = torch.minimum(lo, hi).clamp(max=c["sinks"])                 # first tokens, apart
        pairs += int((first + (hi - lo).clamp(min=0)).sum())
        if len(p):
            end = int(hi.max())
            begin = min(int(lo.min()), end)
            keys += end - begin + min(begin, c["sinks"])
    return pairs, keys


def work(c):
    if c["op"] == "append":
        return {"bytes": 8 * sum(_counts(c)) * c["kv_heads"] * c["d"] + 4 * c["b"], "flops": 0}
    pairs, keys = _pairs_and_keys(c)
    rows = c["b"] * c["q_tokens"] * c["heads"]
    q, kv = rows * c["d"], keys * c["kv_heads"] * c["d"]
    flops = 4 * c["d"] * pairs * c["heads"]
    if c["op"] != "window_backward":
        return {"bytes": 2 * (2 * q + 2 * kv) + 4 * rows, "flops": flops}
    whole = c["b"] * c["kv_tokens"] * c["kv_heads"] * c["d"]
    # q, o, dO, dq; k, v read where visible; dk, dv written whole
    return {"bytes": 2 * (4 * q + 2 * kv + 2 * whole) + 4 * rows, "flops": 5 * flops // 2}


# ---- inputs -------------------------------------------------------------------------------------

class _Gen:
    def __init__(self, seed, dtype):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        self.dtype = getattr(torch, dtype)

    def randn(self, *shape):
        return torch.randn(shape, generator=self.g, device="cuda", dtype=self.dtype)

    def heads(self, *shape):
        """Normalised head rows scaled by a weight per column, as they leave a QK norm."""
        x = torch.randn(shape, generator=self.g, device="cuda")
        x *= torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + 1e-6)
        x *= 1.0 + 0.3 * torch.randn(shape[-1], generator=self.g, device="cuda")
        return x.to(self.dtype)


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _pages(c, gen, held, kept):
    """A pool's page table for sequences of `held` tokens, pages in no order; the tokens that `kept`
    (per sequence, pairs of positions) leaves out have had their pages given back (-1)."""
    page, b = c["page"], c["b"]
    most = max(1, max(-(-n // page) for n in held))
    at = torch.arange(most)[None, :].expand(b, most)
    need = torch.zeros(b, most, dtype=torch.bool)
    for first, last in kept:
        first, last = torch.tensor(first)[:, None], torch.tensor(last)[:, None]
        need |= (at * page < last) & ((at + 1) * page > first)
    total = int(need.sum())
    pages = total + total // 8 + 1
    order = torch.randperm(pages, generator=gen.g, device="cuda")[:total].to(torch.int32)
    table = torch.full((b, most), -1, dtype=torch.int32, device="cuda")
    table[need.cuda()] = order
    return table, pages


def prepare(case, seed):
    c = case
    gen = _Gen(seed, c["dtype"])
    W, b, d, op = c["W"], c["b"], c["d"], c["op"]
    kn = _share(c["kv_heads"], W)
    st = {"case": c}
    lens = _lens(c)
    if op == "append":
        counts = _counts(c)
        held = [n + m for n, m in zip(lens, counts)]
        st["table"], pages = _pages(c, gen, held, [([0] * b, held)])
        st["k"] = [gen.randn(b, c["tokens"], n, d) for n in kn]
        st["v"] = [gen.randn(b, c["tokens"], n, d) for n in kn]
        st["starts"] = _int32(lens)
        st["counts"] = _int32(counts) if c["ragged"] else None
    else:
        qn = _share(c["heads"], W)
        st["scale"] = d ** -0.5
        st["q"] = [gen.heads(b, c["q_tokens"], n, d) for n in qn]
    if op == "paged":
        end = [max(0, n - c["q_tokens"] + 1 - _window(c)) for n in lens]
        st["table"], pages = _pages(c, gen, lens, [([0] * b, [min(c["sinks"], n) for n in lens]),
                                                   (end, lens)])
        st["kv_lens"] = _int32(lens)
    if op.startswith("window"):
        st["k"] = [gen.heads(b, c["kv_tokens"], n, d) for n in kn]
        st["v"] = [gen.randn(b, c["kv_tokens"], n, d) for n in kn]
        st["kv_lens"] = _int32(lens) if c["ragged"] else None
        st["q_start"] = None if c["q_tokens"] == c["kv_tokens"] else _int32(_starts(c))
    else:
        st["k_pages"] = [gen.randn(pages, c["page"], n, d) for n in kn]
        st["v_pages"] = [gen.randn(pages, c["page"], n, d) for n in kn]
    if op == "window_backward":
        # the forward's outputs, which a training step keeps for the backward
        o, lse = _plain_window(st)
        # (a tensor each: a rank's rows of one tensor need not begin at a 16-byte boundary)
        st["o"], st["lse"] = o, [x.clone() for x in lse]
        st["go"] = [gen.randn(b, c["q_tokens"], n, d) for n in qn]
    if own:
        from ulysses_sequence_all_gb300 import binding as B
        plan = lambda batch, tokens, heads: B.ulysses_plan(W, batch, _share(tokens, W), heads, d,
                                                           c["dtype"])
        need = 0
        if op == "append":
            st["kv_plan"] = plan(b, c["tokens"], kn)
        else:
            st["q_plan"] = plan(b, c["q_tokens"], qn)
        if op.startswith("window"):
            st["kv_plan"] = plan(b, c["kv_tokens"], kn)
        else:
            st["cache_plan"] = plan(pages, c["page"], kn)
        if op in ("window", "paged"):
            st["out"] = [torch.empty_like(x) for x in st["q"]]
            st["out_lse"] = [torch.empty(b, n, c["q_tokens"], device="cuda") for n in qn]
        if op == "window":
            need = B.ulysses_attention_window_workspace(st["q_plan"], st["kv_plan"], c["window"],
                                                        c["sinks"])
        if op == "paged":
            need = B.ulysses_attention_paged_workspace(st["q_plan"], st["cache_plan"])
        if op == "window_backward":
            st["grads"] = [[torch.empty_like(x) for x in st[t]] for t in "qkv"]
            need = B.ulysses_attention_window_backward_workspace(st["q_plan"], st["kv_plan"],
                                                                 c["window"], c["sinks"])
        st["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    return st


# ---- one pass -----------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _run_own(state, state["case"])
    if op == "window":
        return list(_plain_window(state))
    if op == "window_backward":
        return _plain_window_backward(state)
    if op == "paged":
        return _plain_paged(state)
    return _plain_append(state)


def _run_own(st, c):
    from ulysses_sequence_all_gb300 import binding as B
    if c["op"] == "window":
        B.ulysses_attention_window(st["q_plan"], st["kv_plan"], st["q"], st["k"], st["v"], st["out"],
                                   st["out_lse"], scale=st["scale"], window=c["window"],
                                   sinks=c["sinks"], kv_lens=st["kv_lens"], q_start=st["q_start"],
                                   workspace=st["ws"])
        return [st["out"], st["out_lse"]]
    if c["op"] == "window_backward":
        dq, dk, dv = st["grads"]
        B.ulysses_attention_window_backward(
            st["q_plan"], st["kv_plan"], dq, dk, dv, st["q"], st["k"], st["v"], st["o"], st["lse"],
            st["go"], scale=st["scale"], window=c["window"], sinks=c["sinks"], kv_lens=st["kv_lens"],
            q_start=st["q_start"], workspace=st["ws"])
        return [dq, dk, dv]
    if c["op"] == "paged":
        B.ulysses_attention_paged(st["q_plan"], st["cache_plan"], st["q"], st["k_pages"],
                                  st["v_pages"], st["out"], st["out_lse"], st["table"], st["kv_lens"],
                                  scale=st["scale"], window=c["window"], sinks=c["sinks"],
                                  workspace=st["ws"])
        return [st["out"], st["out_lse"]]
    B.ulysses_cache_append(st["kv_plan"], st["cache_plan"], st["k"], st["v"], st["k_pages"],
                           st["v_pages"], st["table"], st["starts"], counts=st["counts"])
    return [st["k_pages"], st["v_pages"]]


# ---- plain forms --------------------------------------------------------------------------------

def _tiles(c):
    """Query tokens at a time, and for each batch element and such a tile: the element, the tile's
    first token, its keys' positions (first tokens, then the window), and which the rows see."""
    most = 2 ** 28 // max(1, c["heads"] * min(c["kv_tokens"], _window(c) + c["sinks"]))
    step = max(64, min(2048, _window(c), most))
    for bb, (n, s) in enumerate(zip(_lens(c), _starts(c))):
        for i in range(0, c["q_tokens"], step):
            last = min(i + step, c["q_tokens"])
            hi = max(0, min(n, s + last))
            lo = min(hi, max(0, s + i + 1 - _window(c)))
            j = torch.cat((torch.arange(min(c["sinks"], lo), device="cuda"),
                           torch.arange(lo, hi, device="cuda")))
            p = torch.arange(s + i, s + last, device="cuda")[:, None]
            yield bb, i, last, j, (j <= p) & ((j > p - _window(c)) | (j < c["sinks"]))


def _rows(x, bb, i, last, nk):
    """(key heads, query heads of each x tokens, d) of a tile of queries, in 32 bits."""
    t = x[bb, i:last].float()
    return t.view(t.shape[0], nk, -1, t.shape[-1]).permute(1, 2, 0, 3).flatten(1, 2)


def _back(x, tokens):
    """_rows' layout to (tokens, query heads, d)."""
    return x.view(x.shape[0], -1, tokens, x.shape[-1]).permute(2, 0, 1, 3).flatten(1, 2)


def _softmax(s):
    """Probabilities and log-sum-exp of masked scores; zeros and minus infinity where all are masked."""
    m = s.amax(-1, keepdim=True) if s.shape[-1] else torch.full_like(s.sum(-1, keepdim=True), -math.inf)
    m = torch.where(m == -math.inf, 0.0, m)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    return p.div_(torch.where(l == 0, 1.0, l)), (m + l.log()).squeeze(-1)


def _plain_window(st):
    c = st["case"]
    sizes, nk = [x.shape[2] for x in st["q"]], c["kv_heads"]
    q, k, v = (torch.cat(st[t], dim=2) for t in "qkv")
    o = torch.empty_like(q)
    lse = torch.empty((c["b"], c["heads"], c["q_tokens"]), device="cuda")
    for bb, i, last, j, see in _tiles(c):
        r = last - i
        s = torch.matmul(_rows(q, bb, i, last, nk), k[bb, j].float().permute(1, 2, 0)) * st["scale"]
        s.view(nk, c["heads"] // nk, r, len(j)).masked_fill_(~see, -math.inf)
        p, z = _softmax(s)
        o[bb, i:last] = _back(torch.matmul(p, v[bb, j].float().transpose(0, 1)), r).to(q.dtype)
        lse[bb, :, i:last] = z.view(c["heads"], r)
    return [x.contiguous() for x in o.split(sizes, 2)], [x.contiguous() for x in lse.split(sizes, 1)]


def _plain_window_backward(st):
    c = st["case"]
    qs, ks, nk = [x.shape[2] for x in st["q"]], [x.shape[2] for x in st["k"]], c["kv_heads"]
    q, k, v, o, go = (torch.cat(st[t], dim=2) for t in ("q", "k", "v", "o", "go"))
    lse = torch.cat(st["lse"], dim=1)
    dq = torch.empty_like(q)
    dk, dv = (torch.zeros((c["b"], nk, c["kv_tokens"], c["d"]), device="cuda") for _ in range(2))
    for bb, i, last, j, see in _tiles(c):
        r = last - i
        tq, to, tg = (_rows(x, bb, i, last, nk) for x in (q, o, go))
        tk, tv = (x[bb, j].float().transpose(0, 1) for x in (k, v))
        z = lse[bb, :, i:last].reshape(nk, -1, 1)
        s = torch.matmul(tq, tk.transpose(1, 2)) * st["scale"]
        p = s.sub_(torch.where(z == -math.inf, 0.0, z)).exp_()
        p.view(nk, c["heads"] // nk, r, len(j)).masked_fill_(~see, 0.0)
        dv[bb].index_add_(1, j, torch.matmul(p.transpose(1, 2), tg))
        ds = torch.matmul(tg, tv.transpose(1, 2)).sub_((tg * to).sum(-1, keepdim=True)).mul_(p)
        dk[bb].index_add_(1, j, torch.matmul(ds.transpose(1, 2), tq) * st["scale"])
        dq[bb, i:last] = _back(torch.matmul(ds, tk) * st["scale"], r).to(q.dtype)
    part = lambda x: [y.contiguous() for y in x.transpose(1, 2).to(k.dtype).split(ks, 2)]
    return [[x.contiguous() for x in dq.split(qs, 2)], part(dk), part(dv)]


def _plain_paged(st):
    c = st["case"]
    sizes, nk, t, page = [x.shape[2] for x in st["q"]], c["kv_heads"], c["q_tokens"], c["page"]
    q = torch.cat(st["q"], dim=2)
    o = torch.empty_like(q)
    lse = torch.empty((c["b"], c["heads"], t), device="cuda")
    longest = st["table"].shape[1] * page
    span = min(longest, _window(c) + t)
    step = max(1, 2 ** 28 // max(1, (span + c["sinks"]) * nk * c["d"]))
    for at in range(0, c["b"], step):
        n = st["kv_lens"][at:at + step, None].long()
        lo = (n - t + 1 - _window(c)).clamp(min=0)
        first = torch.arange(c["sinks"], device="cuda")[None].expand(len(n), -1)
        j = torch.cat((first, lo + torch.arange(span, device="cuda")), 1)   # positions
        fresh = torch.cat((first < lo, (j >= lo)[:, c["sinks"]:]), 1) & (j < n)
        p = n + torch.arange(t, device="cuda") - t                           # of the new tokens
        see = (j[:, None] <= p[..., None]) & ((j[:, None] > p[..., None] - _window(c))
                                              | (j[:, None] < c["sinks"])) & fresh[:, None]
        where = torch.gather(st["table"][at:at + step].long(), 1, (j // page).clamp(max=longest // page - 1))
        where = (where.clamp(min=0), j % page)
        k = torch.cat([x[where] for x in st["k_pages"]], dim=2).float().permute(0, 2, 3, 1)
        x = q[at:at + step].float().view(len(n), t, nk, -1, c["d"]).permute(0, 2, 3, 1, 4)
        s = torch.matmul(x.flatten(2, 3), k) * st["scale"]
        s.view(len(n), nk, c["heads"] // nk, t, s.shape[-1]).masked_fill_(~see[:, None, None], -math.inf)
        pr, z = _softmax(s)
        v = torch.cat([x[where] for x in st["v_pages"]], dim=2).float().transpose(1, 2)
        v.masked_fill_(~fresh[:, None, :, None], 0.0)
        x = torch.matmul(pr, v).view(len(n), nk, -1, t, c["d"])
        o[at:at + step] = x.permute(0, 3, 1, 2, 4).flatten(2, 3).to(q.dtype)
        lse[at:at + step] = z.view(len(n), c["heads"], t)
    return [[x.contiguous() for x in o.split(sizes, 2)], [x.contiguous() for x in lse.split(sizes, 1)]]


def _plain_append(st):
    c = st["case"]
    i = torch.arange(c["tokens"], device="cuda")[None]
    j = st["starts"].long()[:, None] + i
    put = (i < st["counts"][:, None]) if st["counts"] is not None else torch.ones_like(j, dtype=torch.bool)
    last = st["table"].shape[1] - 1
    where = torch.gather(st["table"].long(), 1, (j // c["page"]).clamp(max=last))[put], (j % c["page"])[put]
    for new, pool in ((st["k"], st["k_pages"]), (st["v"], st["v_pages"])):
        for x, y in zip(new, pool):
            y[where] = x[put]
    return [st["k_pages"], st["v_pages"]]


# ---- the definition in 64 bits ------------------------------------------------------------------

def exact(case, seed):
    c = case
    if c["op"] == "append":
        return _exact_append(prepare(case, seed))
    # about 0.8e12 multiply-adds a second in 64 bits, several passes over the scores
    if work(c)["flops"] > (5e12 if c["op"] == "window" else 2e12):
        return None
    st = prepare(case, seed)
    if c["op"] == "window_backward":
        return _exact_window_backward(st)
    return _exact_attention(st)


def _exact_keys(st, r, bb):
    """Batch element bb's keys and values on rank r, (positions, key heads, d) in 64 bits."""
    c = st["case"]
    if c["op"] != "paged":
        return st["k"][r][bb].double(), st["v"][r][bb].double()
    n = _lens(c)[bb]
    held = st["table"][bb, :-(-n // c["page"])].long()
    out = []
    for pool in (st["k_pages"][r], st["v_pages"][r]):
        x = pool[held.clamp(min=0)].flatten(0, 1)[:n].double()
        x[(held < 0).repeat_interleave(c["page"])[:n]] = 0.0  # (given back: no query sees them)
        out.append(x)
    return out


def _exact_blocks(st, bb, total):
    """Blocks of query rows of element bb, and for each the columns any of them sees and the mask."""
    c = st["case"]
    n, s = _lens(c)[bb], _starts(c)[bb]
    j = torch.arange(total, device="cuda")
    for i in range(0, c["q_tokens"], 1000):
        pos = s + torch.arange(i, min(i + 1000, c["q_tokens"]), device="cuda")[:, None]
        far = pos - j
        near = torch.logical_and(far >= 0, far < _window(c))
        see = torch.logical_and(j < n, torch.logical_or(near, torch.logical_and(far >= 0, j < c["sinks"])))
        cols = torch.nonzero(see.any(0)).flatten()
        if len(cols):
            yield slice(i, i + len(pos)), cols, see[:, cols]


def _exact_attention(st):
    outs, lses = [], []
    for r, q in enumerate(st["q"]):
        o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
        lse = torch.full((q.shape[0], q.shape[2], q.shape[1]), -math.inf, dtype=torch.float64, device="cuda")
        for bb in range(q.shape[0]):
            k, v = _exact_keys(st, r, bb)
            g = q.shape[2] // k.shape[1]
            for rows, cols, see in _exact_blocks(st, bb, k.shape[0]):
                x = q[bb, rows].double().unflatten(1, (-1, g))
                s = torch.einsum("imgd,jmd->mgij", x, k[cols]) * st["scale"]
                s = torch.where(see, s, -math.inf)
                z = torch.logsumexp(s, dim=-1)
                e = torch.exp(s - torch.where(z == -math.inf, 0.0, z)[..., None])
                o[bb, rows] = torch.einsum("mgij,jmd->imgd", e, v[cols]).flatten(1, 2)
                lse[bb, :, rows] = z.flatten(0, 1)
        outs.append(o)
        lses.append(lse)
    return [outs, lses]


def _exact_window_backward(st):
    res = [[], [], []]
    for r, (q, k, v) in enumerate(zip(st["q"], st["k"], st["v"])):
        dq, dk, dv = (torch.zeros(x.shape, dtype=torch.float64, device="cuda") for x in (q, k, v))
        g = q.shape[2] // max(1, k.shape[2])
        for bb in range(q.shape[0]):
            for rows, cols, see in _exact_blocks(st, bb, k.shape[1]):
                wide = lambda x: x[bb, rows].double().unflatten(1, (-1, g))
                tq, to, tg = wide(q), wide(st["o"][r]), wide(st["go"][r])
                tk, tv = k[bb, cols].double(), v[bb, cols].double()
                z = st["lse"][r][bb, :, rows].double().unflatten(0, (-1, g))[..., None]
                e = torch.exp(torch.einsum("imgd,jmd->mgij", tq, tk) * st["scale"] - z)
                e = torch.where(torch.logical_and(see, z != -math.inf), e, 0.0)
                dv[bb, cols] += torch.einsum("mgij,imgd->jmd", e, tg)
                e = e * (torch.einsum("imgd,jmd->mgij", tg, tv)
                         - torch.einsum("imgd,imgd->mgi", tg, to)[..., None])
                dq[bb, rows] = st["scale"] * torch.einsum("mgij,jmd->imgd", e, tk).flatten(1, 2)
                dk[bb, cols] += st["scale"] * torch.einsum("mgij,imgd->jmd", e, tq)
        for acc, x in zip(res, (dq, dk, dv)):
            acc.append(x)
    return res


def _exact_append(st):
    c = st["case"]
    counts = _counts(c)
    table = st["table"].cpu()
    res = []
    for new, pools in ((st["k"], st["k_pages"]), (st["v"], st["v_pages"])):
        outs = []
        for x, pool in zip(new, pools):
            y = pool.double()
            flat = y.view(-1, *y.shape[2:])
            for bb, start in enumerate(_lens(c)):
                pos = torch.arange(start, start + counts[bb])
                row = table[bb, pos // c["page"]].long() * c["page"] + pos % c["page"]
                flat[row.cuda()] = x[bb, :counts[bb]].double()
            outs.append(y)
        res.append(outs)
    return res
