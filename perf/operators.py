"""What is measured of the attention operators that a sequence-parallel transformer block runs
between its two relayouts, and of the rotary positions with several axes in front of them.

Four operators, each over W virtual ranks in one call:

* ``rope``: mode 0 with QK RMSNorm and a rotary position of two or three axes (rows and columns of
  an image; time, height and width of a video), text tokens before and after the grid unrotated.
* ``rope_backward``: its gradient (dq, dk and the gradient of the two norm weights).
* ``attention``: softmax(q k^T scale) v of every rank's heads over the whole sequence, with shared
  key heads, causal masks and ragged key lengths; from one query token to tens of thousands.
* ``attention_backward``: dq, dk and dv from the forward's output and log-sum-exp.

``own`` selects the library's calls; otherwise ``run`` computes the same in plain torch, in 32 bits.
"""
import math
import random

import torch

own = False

EPS, THETA = 1e-6, 1e4


# ---- cases --------------------------------------------------------------------------------------

def listed():
    def rope(name, op, **kw):
        return dict(dict(name=name, op=op, W=8, b=1, heads=40, d=128, dtype="bfloat16", axes=3,
                         grid_t=21, grid_h=45, grid_w=80, prefix=0, suffix=0, half_pairs=False,
                         uneven=False), **kw)

    def attn(name, op, **kw):
        return dict(dict(name=name, op=op, W=8, b=1, q_tokens=1, kv_tokens=1, heads=8, kv_heads=8,
                         d=128, dtype="bfloat16", causal=False, align="start", ragged=False,
                         lens_seed=0), **kw)

    return [
        # the video shape of this repository's benchmark: 21 latent frames of 45 x 80 patches
        rope("rope video 75600 tokens", "rope"),
        # the smallest call, where launch latency is all there is
        rope("rope tiny", "rope", W=2, heads=8, grid_t=2, grid_h=4, grid_w=4),
        # the training step of the video shape
        rope("rope backward video", "rope_backward"),
        # text and image tokens in one sequence, two position axes, uneven ranks, fp16 rotate-half
        rope("rope backward text and image", "rope_backward", W=3, b=2, heads=40, axes=2, grid_t=1,
             grid_h=64, grid_w=64, prefix=253, suffix=2, dtype="float16", half_pairs=True,
             uneven=True),
        # self-attention of a video transformer over the whole clip, one head per rank
        attn("attention video 75600 tokens", "attention", q_tokens=75600, kv_tokens=75600),
        # its cross-attention to padded text embeddings
        attn("attention video to text", "attention", q_tokens=75600, kv_tokens=512, heads=40,
             kv_heads=40, ragged=True, lens_seed=1),
        # a causal prompt with shared key heads and an odd length
        attn("attention causal prompt", "attention", W=4, b=2, q_tokens=4095, kv_tokens=4095,
             heads=32, kv_heads=8, causal=True),
        # one new token per sequence against a long, ragged cache
        attn("attention one token, long cache", "attention", W=2, b=16, q_tokens=1,
             kv_tokens=32768, heads=32, kv_heads=4, ragged=True, lens_seed=2),
        # one new token against a short cache: latency
        attn("attention one token, short cache", "attention", W=1, q_tokens=1, kv_tokens=1000,
             heads=8, kv_heads=8, d=64),
        # training: a long clip, full attention
        attn("attention backward long", "attention_backward", q_tokens=16380, kv_tokens=16380),
        # training: causal, shared key heads, padded batch, fp16
        attn("attention backward causal", "attention_backward", W=2, b=3, q_tokens=2047,
             kv_tokens=2047, heads=24, kv_heads=8, d=64, dtype="float16", causal=True, ragged=True,
             lens_seed=3),
        # training: short cross-attention with a head dimension that is no power of two
        attn("attention backward short", "attention_backward", W=2, b=2, q_tokens=333, kv_tokens=77,
             heads=4, kv_heads=4, d=80),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope_backward", "attention", "attention", "attention_backward"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float16"])
    if op.startswith("rope"):
        W = rng.randint(1, 8)
        d = rng.choice([64, 72, 80, 96, 128, 128, 128])
        heads = W * rng.randint(1, max(1, 40 // W))
        uneven = W > 1 and rng.random() < 0.4
        axes = rng.choice([2, 3, 3])
        t = _log(rng, 1, 24) if axes == 3 else 1
        h, w = _log(rng, 3, 96), _log(rng, 3, 96)
        prefix = rng.choice([0, 0, rng.randint(1, 512)])
        suffix = rng.choice([0, 0, rng.randint(1, 64)])
        tokens = t * h * w + prefix + suffix
        limit = 75600 * 40 * 128
        b = max(1, min(rng.choice([1, 1, 2, 3]), limit // (tokens * heads * d)))
        while tokens * heads * d * b > limit:
            h = max(3, h // 2)
            tokens = t * h * w + prefix + suffix
        return dict(op=op, W=W, b=b, heads=heads, d=d, dtype=dtype, axes=axes, grid_t=t, grid_h=h,
                    grid_w=w, prefix=prefix, suffix=suffix, half_pairs=rng.random() < 0.4,
                    uneven=uneven)
    W = rng.choice([1, 2, 3, 4, 8])
    d = rng.choice([64, 64, 72, 80, 96, 120, 128, 128, 128])
    group = rng.choice([1, 1, 1, 2, 3, 4, 8])
    kv_heads = W * rng.choice([1, 1, 2, 5])
    heads = kv_heads * group
    b = rng.choice([1, 1, 2, 3, 8])
    kind = rng.choice(["self", "self", "cross", "one", "few"])
    if op == "attention_backward" and kind in ("one", "few"):
        kind = "self"
    kv = _log(rng, 60, 32768)
    q = {"self": kv, "cross": _log(rng, 60, 32768), "one": 1, "few": rng.randint(2, 40)}[kind]
    kv = max(kv, q) if kind == "few" else kv
    causal = kind != "cross" and rng.random() < 0.5
    limit = 2.0e12 if op == "attention" else 1.0e12
    while float(q) * kv * heads * d * b * 4 > limit:
        if b > 1:
            b = b // 2
        else:
            kv = max(1, kv // 2 + 1)
            q = kv if kind == "self" else max(1, q // 2 + 1) if kind == "cross" else q
    while kv * kv_heads * d * b > 2 ** 29:
        b, kv = max(1, b // 2), kv // 2 + 1
    return dict(op=op, W=W, b=b, q_tokens=q, kv_tokens=kv, heads=heads, kv_heads=kv_heads, d=d,
                dtype=dtype, causal=causal, align="start" if kind == "self" else "end",
                ragged=rng.random() < 0.5, lens_seed=rng.randint(0, 10 ** 6))


# ---- geometry of a case -------------------------------------------------------------------------

def _tokens(c):
    return c["prefix"] + c["grid_t"] * c["grid_h"] * c["grid_w"] + c["suffix"]


def _share(total, W, uneven):
    """`total` over W ranks: even with the remainder on the lowest, or a tenth of the last rank's
    share (one at least) moved to the first."""
    out = [total // W + (1 if r < total % W else 0) for r in range(W)]
    if uneven and W > 1 and out[-1] > 0:
        move = max(1, out[-1] // 10)
        out[0] += move
        out[-1] -= move
    return out


def _rope_splits(c):
    return _share(_tokens(c), c["W"], c["uneven"]), _share(c["heads"], c["W"], c["uneven"])


def _grid(c):
    """(extents, pairs) of the position axes: the d/2 rotary pairs split over the axes."""
    d = c["d"]
    if c["axes"] == 3:
        return [c["grid_t"], c["grid_h"], c["grid_w"]], [d // 2 - 2 * (d // 6), d // 6, d // 6]
    return [c["grid_h"], c["grid_w"]], [d // 2 - d // 4, d // 4]


def _lens(c):
    """Keys each batch element holds: all, or a ragged batch that goes with the case."""
    if not c["ragged"]:
        return [c["kv_tokens"]] * c["b"]
    rng = random.Random(c["lens_seed"])
    return [rng.randint(min(c["kv_tokens"], max(1, c["kv_tokens"] // 3)), c["kv_tokens"])
            for _ in range(c["b"])]


def _starts(c):
    """Position of the first query of each batch element (causal cases)."""
    if c["align"] == "start":
        return [0] * c["b"]
    return [n - c["q_tokens"] for n in _lens(c)]


def _pairs(c):
    """Visible (query, key) pairs of one head, over the batch."""
    total = 0
    for n, s in zip(_lens(c), _starts(c)):
        if not c["causal"]:
            total += c["q_tokens"] * n
            continue
        for_full = max(0, min(c["q_tokens"], c["q_tokens"] + s + 1 - n))  # rows that see all n keys
        ramp = c["q_tokens"] - for_full
        first = s + 1                                                    # keys the first row sees
        skip = min(ramp, max(0, -first + 1)) if first < 1 else 0         # rows that see none
        lo = first + skip
        cnt = ramp - skip
        total += for_full * n + cnt * lo + cnt * (cnt - 1) // 2
    return total


def work(c):
    if c["op"].startswith("rope"):
        elems = c["b"] * _tokens(c) * c["heads"] * c["d"]
        back = c["op"] == "rope_backward"
        return {"bytes": (12 if back else 8) * elems + (16 if back else 8) * c["d"],
                "flops": (24 if back else 14) * elems}
    n = c["b"] * c["q_tokens"] * c["heads"]
    q_elems, kv_elems = n * c["d"], sum(_lens(c)) * c["kv_heads"] * c["d"]
    all_kv = c["b"] * c["kv_tokens"] * c["kv_heads"] * c["d"]
    pairs = _pairs(c) * c["heads"]
    if c["op"] == "attention":
        return {"bytes": 2 * (2 * q_elems + 2 * kv_elems) + 4 * n, "flops": 4 * c["d"] * pairs}
    # q, o, dO, dq; k, v read where visible; dk, dv written whole
    return {"bytes": 2 * (4 * q_elems + 2 * kv_elems + 2 * all_kv) + 4 * n,
            "flops": 10 * c["d"] * pairs}


# ---- inputs -------------------------------------------------------------------------------------

class _Gen:
    def __init__(self, seed, dtype):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        self.dtype = getattr(torch, dtype)

    def randn(self, *shape):
        return torch.randn(shape, generator=self.g, device="cuda").to(self.dtype)

    def heads(self, w, *shape):
        """Normalised head rows scaled by a weight per column, as they leave a QK norm."""
        x = torch.randn(shape, generator=self.g, device="cuda")
        x *= torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + EPS)
        x *= w
        return x.to(self.dtype)


def prepare(case, seed):
    c = case
    gen = _Gen(seed, c["dtype"])
    st = {"case": c}
    W, b, d = c["W"], c["b"], c["d"]
    if c["op"].startswith("rope"):
        seq, heads = _rope_splits(c)
        N, S = c["heads"], _tokens(c)
        st["q"] = [gen.randn(b, s, N, d) for s in seq]
        st["k"] = [gen.randn(b, s, N, d) for s in seq]
        st["w"] = 1.0 + 0.1 * torch.randn((2, d), generator=gen.g, device="cuda")
        if c["op"] == "rope_backward":
            st["gq"] = [gen.randn(b, S, n, d) for n in heads]
            st["gk"] = [gen.randn(b, S, n, d) for n in heads]
        if own:
            from ulysses_sequence_all_gb300 import binding as B
            plan = B.ulysses_plan(W, b, seq, heads, d, c["dtype"])
            B.ulysses_plan_set_rope_pairs(plan, B.ULY_ROPE_HALF if c["half_pairs"]
                                          else B.ULY_ROPE_ADJACENT)
            extents, pairs = _grid(c)
            B.ulysses_plan_set_rope_grid(plan, extents, pairs, first=c["prefix"])
            st["plan"] = plan
            if c["op"] == "rope":
                st["out"] = [[torch.empty(b, S, n, d, dtype=gen.dtype, device="cuda")
                              for n in heads] for _ in range(2)]
            else:
                st["out"] = [[torch.empty_like(x) for x in st[t]] for t in ("q", "k")]
                st["dw"] = torch.empty_like(st["w"])
                st["ws"] = torch.empty(B.ulysses_qk_fused_backward_workspace(plan),
                                       dtype=torch.uint8, device="cuda")
        return st
    qn, kn = _share(c["heads"], W, False), _share(c["kv_heads"], W, False)
    wq = 1.0 + 0.3 * torch.randn(d, generator=gen.g, device="cuda")
    wk = 1.0 + 0.3 * torch.randn(d, generator=gen.g, device="cuda")
    st["q"] = [gen.heads(wq, b, c["q_tokens"], n, d) for n in qn]
    st["k"] = [gen.heads(wk, b, c["kv_tokens"], n, d) for n in kn]
    st["v"] = [gen.randn(b, c["kv_tokens"], n, d) for n in kn]
    st["scale"] = d ** -0.5
    lens = torch.tensor(_lens(c), dtype=torch.int32, device="cuda")
    starts = torch.tensor(_starts(c), dtype=torch.int32, device="cuda")
    st["kv_lens"] = lens if c["ragged"] else None
    st["q_start"] = starts if c["causal"] and c["align"] == "end" else None
    if c["op"] == "attention_backward":
        # the forward's outputs, which a training step keeps for the backward
        o, lse = _plain_attention(st)
        st["o"], st["lse"] = o, lse
        st["go"] = [gen.randn(b, c["q_tokens"], n, d) for n in qn]
    if own:
        from ulysses_sequence_all_gb300 import binding as B
        even = lambda n: _share(n, W, False)
        st["q_plan"] = B.ulysses_plan(W, b, even(c["q_tokens"]), qn, d, c["dtype"])
        st["kv_plan"] = B.ulysses_plan(W, b, even(c["kv_tokens"]), kn, d, c["dtype"])
        if c["op"] == "attention":
            st["out"] = [torch.empty_like(x) for x in st["q"]]
            st["out_lse"] = [torch.empty(b, n, c["q_tokens"], device="cuda") for n in qn]
            need = B.ulysses_attention_workspace(st["q_plan"], st["kv_plan"])
        else:
            st["grads"] = [[torch.empty_like(x) for x in st[t]] for t in "qkv"]
            need = B.ulysses_attention_backward_workspace(st["q_plan"], st["kv_plan"])
        st["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    return st


# ---- one pass -----------------------------------------------------------------------------------

def run(state):
    c = state["case"]
    if own:
        return _run_own(state, c)
    if c["op"] == "rope":
        return _plain_rope(state)
    if c["op"] == "rope_backward":
        return _plain_rope_backward(state)
    if c["op"] == "attention":
        return list(_plain_attention(state))
    return _plain_attention_backward(state)


def _run_own(st, c):
    from ulysses_sequence_all_gb300 import binding as B
    if c["op"] == "rope":
        q, k = st["out"]
        B.ulysses_a2a_4d_qk_fused(st["plan"], st["q"], st["k"], q, k, st["w"], EPS, THETA)
        return [q, k]
    if c["op"] == "rope_backward":
        dq, dk = st["out"]
        B.ulysses_a2a_4d_qk_fused_backward(st["plan"], dq, dk, st["q"], st["k"], st["gq"], st["gk"],
                                           st["w"], st["dw"], EPS, THETA, st["ws"])
        return [dq, dk, st["dw"]]
    if c["op"] == "attention":
        B.ulysses_attention(st["q_plan"], st["kv_plan"], st["q"], st["k"], st["v"], st["out"],
                            st["out_lse"], scale=st["scale"], causal=c["causal"],
                            kv_lens=st["kv_lens"], q_start=st["q_start"], workspace=st["ws"])
        return [st["out"], st["out_lse"]]
    dq, dk, dv = st["grads"]
    B.ulysses_attention_backward(st["q_plan"], st["kv_plan"], dq, dk, dv, st["q"], st["k"], st["v"],
                                 st["o"], st["lse"], st["go"], scale=st["scale"],
                                 causal=c["causal"], kv_lens=st["kv_lens"], q_start=st["q_start"],
                                 workspace=st["ws"])
    return [dq, dk, dv]


# ---- plain forms --------------------------------------------------------------------------------

def _plain_angles(c, lo, hi):
    """cos and sin (tokens lo .. hi - 1 of the sequence, d/2 pairs), angles formed in 64 bits."""
    extents, pairs = _grid(c)
    p = torch.arange(lo, hi, device="cuda") - c["prefix"]
    inside = (p >= 0) & (p < math.prod(extents))
    stride = math.prod(extents)
    cols = []
    for ext, m in zip(extents, pairs):
        stride //= ext
        coord = torch.where(inside, (p // stride) % ext, 0).double()
        freq = THETA ** (-torch.arange(m, device="cuda", dtype=torch.float64) / m)
        cols.append(coord[:, None] * freq)
    ang = torch.cat(cols, 1)
    return ang.cos().float()[:, None, :], ang.sin().float()[:, None, :]


def _split(x, half):
    d = x.shape[-1]
    return (x[..., :d // 2], x[..., d // 2:]) if half else (x[..., 0::2], x[..., 1::2])


def _join(a, b, half):
    return torch.cat((a, b), -1) if half else torch.stack((a, b), -1).flatten(-2)


def _plain_rope(st):
    c = st["case"]
    seq, heads = _rope_splits(c)
    out = []
    for which, xs in enumerate((st["q"], st["k"])):
        rows, off = [], 0
        for x, s in zip(xs, seq):
            cos, sin = _plain_angles(c, off, off + s)
            y = x.float()
            y = y * torch.rsqrt(y.pow(2).mean(-1, keepdim=True) + EPS) * st["w"][which]
            a, b = _split(y, c["half_pairs"])
            y = _join(a * cos - b * sin, a * sin + b * cos, c["half_pairs"]).to(x.dtype)
            rows.append(torch.split(y, heads, dim=2))
            off += s
        out.append([torch.cat([r[k] for r in rows], dim=1) for k in range(c["W"])])
    return out


def _plain_rope_backward(st):
    c = st["case"]
    seq, heads = _rope_splits(c)
    out, dw = [], []
    for which, (xs, gs) in enumerate(((st["q"], st["gq"]), (st["k"], st["gk"]))):
        w, off, dxs = st["w"][which], 0, []
        total = torch.zeros(c["d"], dtype=torch.float64, device="cuda")
        for x, s in zip(xs, seq):
            cos, sin = _plain_angles(c, off, off + s)
            g = torch.cat([t[:, off:off + s] for t in gs], dim=2).float()
            a, b = _split(g, c["half_pairs"])
            u = _join(a * cos + b * sin, b * cos - a * sin, c["half_pairs"])
            y = x.float()
            r = torch.rsqrt(y.pow(2).mean(-1, keepdim=True) + EPS)
            y = y * r
            total += (u * y).sum(dim=(0, 1, 2), dtype=torch.float64)
            u = u * w
            dxs.append((r * (u - y * (u * y).mean(-1, keepdim=True))).to(x.dtype))
            off += s
        out.append(dxs)
        dw.append(total.float())
    return [out[0], out[1], torch.stack(dw)]


def _visible(st):
    """(b, q_tokens, 1): the number of keys each query row sees."""
    c = st["case"]
    n = torch.tensor(_lens(c), device="cuda")[:, None]
    if c["causal"]:
        i = torch.arange(c["q_tokens"], device="cuda")[None]
        s = torch.tensor(_starts(c), device="cuda")[:, None]
        n = torch.minimum(n, (s + i + 1).clamp(min=0))
    else:
        n = n.expand(c["b"], c["q_tokens"])
    return n[..., None]


def _row_chunk(c, n):
    """Query tokens at a time, so that a block of scores stays near 2 GiB."""
    return max(1, min(c["q_tokens"], 2 ** 29 // max(1, n * c["kv_tokens"])))


def _plain_attention(st):
    c = st["case"]
    vis = _visible(st)
    cols = torch.arange(c["kv_tokens"], device="cuda")
    outs, lses = [], []
    for q, k, v in zip(st["q"], st["k"], st["v"]):
        nk = k.shape[2]
        g = q.shape[2] // nk
        o = torch.empty_like(q)
        lse = torch.empty((c["b"], q.shape[2], c["q_tokens"]), device="cuda")
        step = _row_chunk(c, q.shape[2])
        for bb in range(c["b"]):
            kt = k[bb].float().permute(1, 2, 0)                      # (nk, d, keys)
            vt = v[bb].float().permute(1, 0, 2)                      # (nk, keys, d)
            for i in range(0, c["q_tokens"], step):
                t = q[bb, i:i + step].float()                        # (rows, nk * g, d)
                r = t.shape[0]
                t = t.view(r, nk, g, -1).permute(1, 2, 0, 3).reshape(nk, g * r, -1)
                s = torch.matmul(t, kt).view(nk, g, r, -1) * st["scale"]
                s.masked_fill_(cols >= vis[bb, i:i + step], -math.inf)
                m = s.amax(-1, keepdim=True)
                m = torch.where(m == -math.inf, 0.0, m)
                p = s.sub_(m).exp_()
                l = p.sum(-1, keepdim=True)
                x = torch.matmul(p.view(nk, g * r, -1), vt).view(nk, g, r, -1)
                x = x / torch.where(l == 0, 1.0, l)
                o[bb, i:i + step] = x.permute(2, 0, 1, 3).reshape(r, nk * g, -1).to(q.dtype)
                lse[bb, :, i:i + step] = (m + l.log()).squeeze(-1).view(nk * g, r)
        outs.append(o)
        lses.append(lse)
    return outs, lses


def _plain_attention_backward(st):
    c = st["case"]
    vis = _visible(st)
    cols = torch.arange(c["kv_tokens"], device="cuda")
    dqs, dks, dvs = [], [], []
    for q, k, v, o, lse, go in zip(st["q"], st["k"], st["v"], st["o"], st["lse"], st["go"]):
        nk = k.shape[2]
        g = q.shape[2] // nk
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        step = max(1, _row_chunk(c, q.shape[2]) // 2)
        for bb in range(c["b"]):
            kt, vt = k[bb].float().permute(1, 0, 2), v[bb].float().permute(1, 0, 2)
            ak, av = torch.zeros_like(kt), torch.zeros_like(vt)

            def rows(x, i):
                t = x[bb, i:i + step].float()
                return t.view(t.shape[0], nk, g, -1).permute(1, 2, 0, 3).reshape(nk, g * t.shape[0], -1)

            for i in range(0, c["q_tokens"], step):
                tq, to, tg = rows(q, i), rows(o, i), rows(go, i)
                r = tq.shape[1] // g
                z = lse[bb, :, i:i + step].reshape(nk, g, r, 1)
                s = torch.matmul(tq, kt.transpose(1, 2)).view(nk, g, r, -1) * st["scale"]
                hide = cols >= vis[bb, i:i + step]
                p = s.sub_(torch.where(z == -math.inf, 0.0, z)).exp_().masked_fill_(hide, 0.0)
                p = p.view(nk, g * r, -1)
                dp = torch.matmul(tg, vt.transpose(1, 2)).sub_((tg * to).sum(-1, keepdim=True))
                ds = dp.mul_(p)
                av += torch.matmul(p.transpose(1, 2), tg)
                ak += torch.matmul(ds.transpose(1, 2), tq)
                x = torch.matmul(ds, kt) * st["scale"]
                dq[bb, i:i + step] = (x.view(nk, g, r, -1).permute(2, 0, 1, 3)
                                      .reshape(r, nk * g, -1).to(q.dtype))
            dk[bb] = (ak * st["scale"]).permute(1, 0, 2).to(k.dtype)
            dv[bb] = av.permute(1, 0, 2).to(v.dtype)
        dqs.append(dq)
        dks.append(dk)
        dvs.append(dv)
    return [dqs, dks, dvs]


# ---- the definition in 64 bits ------------------------------------------------------------------

def exact(case, seed):
    c = case
    if c["op"].startswith("attention"):
        factor = 4 if c["op"] == "attention" else 10
        # about 0.8e12 multiply-adds a second in 64 bits, several passes over the scores
        if factor * float(c["b"]) * c["q_tokens"] * c["kv_tokens"] * c["heads"] * c["d"] > 8e12:
            return None
        st = prepare(case, seed)
        return _exact_attention(st) if c["op"] == "attention" else _exact_attention_backward(st)
    st = prepare(case, seed)
    return _exact_rope(st) if c["op"] == "rope" else _exact_rope_backward(st)


def _exact_turn(c, p0, s):
    """The unit complex numbers that rotate tokens p0 .. p0 + s - 1, one per rotary pair."""
    extents, pairs = _grid(c)
    inner = math.prod(extents)
    p = torch.arange(p0, p0 + s, device="cuda", dtype=torch.int64) - c["prefix"]
    on_grid = ((p >= 0) & (p < inner)).to(torch.float64)
    turn = torch.empty((s, c["d"] // 2), dtype=torch.float64, device="cuda")
    col = 0
    for ext, m in zip(extents, pairs):
        inner //= ext
        x = torch.remainder(torch.div(p, inner, rounding_mode="floor"), ext).to(torch.float64)
        for i in range(m):
            turn[:, col] = x * on_grid * math.exp(-math.log(THETA) * i / m)
            col += 1
    return torch.polar(torch.ones_like(turn), turn)


def _exact_complex(x, half):
    if half:
        n = x.shape[-1] // 2
        return torch.complex(x[..., :n].contiguous(), x[..., n:].contiguous())
    return torch.view_as_complex(x.unflatten(-1, (-1, 2)).contiguous())


def _exact_real(z, half):
    return torch.cat((z.real, z.imag), -1) if half else torch.view_as_real(z).flatten(-2)


def _exact_rope(st):
    c = st["case"]
    seq, heads = _rope_splits(c)
    res = []
    for xs, w in zip((st["q"], st["k"]), st["w"].double()):
        outs = [torch.empty((c["b"], _tokens(c), n, c["d"]), dtype=torch.float64, device="cuda")
                for n in heads]
        at = 0
        for x, s in zip(xs, seq):
            h0 = 0
            for o, n in zip(outs, heads):
                y = x[:, :, h0:h0 + n].double()
                y = y / (y.square().sum(-1, keepdim=True) / c["d"] + EPS).sqrt() * w
                z = _exact_complex(y, c["half_pairs"]) * _exact_turn(c, at, s)[:, None, :]
                o[:, at:at + s] = _exact_real(z, c["half_pairs"])
                h0 += n
            at += s
        res.append(outs)
    return res


def _exact_rope_backward(st):
    c = st["case"]
    seq, heads = _rope_splits(c)
    res, dws = [], []
    for xs, gs, w in zip((st["q"], st["k"]), (st["gq"], st["gk"]), st["w"].double()):
        dw = torch.zeros(c["d"], dtype=torch.float64, device="cuda")
        dxs, at = [], 0
        for x, s in zip(xs, seq):
            dx = torch.empty(x.shape, dtype=torch.float64, device="cuda")
            h0 = 0
            for g, n in zip(gs, heads):
                turn = _exact_turn(c, at, s)[:, None, :].conj()
                u = _exact_real(_exact_complex(g[:, at:at + s].double(), c["half_pairs"]) * turn,
                                c["half_pairs"])
                y = x[:, :, h0:h0 + n].double()
                rms = (y.square().sum(-1, keepdim=True) / c["d"] + EPS).sqrt()
                dw += torch.einsum("bsnd,bsnd->d", u, y / rms)
                uw = u * w
                dot = torch.einsum("bsnd,bsnd->bsn", uw, y)[..., None]
                dx[:, :, h0:h0 + n] = uw / rms - y * dot / (c["d"] * rms ** 3)
                h0 += n
            dxs.append(dx)
            at += s
        res.append(dxs)
        dws.append(dw)
    return [res[0], res[1], torch.stack(dws)]


def _exact_scores(st, q, k, bb, h, g):
    """Scaled scores of one head, minus infinity where the key is not visible."""
    c = st["case"]
    s = torch.einsum("id,jd->ij", q[bb, :, h].double(), k[bb, :, h // g].double()) * st["scale"]
    j = torch.arange(c["kv_tokens"], device="cuda")[None, :]
    hidden = j >= _lens(c)[bb]
    if c["causal"]:
        i = torch.arange(c["q_tokens"], device="cuda")[:, None]
        hidden = hidden | (j > i + _starts(c)[bb])
    return torch.where(hidden, -math.inf, s)


def _exact_attention(st):
    outs, lses = [], []
    for q, k, v in zip(st["q"], st["k"], st["v"]):
        g = q.shape[2] // k.shape[2]
        o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
        lse = torch.empty((q.shape[0], q.shape[2], q.shape[1]), dtype=torch.float64, device="cuda")
        for bb in range(q.shape[0]):
            for h in range(q.shape[2]):
                s = _exact_scores(st, q, k, bb, h, g)
                z = torch.logsumexp(s, dim=1)
                lse[bb, h] = z
                e = torch.exp(s - z[:, None])
                e[z == -math.inf] = 0.0
                o[bb, :, h] = e @ v[bb, :, h // g].double()
        outs.append(o)
        lses.append(lse)
    return [outs, lses]


def _exact_attention_backward(st):
    res = [[], [], []]
    for q, k, v, o, lse, go in zip(st["q"], st["k"], st["v"], st["o"], st["lse"], st["go"]):
        g = q.shape[2] // k.shape[2]
        dq, dk, dv = (torch.zeros(x.shape, dtype=torch.float64, device="cuda") for x in (q, k, v))
        for bb in range(q.shape[0]):
            for h in range(q.shape[2]):
                z = lse[bb, h].double()[:, None]
                e = torch.exp(_exact_scores(st, q, k, bb, h, g) - z)
                e[(z == -math.inf).squeeze(1)] = 0.0
                d_out = go[bb, :, h].double()
                dv[bb, :, h // g] += e.T @ d_out
                mean = torch.einsum("id,id->i", d_out, o[bb, :, h].double())
                e *= d_out @ v[bb, :, h // g].double().T - mean[:, None]
                dq[bb, :, h] = st["scale"] * (e @ k[bb, :, h // g].double())
                dk[bb, :, h // g] += st["scale"] * (e.T @ q[bb, :, h].double())
        for acc, x in zip(res, (dq, dk, dv)):
            acc.append(x)
    return res
