"""Attention with a sliding window and first tokens that stay visible, and its gradient, from the
definition in 64 bits, with the sums that the tolerances of its tests are made of; and a paged cache
built from contiguous keys."""
import math

import torch


def visible(b, sq, skv, window=0, sinks=0, kv_lens=None, q_start=None, device="cuda"):
    """(b, sq, skv): whether the query at position p = q_start + i sees key j: j < kv_lens, j <= p and
    j > p - window or j < sinks (window 0: every earlier key). kv_lens, q_start: lists of b or None."""
    j = torch.arange(skv, device=device)[None, None, :]
    n = torch.tensor([skv] * b if kv_lens is None else list(kv_lens), device=device)[:, None, None]
    s = torch.tensor([0] * b if q_start is None else list(q_start), device=device)[:, None, None]
    p = s + torch.arange(sq, device=device)[None, :, None]
    near = (j > p - window) if window else torch.ones_like(j, dtype=torch.bool)
    return (j < n) & (j <= p) & (near | (j < sinks))


def clean(x, see):
    """Keys or values with everything that no row sees zeroed."""
    return torch.where(see.any(1)[:, :, None, None], x, torch.zeros_like(x))


def _probabilities(q, k, h, bb, g, scale, see):
    s = (q[bb, :, h].double() @ k[bb, :, h // g].double().T) * scale
    s = torch.where(see, s, -math.inf)
    z = torch.logsumexp(s, -1)
    p = torch.where(see, torch.exp(s - torch.where(z == -math.inf, 0.0, z)[:, None]), 0.0)
    return p, z


def forward(q, k, v, scale, see):
    """(o, lse, mean |v| under the probabilities) of one rank."""
    b, sq, n, d = q.shape
    g = n // max(1, k.shape[2])
    k, v = clean(k, see), clean(v, see)
    o = torch.empty(b, sq, n, d, dtype=torch.float64, device=q.device)
    a = torch.empty_like(o)
    lse = torch.empty(b, n, sq, dtype=torch.float64, device=q.device)
    for bb in range(b):
        for h in range(n):
            p, z = _probabilities(q, k, h, bb, g, scale, see[bb])
            vv = v[bb, :, h // g].double()
            o[bb, :, h], a[bb, :, h], lse[bb, h] = p @ vv, p @ vv.abs(), z
    return o, lse, a


def backward(q, k, v, o, lse, go, scale, see):
    """(dq, dk, dv) of one rank from the formulas, with the given o and lse, and two sums of magnitudes
    for each that bound its rounding: of the factors rounded to the element type (P for dv, dS for dq and
    dk) times |go|, |k|, |q|; and of all that fp32 sums up on the way (each dS is a difference)."""
    g = q.shape[2] // max(1, k.shape[2])
    k, v = clean(k, see), clean(v, see)
    some = see.any(2)[:, :, None, None]
    q, go = (torch.where(some, x, torch.zeros_like(x)) for x in (q, go))
    new = lambda: [torch.zeros(x.shape, dtype=torch.float64, device=q.device) for x in (q, k, v)]
    (dq, dk, dv), (aq, ak, av), (mq, mk, mv) = new(), new(), new()
    for bb in range(q.shape[0]):
        for h in range(q.shape[2]):
            kk, vv, qq = k[bb, :, h // g].double(), v[bb, :, h // g].double(), q[bb, :, h].double()
            gg, oo, z = go[bb, :, h].double(), o[bb, :, h].double(), lse[bb, h].double()
            p = torch.exp(qq @ kk.T * scale - torch.where(z == -math.inf, 0.0, z)[:, None])
            p = torch.where(see[bb] & (z != -math.inf)[:, None], p, 0.0)
            ds = p * (gg @ vv.T - (gg * oo).sum(-1, keepdim=True))
            mag = p * (gg.abs() @ vv.abs().T + (gg.abs() * oo.abs()).sum(-1, keepdim=True))
            dv[bb, :, h // g] += p.T @ gg
            av[bb, :, h // g] += p.T @ gg.abs()
            dq[bb, :, h] = scale * ds @ kk
            aq[bb, :, h] = scale * ds.abs() @ kk.abs()
            mq[bb, :, h] = scale * mag @ kk.abs()
            dk[bb, :, h // g] += scale * ds.T @ qq
            ak[bb, :, h // g] += scale * ds.abs().T @ qq.abs()
            mk[bb, :, h // g] += scale * mag.T @ qq.abs()
    return (dq, dk, dv), (aq, ak, av), (mq, mk, av)


def paged(x, lens, page, table, pages, fill):
    """A pool (pages, page, m, d) that holds x's tokens (b, S, m, d), lens of them, where the table
    (a CPU tensor) says; every other row is `fill`."""
    pool = torch.full((pages, page) + x.shape[2:], fill, dtype=x.dtype, device=x.device)
    for bb, n in enumerate(lens):
        for p in range((max(0, n) + page - 1) // page):
            at = int(table[bb, p])
            if 0 <= at < pages:
                rows = x[bb, p * page:min(n, (p + 1) * page)]
                pool[at, :len(rows)] = rows
    return pool
