"""Attention and its gradient from the definition, in 64 bits, one head at a time, with the sums that
the tolerances of the attention tests are made of."""
import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def visible(b, sq, skv, causal, kv_lens, q_start, device):
    """(b, sq, skv): whether the query sees the key."""
    j = torch.arange(skv, device=device)[None, None, :]
    i = torch.arange(sq, device=device)[None, :, None]
    n = torch.full((b,), skv, device=device) if kv_lens is None else kv_lens.clamp(0, skv)
    see = (j < n[:, None, None]).expand(b, sq, skv)
    if causal:
        s = torch.zeros(b, dtype=torch.int64, device=device) if q_start is None else q_start
        see = see & (j <= i + s[:, None, None])
    return see


def probabilities(q, k, h, bb, g, scale, see):
    s = (q[bb, :, h].double() @ k[bb, :, h // g].double().T) * scale
    s = torch.where(see, s, -math.inf)
    z = torch.logsumexp(s, -1)
    p = torch.where(see, torch.exp(s - torch.where(z == -math.inf, 0.0, z)[:, None]), 0.0)
    return p, z


def clean(x, kv_lens):
    """Keys or values with everything past the batch element's length zeroed."""
    if kv_lens is None:
        return x
    j = torch.arange(x.shape[1], device=x.device)[None, :, None, None]
    return torch.where(j < kv_lens[:, None, None, None], x, torch.zeros_like(x))


def forward(q, k, v, scale, causal=False, kv_lens=None, q_start=None):
    """(o, lse, mean |v| under the probabilities) of one rank."""
    b, sq, n, d = q.shape
    k, v = clean(k, kv_lens), clean(v, kv_lens)
    g = n // max(1, k.shape[2])
    see = visible(b, sq, k.shape[1], causal, kv_lens, q_start, q.device)
    o = torch.empty(b, sq, n, d, dtype=torch.float64, device=q.device)
    a = torch.empty_like(o)
    lse = torch.empty(b, n, sq, dtype=torch.float64, device=q.device)
    for bb in range(b):
        for h in range(n):
            p, z = probabilities(q, k, h, bb, g, scale, see[bb])
            vv = v[bb, :, h // g].double()
            o[bb, :, h], a[bb, :, h], lse[bb, h] = p @ vv, p @ vv.abs(), z
    return o, lse, a


def backward(q, k, v, o, lse, go, scale, causal=False, kv_lens=None, q_start=None):
    """(dq, dk, dv) of one rank from the formulas, with the given o and lse, and two sums of
    magnitudes for each that bound its rounding: of the factors rounded to the element type (P for
    dv, dS for dq and dk) times |go|, |k|, |q|; and of all that fp32 sums up on the way (for dS,
    P (|go| |v|^T + sum |go| |o|): each dS is a difference)."""
    b, sq, n, d = q.shape
    k, v = clean(k, kv_lens), clean(v, kv_lens)
    g = n // max(1, k.shape[2])
    see = visible(b, sq, k.shape[1], causal, kv_lens, q_start, q.device)
    new = lambda: [torch.zeros(x.shape, dtype=torch.float64, device=q.device) for x in (q, k, v)]
    (dq, dk, dv), (aq, ak, av), (mq, mk, mv) = new(), new(), new()
    for bb in range(b):
        for h in range(n):
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
