"""The differentiable forms of attention with a window: against the formulas in 64 bits, and the
sequence-parallel block that uses them (packed QKV, norm, rotation, both relayouts) against the same block
written out. The blocks differ in rounding only (bf16 between the steps, the order of the sums), so they agree
to about 1e-2 of the largest value; a wrong mask, head or position gives errors of order 1."""
import math

import pytest
import torch

import window_reference as R
from test_gpu_attention_window import Case
from ulysses_sequence_all_gb300 import autograd as A
from ulysses_sequence_all_gb300 import binding as B
from ulysses_sequence_all_gb300.attention_block import attention_block

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    B.library()
    yield
    assert B.ulysses_device_status() == 0


@pytest.mark.parametrize("shape, lens", [((2, 2, 300, 300, [1, 2], 2, 64), [300, 123]),
                                         ((1, 1, 500, 500, [2], 1, 128), None),
                                         ((1, 3, 5, 400, [1], 4, 72), [400, 9, 0])])
def test_autograd(shape, lens):
    sq, skv = shape[2], shape[3]
    start = None if sq == skv else [n - sq for n in lens]
    c = Case(*shape, 70, 3, kv_lens=lens, q_start=start, fill=0.0)
    leaves = [[x.clone().requires_grad_() for x in t] for t in (c.q, c.k, c.v)]
    o = A.attention(c.qp, c.kp, *leaves, kv_lens=lens, q_start=start, window=70, sinks=3)
    torch.autograd.backward(o, c.go)
    lse = c.forward()[1]
    o = [x.detach() for x in o]
    c.check(o, lse)
    c.check_backward(o, lse, [[x.grad for x in t] for t in leaves])


def plain_block(qkv, w, window, sinks, eps=1e-6, theta=1e4):
    """(b, S, 3, N, d) -> (b, S, N, d), in the input's precision."""
    b, S, _, N, d = qkv.shape
    ang = torch.arange(S, device="cuda").double()[:, None] * theta ** (
        -2.0 * torch.arange(d // 2, device="cuda").double() / d)
    cos, sin = ang.cos()[:, None], ang.sin()[:, None]

    def turned(x, w):
        x = x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + eps) * w
        e, o = x[..., 0::2], x[..., 1::2]
        return torch.stack((e * cos - o * sin, e * sin + o * cos), -1).flatten(-2)
    q, k, v = turned(qkv[:, :, 0], w[0]), turned(qkv[:, :, 1], w[1]), qkv[:, :, 2]
    s = torch.einsum("bind,bjnd->bnij", q, k) * d ** -0.5
    s = s.masked_fill(~R.visible(b, S, S, window, sinks)[:, None], -math.inf)
    return torch.einsum("bnij,bjnd->bind", s.softmax(-1), v)


@pytest.mark.parametrize("window, sinks", [(40, 4), (1, 0), (1000, 0)])
def test_block(window, sinks):
    seq, heads, b, d = [70, 90, 0, 96], [2, 1, 1, 2], 2, 64
    plan = B.ulysses_plan(4, b, seq, heads, d, "bfloat16")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")
    x = rnd(b, sum(seq), 3, sum(heads), d).bfloat16()
    w, go = 1 + 0.1 * rnd(2, d), rnd(b, sum(seq), sum(heads), d).bfloat16()
    shards = [t.clone().requires_grad_() for t in x.split(seq, 1)]
    wl = w.clone().requires_grad_()
    out = attention_block(plan, shards, wl, window=window, sinks=sinks)
    torch.autograd.backward(out, [t.contiguous() for t in go.split(seq, 1)])
    xd, wd = x.double().requires_grad_(), w.double().requires_grad_()
    want = plain_block(xd, wd, window, sinks)
    want.backward(go.double())
    # A row that sees one key (a window of 1) has P = 1 and dS = go . v - go . o = 0. Both are fp32 sums of 64
    # products, 41 of magnitude together, so dS comes out as 2^-22 * 41 at most, and the norm weights' gradient
    # as that times scale * |k| (1/8) over 2 * 256 * 6 rows: 3.8e-3 in place of the 0 that is exact.
    near_zero = 2 * sum(seq) * sum(heads) / 8 * 41 * 2.0 ** -22
    for got, ref, least in ((torch.cat(out, 1), want, 0.0),
                            (torch.cat([t.grad for t in shards], 1), xd.grad, 0.0),
                            (wl.grad, wd.grad, near_zero)):
        assert float((got.double() - ref).detach().abs().max()) < 2e-2 * float(ref.detach().abs().max()) + least


def test_prompt_with_a_window_then_tokens_over_the_pages():
    """A prompt attends with a window and is appended to the pages; new tokens are appended and attend with
    the same window; pages that no later token sees are given back on the way. Against the definition over the
    whole sequence, each output rounded once and each probability once."""
    W, b, S, new, heads, g, d, page, window, sinks = 2, 2, 200, 40, [1, 2], 2, 64, 16, 50, 3
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    rnd = lambda n, m: torch.randn((b, n, m, d), generator=gen, device="cuda").bfloat16()
    T = S + new
    q, k, v = [rnd(T, g * m) for m in heads], [rnd(T, m) for m in heads], [rnd(T, m) for m in heads]
    plan = lambda n, hs, batch=b: B.ulysses_plan(W, batch, [n, 0], hs, d, "bfloat16")
    want = [R.forward(x, y, z, d ** -0.5, R.visible(b, T, T, window, sinks)) for x, y, z in zip(q, k, v)]

    def check(out, rows):
        for o, (x, _, a) in zip(out, want):
            err = (o.double() - x[:, rows]).abs()
            assert not (err > 2.0 ** -8 * x[:, rows].abs() + (2.0 ** -8 + 1e-4) * a[:, rows]).any()
    part = lambda xs, rows: [x[:, rows].contiguous() for x in xs]
    rows = slice(0, S)
    check(A.attention(plan(S, [g * m for m in heads]), plan(S, heads), part(q, rows), part(k, rows),
                      part(v, rows), window=window, sinks=sinks), rows)
    per = -(-T // page)
    pages = b * per
    table = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32).view(b, per)
    pools = [[torch.full((pages, page, m, d), math.nan, device="cuda").bfloat16() for m in heads]
             for _ in range(2)]
    cp = plan(page, heads, pages)
    i32 = lambda n: torch.full((b,), n, dtype=torch.int32, device="cuda")
    B.ulysses_cache_append(plan(S, heads), cp, part(k, rows), part(v, rows), *pools, table, i32(0))
    qp, kp = plan(1, [g * m for m in heads]), plan(1, heads)
    ws = torch.empty(B.ulysses_attention_paged_workspace(qp, cp), dtype=torch.uint8, device="cuda")
    for at in range(S, T):
        rows = slice(at, at + 1)
        B.ulysses_cache_append(kp, cp, part(k, rows), part(v, rows), *pools, table, i32(at))
        for p in range(1, (at + 1 - window) // page):  # (page 0 holds the first tokens)
            if int(table[0, p]) >= 0:
                for pool in pools[0] + pools[1]:
                    pool[table[:, p].long()] = math.nan
                table[:, p] = -1
        out = [torch.empty_like(x) for x in part(q, rows)]
        lse = [torch.empty(b, g * m, 1, device="cuda") for m in heads]
        B.ulysses_attention_paged(qp, cp, part(q, rows), *pools, out, lse, table, i32(at + 1), scale=d ** -0.5,
                                  window=window, sinks=sinks, workspace=ws)
        check(out, rows)
