"""Position axes of the fused calls (ulysses_plan_set_rope_grid): the fused forward, its packed form
and the backward against the definition in 64 bits.

Tolerances: a result is an fp32 value rounded once to the element type, so off by half a step of it
(bf16 2^-8, fp16 2^-11 relative) plus the fp32 arithmetic: about ten roundings of 2^-24 on values
of at most 6 sigma, 1e-5, and for the backward's cancelling terms 1e-4; the angle's error, 1e-6 rad on
values of at most 6 sigma, is inside those. dw sums n products of unit scale in fp32: each lane's
partial sums carry 2^-24 of their size, a random walk of n steps, well inside 1e-4 sqrt(n)."""
import math

import pytest
import torch

from ulysses_sequence_all_gb300 import autograd as A
from ulysses_sequence_all_gb300 import binding as B

pytestmark = pytest.mark.gpu

EPS, THETA = 1e-6, 1e4
HALF_STEP = {"bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    B.library()
    yield
    assert B.ulysses_device_status() == 0, "a kernel recorded a wait timeout"


def turns(S, d, extents, pairs, first):
    """Angles (S, d/2) in 64 bits, token by token from the definition."""
    total = math.prod(extents)
    ang = torch.zeros(S, d // 2, dtype=torch.float64, device="cuda")
    p = torch.arange(S, device="cuda") - first
    on = (p >= 0) & (p < total)
    col, inner = 0, total
    for ext, m in zip(extents, pairs):
        inner //= ext
        coord = ((p // inner) % ext).double() * on
        for i in range(m):
            ang[:, col] = coord * THETA ** (-i / m)
            col += 1
    return ang


def rotate(x, ang, half):
    d = x.shape[-1]
    a, b = (x[..., :d // 2], x[..., d // 2:]) if half else (x[..., 0::2], x[..., 1::2])
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    y = (a * c - b * s, a * s + b * c)
    return torch.cat(y, -1) if half else torch.stack(y, -1).flatten(-2)


def norm(x, w):
    x = x.double()
    return x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double()


CASES = [
    # W, b, seq, heads, d, extents, pairs, first
    (2, 1, [16, 16], [4, 4], 128, (2, 4, 4), (22, 21, 21), 0),
    (3, 2, [70, 61, 90], [3, 2, 2], 64, (13, 16), (16, 16), 5),          # text on both sides
    (2, 1, [0, 105], [2, 2], 128, (3, 5, 7), (0, 32, 32), 0),            # an axis that turns nothing
    (1, 2, [77], [3], 72, (7, 11), (10, 10), 0),                         # pairs left unturned
    (4, 1, [150, 151, 149, 150], [2, 2, 2, 2], 128, (2, 3, 4, 25), (16, 16, 16, 16), 0),
    (2, 1, [1, 0], [1, 1], 64, (1,), (32,), 0),                          # one token
    (2, 1, [100, 90], [5, 3], 96, (10, 3, 6), (16, 16, 16), 10),
    (1, 1, [40], [2], 256, (5, 8), (64, 64), 0),
    (1, 1, [33], [1], 8, (3, 11), (2, 2), 0),
]


def make(c, dtype, half, seed=0):
    W, b, seq, heads, d, extents, pairs, first = c
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    N, S = sum(heads), sum(seq)
    dt = getattr(torch, dtype)
    rnd = lambda *sh: torch.randn(sh, generator=g, device="cuda").to(dt)
    q, k = ([rnd(b, s, N, d) for s in seq] for _ in range(2))
    gq, gk = ([rnd(b, S, n, d) for n in heads] for _ in range(2))
    w = 1.0 + 0.1 * torch.randn((2, d), generator=g, device="cuda")
    plan = B.ulysses_plan(W, b, seq, heads, d, dtype)
    B.ulysses_plan_set_rope_pairs(plan, B.ULY_ROPE_HALF if half else B.ULY_ROPE_ADJACENT)
    B.ulysses_plan_set_rope_grid(plan, extents, pairs, first)
    return plan, q, k, gq, gk, w


def close(got, want, dtype, atol):
    want = want.double()
    bad = (got.double() - want).abs() > HALF_STEP[dtype] * want.abs() + atol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off"


def engines(plan):
    fits = len(set(plan.head_splits)) == 1
    return [B.ULY_ENGINE_TMA] + ([B.ULY_ENGINE_TENSOR] if fits else [])


@pytest.mark.parametrize("half", [False, True], ids=["adjacent", "half"])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("c", CASES, ids=[f"W{c[0]}d{c[4]}g{'x'.join(map(str, c[5]))}" for c in CASES])
def test_forward_and_backward(c, dtype, half):
    W, b, seq, heads, d, extents, pairs, first = c
    plan, q, k, gq, gk, w = make(c, dtype, half)
    S, N = sum(seq), sum(heads)
    ang = turns(S, d, extents, pairs, first)
    for engine in engines(plan):
        B.ulysses_plan_set_fused_engine(plan, engine)
        qo, ko = ([torch.full((b, S, n, d), 7.0, dtype=q[0].dtype, device="cuda") for n in heads]
                  for _ in range(2))
        B.ulysses_a2a_4d_qk_fused(plan, q, k, qo, ko, w, EPS, THETA)
        dq, dk = ([torch.full_like(x, 7.0) for x in q] for _ in range(2))
        dw = torch.full_like(w, 7.0)
        ws = torch.empty(B.ulysses_qk_fused_backward_workspace(plan), dtype=torch.uint8,
                         device="cuda")
        B.ulysses_a2a_4d_qk_fused_backward(plan, dq, dk, q, k, gq, gk, w, dw, EPS, THETA, ws)
        for t, (xs, ys, gs, dxs) in enumerate(((q, qo, gq, dq), (k, ko, gk, dk))):
            x = torch.cat(xs, 1)
            want = rotate(norm(x, w[t]), ang, half)
            close(torch.cat(ys, 2), want, dtype, 1e-5)
            leaf, wl = x.double().requires_grad_(), w[t].double().requires_grad_()
            y = leaf / (leaf.square().mean(-1, keepdim=True) + EPS).sqrt() * wl
            y = rotate(y, ang, half)
            y.backward(torch.cat(gs, 2).double())
            close(torch.cat(dxs, 1), leaf.grad, dtype, 1e-4)
            n = b * S * N
            err = (dw[t].double() - wl.grad).abs().max().item()
            assert err <= 1e-4 * math.sqrt(n) + 1e-4, err


def test_one_axis_is_the_sequence_index():
    """A grid of one axis with every pair is the default, byte for byte; and the default returns."""
    c = (2, 2, [40, 30], [3, 3], 128, (70,), (64,), 0)
    plan, q, k, gq, gk, w = make(c, "bfloat16", False)
    outs = []
    for extents, pairs in (((70,), (64,)), ((), ())):
        B.ulysses_plan_set_rope_grid(plan, extents, pairs)
        qo, ko = ([torch.empty(2, 70, 3, 128, dtype=torch.bfloat16, device="cuda")
                   for _ in range(2)] for _ in range(2))
        B.ulysses_a2a_4d_qk_fused(plan, q, k, qo, ko, w, EPS, THETA)
        outs.append(qo + ko)
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_long_grid_coordinates():
    """Close to the longest sequence (2^24 - 1): every coordinate of a large odd grid is exact."""
    ext, d = (255, 257, 253), 16
    S = math.prod(ext) + 3
    plan = B.ulysses_plan(1, 1, [S], [1], d, "bfloat16")
    B.ulysses_plan_set_rope_grid(plan, ext, (2, 3, 3), first=2)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.randn((1, S, 1, d), generator=g, device="cuda").bfloat16()
    w = torch.ones(2, d, device="cuda")
    y, y2 = torch.empty_like(x), torch.empty_like(x)
    B.ulysses_a2a_4d_qk_fused(plan, [x], [x], [y], [y2], w, EPS, THETA)
    ang = turns(S, d, ext, (2, 3, 3), 2)
    close(y, rotate(norm(x, w[0]), ang, False), "bfloat16", 1e-5)
    assert torch.equal(y, y2)


def test_packed_chunked_and_differentiable():
    """The packed call with a grid: chunked launches give the same bytes, and the gradients that
    autograd returns are the backward's."""
    c = (2, 1, [48, 42], [2, 2], 64, (3, 5, 6), (12, 10, 10), 0)
    W, b, seq, heads, d, extents, pairs, first = c
    plan, q, k, gq, gk, w = make(c, "bfloat16", False)
    v = [torch.randn_like(x) for x in q]
    packed = [torch.stack(t, 2).contiguous().requires_grad_() for t in zip(q, k, v)]
    wl = w.clone().requires_grad_()
    whole = A.qkv_fused(plan, packed, wl, EPS, THETA)
    B.ulysses_plan_set_chunk_bytes(plan, 8192)
    assert B.ulysses_plan_num_chunks(plan) > 1
    parts = A.qkv_fused(plan, packed, wl, EPS, THETA)
    for a, b_ in zip(whole, parts):
        assert all(torch.equal(x, y) for x, y in zip(a, b_))
    ang = turns(sum(seq), d, extents, pairs, first)
    close(torch.cat(whole[0], 2), rotate(norm(torch.cat(q, 1), w[0]), ang, False), "bfloat16", 1e-5)
    torch.autograd.backward(whole[0] + whole[1], gq + gk)
    dq, dk = ([torch.empty_like(x) for x in q] for _ in range(2))
    dw = torch.empty_like(w)
    B.ulysses_plan_set_chunk_bytes(plan, 1 << 30)
    ws = torch.empty(B.ulysses_qk_fused_backward_workspace(plan), dtype=torch.uint8, device="cuda")
    B.ulysses_a2a_4d_qk_fused_backward(plan, dq, dk, q, k, gq, gk, w, dw, EPS, THETA, ws)
    for p, x, y in zip(packed, dq, dk):
        assert torch.equal(p.grad[:, :, 0], x) and torch.equal(p.grad[:, :, 1], y)


def test_gradient_against_differences():
    """The backward's direction against a central difference of the library's own forward."""
    c = (2, 1, [20, 16], [2, 1], 64, (2, 3, 6), (12, 10, 10), 0)
    plan, q, k, gq, gk, w = make(c, "float16", True)
    x, wl = [t.clone().requires_grad_() for t in q], w.clone()
    out, _ = A.qk_fused(plan, x, [t.clone() for t in k], wl, EPS, THETA)
    torch.autograd.backward(out, gq)
    h = 2.0 ** -3  # fp16 values near 1 step by 2^-10: the step's own rounding stays below 2^-8 of it
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    v = [torch.randn(t.shape, generator=g, device="cuda") for t in q]
    side = []
    for sgn in (1, -1):
        xs = [(t.float() + sgn * h * u).half() for t, u in zip(q, v)]
        o, _ = A.qk_fused(plan, xs, k, wl, EPS, THETA)
        side.append((xs, o))
    num = sum(((a.double() - b_.double()) * gg.double()).sum()
              for a, b_, gg in zip(side[0][1], side[1][1], gq)).item()
    ana = sum(((a.double() - b_.double()) * t.grad.double()).sum()
              for a, b_, t in zip(side[0][0], side[1][0], x)).item()
    # the third-order term of a step of 1/8 in every one of 64 columns: 2 h^3 / 6 of unit-scale
    # derivatives against 2 h, one part in 400, times a few for the norm's curvature
    scale = math.sqrt(sum((t.grad.double() ** 2).sum().item() for t in x)) * 2 * h
    assert abs(num - ana) <= 0.05 * max(scale, abs(ana)), (num, ana)
