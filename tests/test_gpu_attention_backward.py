"""Gradient of attention (ulysses_attention_backward) against the formulas in 64 bits and against
differences, the differentiable form, and graph capture.

Tolerances, u half a step of the element type (bf16 2^-8, fp16 2^-11). Each gradient is rounded once: u
of it. Its 16-bit factor is rounded as well: P for dv, so u sum P |go|; dS for dq and dk, so u scale sum
|dS| |k| (|q|): the reference's first sums, a. What is fp32 on the way (scores off by up to 1e-5, so P by
that share of itself; dP and D, sums of 16-bit products off by 2^-22 of their magnitudes) is covered
tenfold by 1e-4 of the second sums, m. So |x - ref| <= u |ref| + u a + 1e-4 m. fp16 factors below 2^-14
are off by 2^-25 each: times the number of terms, times 8 for the largest of |go|, |k|, |q|, and a scale
below 1."""
import math

import pytest
import torch

from attention_reference import HALF_STEP, backward, forward
from gpu_util import GuardedOutputs
from test_gpu_attention import i32, inputs, plans
from ulysses_sequence_all_gb300 import autograd as A
from ulysses_sequence_all_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    B.library()
    yield


@pytest.fixture(autouse=True)
def no_timeout():
    yield
    assert B.ulysses_device_status() == 0


def given(q, k, v, scale, seed=0, **kw):
    """The forward's outputs (from the definition, rounded as the library rounds them) and go."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(100 + seed)
    o, lse = [], []
    for r in range(len(q)):
        oo, z, _ = forward(q[r], k[r], v[r], scale, **kw)
        o.append(oo.to(q[r].dtype))
        lse.append(z.float())
    go = [torch.randn(x.shape, generator=gen, device="cuda").to(x.dtype) for x in q]
    return o, lse, go


def gradients(qp, kp, q, k, v, o, lse, go, scale, **kw):
    g = [GuardedOutputs([x.shape for x in t], t[0].dtype) for t in (q, k, v)]
    ws = torch.full((B.ulysses_attention_backward_workspace(qp, kp),), 255, dtype=torch.uint8,
                    device="cuda")
    B.ulysses_attention_backward(qp, kp, *[x.tensors for x in g], q, k, v, o, lse, go, scale=scale,
                                 workspace=ws, **kw)
    torch.cuda.synchronize()
    assert all(x.guards_intact() for x in g)
    return [x.tensors for x in g]


def check(got, q, k, v, o, lse, go, scale, **kw):
    for r in range(len(q)):
        if q[r].numel() == 0:
            continue
        want, near, far = backward(q[r], k[r], v[r], o[r], lse[r], go[r], scale, **kw)
        u = HALF_STEP[q[r].dtype]
        n = max(q[r].shape[1] * (q[r].shape[2] // k[r].shape[2]), k[r].shape[1])
        tiny = n * 2.0 ** -25 * 8 if q[r].dtype == torch.float16 else 0.0
        for name, x, y, a, m in zip(("dq", "dk", "dv"), (t[r] for t in got), want, near, far):
            err = (x.double() - y).abs()
            tol = u * y.abs() + u * a + 1e-4 * m + tiny + 2.0 ** -24
            assert not x.isnan().any(), f"rank {r} {name}: NaN"
            assert not (err > tol).any(), \
                f"rank {r} {name}: {int((err > tol).sum())} off, worst {float((err - tol).max())}"


SHAPES = [
    # W, b, sq, skv, kv heads, group, d
    (1, 1, 1, 1, [1], 1, 64),
    (1, 1, 128, 128, [1], 1, 128),
    (1, 1, 256, 384, [1], 1, 64),
    (2, 2, 333, 517, [2, 1], 1, 128),
    (3, 1, 200, 129, [1, 0, 2], 1, 64),
    (1, 3, 65, 700, [2], 1, 72),
    (2, 1, 129, 340, [1, 2], 4, 128),
    (1, 2, 100, 300, [2], 3, 80),
    (1, 1, 17, 260, [1], 64, 64),
    (1, 2, 300, 77, [3], 1, 8),
    (1, 1, 140, 200, [1], 5, 120),
    (8, 1, 515, 515, [1] * 8, 2, 96),
    (1, 1, 1000, 40, [2], 1, 40),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("shape", SHAPES, ids=["x".join(map(str, (s[0], s[1], s[2], s[3], s[5], s[6]))) for s in SHAPES])
def test_matches_formulas(shape, causal, dtype):
    W, b, sq, skv, kv_heads, g, d = shape
    qp, kp = plans(*shape, dtype)
    q, k, v = inputs(*shape, dtype, seed=1)
    scale = d ** -0.5
    kw = {"causal": True} if causal else {}
    if causal and sq < skv:
        kw["q_start"] = i32(*[skv - sq] * b)
    o, lse, go = given(q, k, v, scale, **kw)
    got = gradients(qp, kp, q, k, v, o, lse, go, scale, **kw)
    check(got, q, k, v, o, lse, go, scale, **kw)


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("shape", [(2, 4, 150, 300, [1, 2], 2, 64), (1, 4, 129, 270, [1], 1, 128)],
                         ids=["shared", "odd"])
def test_ragged_keys_and_what_lies_past_them(shape, causal):
    dtype = torch.bfloat16
    W, b, sq, skv, kv_heads, g, d = shape
    qp, kp = plans(*shape, dtype)
    for seed, lens in enumerate(((0, 1, 128, skv + 9), (skv, 129, -3, 255))):
        q, k, v = inputs(*shape, dtype, seed=seed)
        n = i32(*lens)
        kw = {"kv_lens": n}
        if causal:
            kw |= {"causal": True, "q_start": n - sq}
        ref = dict(kw, kv_lens=n.clamp(0, skv))
        o, lse, go = given(q, k, v, 0.2, **ref)
        for t in (k, v):
            for x in t:
                for bb, m in enumerate(lens):
                    x[bb, max(0, m):] = math.nan if bb % 2 else math.inf
        got = gradients(qp, kp, q, k, v, o, lse, go, 0.2, **kw)
        zero = lambda t: [torch.nan_to_num(x, 0, 0, 0) for x in t]
        check(got, q, zero(k), zero(v), o, lse, go, 0.2, **ref)
        for t in got[1:]:
            for x in t:
                for bb, m in enumerate(lens):
                    assert bool((x[bb, max(0, m):] == 0).all())


@pytest.mark.parametrize("ctas", [1, 3, 0])
def test_many_ragged_units_on_few_ctas(ctas):
    """Each CTA runs through many units of different lengths, its rings of stages round many times,
    with NaN past the keys of every batch element."""
    shape = (2, 6, 300, 900, [1, 2], 3, 64)
    W, b, sq, skv, kv_heads, g, d = shape
    qp, kp = plans(*shape, torch.float16)
    B.ulysses_plan_set_max_ctas(qp, ctas)
    for seed, lens in enumerate(((900, 100, 5, 800, 0, 899), (640, 768, 1, 2, 130, 129))):
        q, k, v = inputs(*shape, torch.float16, seed=seed)
        n = i32(*lens)
        for kw in ({"kv_lens": n}, {"kv_lens": n, "causal": True}):
            o, lse, go = given(q, k, v, 0.2, **kw)
            dirty = [[x.clone() for x in t] for t in (k, v)]
            for t in dirty:
                for x in t:
                    for bb, m in enumerate(lens):
                        x[bb, m:] = math.nan
            got = gradients(qp, kp, q, *dirty, o, lse, go, 0.2, **kw)
            check(got, q, k, v, o, lse, go, 0.2, **kw)


def test_same_bits_every_time():
    shape = (2, 2, 300, 700, [1, 2], 2, 128)
    qp, kp = plans(*shape, torch.bfloat16)
    q, k, v = inputs(*shape, torch.bfloat16, seed=8)
    o, lse, go = given(q, k, v, 0.1)
    one = gradients(qp, kp, q, k, v, o, lse, go, 0.1)
    B.ulysses_plan_set_max_ctas(qp, 5)
    two = gradients(qp, kp, q, k, v, o, lse, go, 0.1)
    assert all(torch.equal(x, y) for a, b in zip(one, two) for x, y in zip(a, b))


def test_differentiable_form_and_differences():
    """autograd against the direct call, and against differences of the forward in 64 bits."""
    shape = (2, 2, 90, 150, [2, 1], 2, 64)
    qp, kp = plans(*shape, torch.float16)
    q, k, v = inputs(*shape, torch.float16, seed=3)
    lens = i32(150, 77)
    kw = {"kv_lens": lens, "causal": True, "q_start": i32(60, -5)}
    leaves = [[x.clone().requires_grad_() for x in t] for t in (q, k, v)]
    out = A.attention(qp, kp, *leaves, **kw)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    go = [torch.randn(x.shape, generator=gen, device="cuda").half() for x in out]
    torch.autograd.backward(out, go)
    lse = [torch.empty(x.shape[0], x.shape[2], x.shape[1], device="cuda") for x in q]
    o = [torch.empty_like(x) for x in q]
    need = B.ulysses_attention_workspace(qp, kp)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    B.ulysses_attention(qp, kp, q, k, v, o, lse, scale=64 ** -0.5, workspace=ws, **kw)
    assert all(torch.equal(a, b) for a, b in zip(o, out))
    direct = gradients(qp, kp, q, k, v, o, lse, go, 64 ** -0.5, **kw)
    for t, d in zip(leaves, direct):
        assert all(torch.equal(x.grad, y) for x, y in zip(t, d))
    # a step h along a random direction, the forward evaluated in 64 bits on both sides: the
    # gradient's own rounding is u of it and averages over the sum, h^2 is the difference's error
    h = 1e-4
    for t in range(3):
        dirs = [torch.randn(x.shape, generator=gen, device="cuda", dtype=torch.float64)
                for x in (q, k, v)[t]]
        num = 0.0
        for r in range(2):
            side = []
            for sgn in (1, -1):
                args = [q[r].double(), k[r].double(), v[r].double()]
                args[t] = args[t] + sgn * h * dirs[r]
                side.append(forward(*args, 64 ** -0.5, **kw)[0])
            num += ((side[0] - side[1]) * go[r].double()).sum().item() / (2 * h)
        ana = sum((x.grad.double() * d).sum().item() for x, d in zip(leaves[t], dirs))
        size = math.sqrt(sum((x.grad.double() ** 2).sum().item() for x in leaves[t]))
        assert abs(num - ana) <= 0.02 * size, (t, num, ana, size)


def test_graph_capture():
    """Forward and backward recorded in a CUDA graph after their first use, replayed on new
    values."""
    shape = (1, 1, 200, 200, [2], 2, 64)
    qp, kp = plans(*shape, torch.bfloat16)
    q, k, v = inputs(*shape, torch.bfloat16, seed=3)
    o, lse, go = given(q, k, v, 0.125, causal=True)
    grads = [[torch.empty_like(x) for x in t] for t in (q, k, v)]
    ws = torch.empty(B.ulysses_attention_backward_workspace(qp, kp), dtype=torch.uint8, device="cuda")

    def step():
        B.ulysses_attention(qp, kp, q, k, v, o, lse, scale=0.125, causal=True)
        B.ulysses_attention_backward(qp, kp, *grads, q, k, v, o, lse, go, scale=0.125, causal=True,
                                     workspace=ws)

    assert B.ulysses_attention_workspace(qp, kp) == 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, n in zip((q, k, v), inputs(*shape, torch.bfloat16, seed=4)):
        t[0].copy_(n[0])
    graph.replay()
    torch.cuda.synchronize()
    replayed = [g[0].clone() for g in grads]
    step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, g[0]) for a, g in zip(replayed, grads))
