"""Attention with a sliding window and first tokens that stay visible (ulysses_attention_window) and its
gradient, against the definition in 64 bits.

Tolerances of the forward: those of attention without a window, for the same roundings. The output is
rounded once (u, half a step: bf16 2^-8, fp16 2^-11), each probability by u p_j: u sum_j p_j |v_j| =: u a;
the fp32 parts 1e-4 a; fp16 probabilities below 2^-14 are off by 2^-25 each: keys 2^-25 max|v|, max|v| < 8.
lse is fp32: 2^-22 of its size plus the score's error, 3e-5.
The gradient: each result is rounded once (u of itself); P (for dv) or dS (for dq, dk) is rounded to the
element type, u of the sum of magnitudes that it enters; what is fp32 on the way (scores off by up to 1e-5, so
P by that share of itself; lse 3e-5; dP and D, sums of 16-bit products off by 2^-22 of their magnitudes) is
covered by 1e-4 of the sum of magnitudes of all that is summed. fp16 holds P times 2^14 and dS times a power of
two from a bound: what lies below its range is off by 2^-25 of that scale, below the other terms' 1e-4."""
import math

import pytest
import torch

import window_reference as R
from gpu_util import GuardedOutputs
from ulysses_sequence_all_gb300 import binding as B

pytestmark = pytest.mark.gpu
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    B.library()


@pytest.fixture(autouse=True)
def status():
    yield
    assert B.ulysses_device_status() == 0


def split(total, W):
    return [total // W + (r < total % W) for r in range(W)]


def i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    """Keys, values and rows of q and go that nothing sees hold `fill`."""

    def __init__(self, W, b, sq, skv, kv_heads, g, d, window, sinks, dtype=torch.bfloat16, kv_lens=None,
                 q_start=None, seed=0, fill=math.nan):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dtype)
        self.see = R.visible(b, sq, skv, window, sinks, kv_lens, q_start)
        keys, rows = self.see.any(1)[:, :, None, None], self.see.any(2)[:, :, None, None]
        hide = lambda x, some: torch.where(some, x, torch.full_like(x, fill))
        self.q = [hide(rnd(b, sq, g * m, d), rows) for m in kv_heads]
        self.go = [hide(rnd(b, sq, g * m, d), rows) for m in kv_heads]
        self.k, self.v = ([hide(rnd(b, skv, m, d), keys) for m in kv_heads] for _ in range(2))
        self.window, self.sinks, self.kv_lens, self.q_start = window, sinks, i32(kv_lens), i32(q_start)
        self.scale, self.dtype = d ** -0.5, dtype
        name = str(dtype).split(".")[1]
        self.qp = B.ulysses_plan(W, b, split(sq, W), [g * m for m in kv_heads], d, name)
        self.kp = B.ulysses_plan(W, b, split(skv, W), kv_heads, d, name)

    def masks(self):
        return dict(scale=self.scale, window=self.window, sinks=self.sinks, kv_lens=self.kv_lens,
                    q_start=self.q_start)

    def workspace(self, need):
        return torch.full((need,), 255, dtype=torch.uint8, device="cuda") if need else None  # NaN patterns

    def forward(self):
        o = GuardedOutputs([x.shape for x in self.q], self.dtype)
        lse = GuardedOutputs([(x.shape[0], x.shape[2], x.shape[1]) for x in self.q], torch.float32)
        ws = self.workspace(B.ulysses_attention_window_workspace(self.qp, self.kp, self.window, self.sinks))
        B.ulysses_attention_window(self.qp, self.kp, self.q, self.k, self.v, o.tensors, lse.tensors,
                                   workspace=ws, **self.masks())
        torch.cuda.synchronize()
        assert o.guards_intact() and lse.guards_intact()
        return o.tensors, lse.tensors

    def check(self, o, lse):
        u = HALF_STEP[self.dtype]
        for r in range(len(self.q)):
            if self.q[r].numel() == 0:
                continue
            want, z, a = R.forward(self.q[r], self.k[r], self.v[r], self.scale, self.see)
            tiny = self.k[r].shape[1] * 2.0 ** -25 * 8 if self.dtype == torch.float16 else 0.0
            err = (o[r].double() - want).abs()
            tol = u * want.abs() + (u + 1e-4) * a + tiny + 2.0 ** -24
            assert not (err > tol).any() and not o[r].isnan().any(), \
                f"rank {r}: {int((err > tol).sum())} off, worst {float((err - tol).max())}"
            empty = z == -math.inf
            assert torch.equal(lse[r] == -math.inf, empty)
            assert bool((o[r].transpose(1, 2)[empty] == 0).all())
            le = (lse[r].double() - z)[~empty].abs()
            assert not (le > 3e-5 + 2.0 ** -22 * z[~empty].abs()).any(), float(le.max())

    def backward(self, o, lse):
        out = [GuardedOutputs([x.shape for x in t], self.dtype) for t in (self.q, self.k, self.v)]
        ws = self.workspace(B.ulysses_attention_window_backward_workspace(self.qp, self.kp, self.window,
                                                                          self.sinks))
        B.ulysses_attention_window_backward(self.qp, self.kp, *[x.tensors for x in out], self.q, self.k,
                                            self.v, o, lse, self.go, workspace=ws, **self.masks())
        torch.cuda.synchronize()
        assert all(x.guards_intact() for x in out)
        return [x.tensors for x in out]

    def tolerance(self, x, y, z):
        """Of a gradient x with its two sums of magnitudes."""
        u = HALF_STEP[self.dtype]
        return u * x.abs() + u * y + 1e-4 * z + 2.0 ** -24

    def check_backward(self, o, lse, grads):
        for r in range(len(self.q)):
            if self.q[r].numel() == 0:
                continue
            want, a, m = R.backward(self.q[r], self.k[r], self.v[r], o[r], lse[r], self.go[r], self.scale,
                                    self.see)
            for name, got, x, y, z in zip(("dq", "dk", "dv"), (g[r] for g in grads), want, a, m):
                err = (got.double() - x).abs()
                tol = self.tolerance(x, y, z)
                assert not (err > tol).any() and not got.isnan().any(), \
                    f"rank {r} {name}: {int((err > tol).sum())} off, worst {float((err - tol).max())}"


SHAPES = [
    # W, b, queries, keys, kv heads, group, d
    (1, 1, 1, 1, [1], 1, 64),
    (1, 1, 33, 33, [1], 1, 128),
    (1, 2, 300, 300, [2], 1, 64),
    (2, 1, 700, 700, [1, 2], 1, 128),
    (3, 2, 500, 517, [1, 0, 2], 2, 72),
    (1, 1, 1029, 1029, [1], 4, 128),
    (1, 2, 400, 333, [1], 3, 80),         # more rows than keys; three heads share: 42 tokens a tile
    (1, 1, 130, 600, [1], 64, 64),        # two tokens a tile
    (8, 1, 515, 515, [1] * 8, 2, 96),
    (1, 1, 900, 900, [1], 1, 8),
]
IDS = ["x".join(map(str, (s[0], s[1], s[2], s[3], s[5], s[6]))) for s in SHAPES]
WINDOWS = [(1, 0), (1, 3), (64, 4), (128, 0), (200, 130), (257, 1), (5000, 7)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("window, sinks", WINDOWS)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_matches_definition(shape, window, sinks, dtype):
    c = Case(*shape, window, sinks, dtype)
    o, lse = c.forward()
    c.check(o, lse)
    c.check_backward(o, lse, c.backward(o, lse))


@pytest.mark.parametrize("window, sinks", [(1, 0), (50, 0), (50, 5), (300, 140), (2000, 0)])
@pytest.mark.parametrize("fill", [math.nan, math.inf])
def test_ragged_keys_and_starts(window, sinks, fill):
    """Key counts of zero, one, inside and past the tensor; rows before the first key, behind the last one's
    window (which see nothing then), far into a cache whose keys before the window hold anything."""
    for dtype in (torch.bfloat16, torch.float16):
        c = Case(2, 5, 333, 640, [2, 1], 2, 64, window, sinks, dtype, kv_lens=[0, 1, 129, 640, 9000], fill=fill)
        o, lse = c.forward()
        c.check(o, lse)
        c.check_backward(o, lse, c.backward(o, lse))
        c = Case(1, 6, 200, 800, [1], 2, 128, window, sinks, dtype, kv_lens=[800, 700, 300, 10, 800, 750],
                 q_start=[600, 500, 290, -100, -400, 900], fill=fill)
        o, lse = c.forward()
        c.check(o, lse)
        c.check_backward(o, lse, c.backward(o, lse))


@pytest.mark.parametrize("sq", [1, 3, 16, 17, 100])
@pytest.mark.parametrize("window, sinks", [(1, 0), (100, 4), (3000, 0)])
def test_few_rows_on_a_cache(sq, window, sinks):
    for g, d in ((1, 64), (2, 128), (4, 40)):
        lens = [1500, 1, 1400, 77, 0]
        c = Case(2, 5, sq, 1501, [1, 2], g, d, window, sinks, kv_lens=lens, q_start=[n - sq for n in lens])
        o, lse = c.forward()
        c.check(o, lse)
        c.check_backward(o, lse, c.backward(o, lse))


@pytest.mark.parametrize("sinks", [3, 300])
def test_first_tokens_of_many_rows(sinks):
    """Their gradients are summed in several parts, some of them empty."""
    for dtype, lens in ((torch.bfloat16, None), (torch.float16, [9000, 2000])):
        c = Case(1, 1 if lens is None else 2, 9000, 9000, [1], 1, 64, 100, sinks, dtype, kv_lens=lens)
        o, lse = c.forward()
        c.check(o, lse)
        c.check_backward(o, lse, c.backward(o, lse))


def bits(xs):
    return [x.view(torch.uint8) for t in xs for x in t]


def test_the_same_bits_under_a_cap_and_again():
    c = Case(2, 2, 900, 900, [1, 2], 2, 64, 130, 5, kv_lens=[900, 600])
    o, lse = c.forward()
    want = bits([o, lse, *c.backward(o, lse)])
    for cap in (0, 1, 7, 200):
        B.ulysses_plan_set_max_ctas(c.qp, cap)
        got = c.forward()
        for x, y in zip(bits([*got, *c.backward(*got)]), want):
            assert torch.equal(x, y)


def test_a_window_over_everything_is_causal_attention():
    for shape in ((2, 2, 600, 600, [1, 2], 2, 128), (1, 1, 400, 400, [3], 1, 64)):
        c = Case(*shape, 600, 0)
        o, lse = c.forward()
        o2, lse2 = [torch.empty_like(x) for x in o], [torch.empty_like(x) for x in lse]
        need = B.ulysses_attention_workspace(c.qp, c.kp)
        B.ulysses_attention(c.qp, c.kp, c.q, c.k, c.v, o2, lse2, c.scale, causal=True,
                            workspace=c.workspace(need))
        for x, y in zip(bits([o, lse]), bits([o2, lse2])):
            assert torch.equal(x, y)


def test_gradient_against_differences():
    """sum(o * go) along a direction in q, k and v, by central differences in 64 bits of the definition."""
    c = Case(1, 1, 150, 150, [1], 2, 64, 40, 3, torch.float16)
    o, lse = c.forward()
    grads = c.backward(o, lse)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(9)
    loss = lambda q, k, v: float((R.forward(q, k, v, c.scale, c.see)[0] * c.go[0].double()).sum())
    leaves = [c.q[0].double(), c.k[0].double(), c.v[0].double()]
    sums = zip(*R.backward(c.q[0], c.k[0], c.v[0], o[0], lse[0], c.go[0], c.scale, c.see))
    for i, xyz in enumerate(sums):
        step = torch.randn(leaves[i].shape, generator=gen, device="cuda", dtype=torch.float64)
        move = lambda t: loss(*[x + t * step if j == i else x for j, x in enumerate(leaves)])
        want = (move(1e-4) - move(-1e-4)) / 2e-4
        off = abs(float((grads[i][0].double() * step).sum()) - want)
        assert off < float((c.tolerance(*xyz) * step.abs()).sum()) + 1e-5 * abs(want)


def test_graph_and_stream():
    c = Case(1, 2, 500, 500, [2], 2, 64, 100, 4, kv_lens=[500, 300], fill=0.0)
    out, lse = [torch.empty_like(x) for x in c.q], [torch.empty(2, 4, 500, device="cuda")]
    grads = [[torch.empty_like(x) for x in t] for t in (c.q, c.k, c.v)]
    ws = c.workspace(B.ulysses_attention_window_workspace(c.qp, c.kp, 100, 4))
    wb = c.workspace(B.ulysses_attention_window_backward_workspace(c.qp, c.kp, 100, 4))

    def call():
        B.ulysses_attention_window(c.qp, c.kp, c.q, c.k, c.v, out, lse, workspace=ws, **c.masks())
        B.ulysses_attention_window_backward(c.qp, c.kp, *grads, c.q, c.k, c.v, out, lse, c.go, workspace=wb,
                                            **c.masks())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    c.kv_lens.copy_(i32([77, 500]))
    for x in c.q:
        x.mul_(-0.5)
    graph.replay()
    torch.cuda.synchronize()
    c.see = R.visible(2, 500, 500, 100, 4, [77, 500])
    c.check(out, lse)
    c.check_backward(out, lse, grads)


def test_waits_that_run_out_are_reported():
    """With a limit of nothing every kernel gives up, says so, and the next call is whole again."""
    c = Case(1, 1, 9000, 9000, [2], 1, 128, 4000, 4, fill=0.0)
    B.ulysses_plan_set_max_ctas(c.qp, 1)  # more units a CTA than it knows ahead
    o, lse = c.forward()
    few = Case(1, 4, 1, 60000, [2], 4, 128, 50000, 4, q_start=[59999] * 4, fill=0.0)
    few_o = few.forward()
    B.ulysses_selftest_attention_wait_limit(0)
    try:
        c.forward()
        assert B.ulysses_device_status() == 1
        c.backward(o, lse)
        assert B.ulysses_device_status() == 1
        few.forward()
        assert B.ulysses_device_status() in (0, 1)  # (its copies may be there at once)
    finally:
        B.ulysses_selftest_attention_wait_limit(2000000)
    for x, y in zip(bits(c.forward()), bits([o, lse])):
        assert torch.equal(x, y)
    for x, y in zip(bits(few.forward()), bits(few_o)):
        assert torch.equal(x, y)
