"""Attention of every rank's heads (ulysses_attention) against the definition in 64 bits.

Tolerances. The output is rounded once to the element type (u, half a step: bf16 2^-8, fp16 2^-11).
Each probability is rounded to it as well, off by u p_j at most, which moves the output by at most
u sum_j p_j |v_j| =: u a. The fp32 parts are scores (d products of 16-bit values, each sum off by
2^-22 of the sum of magnitudes at most, times the scale: below 1e-5 for the inputs here), exponentials
(2^-21) and their sums: 1e-4 a covers them tenfold. So |o - ref| <= u |ref| + (u + 1e-4) a.
fp16 probabilities below 2^-14 are off by 2^-25 each in absolute terms. They are kept relative to a
maximum that may lag by 2^8 but never leads, so the row's sum is at least 1: skv 2^-25 max|v|, with
max|v| < 8.
lse is fp32: 2^-22 of its size plus the score's error, 3e-5."""
import math

import pytest
import torch

from attention_reference import HALF_STEP, forward
from gpu_util import GuardedOutputs
from ulysses_sequence_all_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    B.library()
    yield
    assert B.ulysses_device_status() == 0, "a kernel recorded a wait timeout"


@pytest.fixture(autouse=True)
def no_timeout():
    yield
    assert B.ulysses_device_status() == 0


def split(total, W):
    return [total // W + (r < total % W) for r in range(W)]


def plans(W, b, sq, skv, kv_heads, g, d, dtype):
    name = str(dtype).split(".")[1]
    return (B.ulysses_plan(W, b, split(sq, W), [g * m for m in kv_heads], d, name),
            B.ulysses_plan(W, b, split(skv, W), kv_heads, d, name))


def inputs(W, b, sq, skv, kv_heads, g, d, dtype, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dtype)
    return ([rnd(b, sq, g * m, d) for m in kv_heads], [rnd(b, skv, m, d) for m in kv_heads],
            [rnd(b, skv, m, d) for m in kv_heads])


def attend(qp, kp, q, k, v, scale, **kw):
    dtype = q[0].dtype
    o = GuardedOutputs([x.shape for x in q], dtype)
    lse = GuardedOutputs([(x.shape[0], x.shape[2], x.shape[1]) for x in q], torch.float32)
    need = B.ulysses_attention_workspace(qp, kp)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda") if need else None  # NaN patterns
    B.ulysses_attention(qp, kp, q, k, v, o.tensors, lse.tensors, scale=scale, workspace=ws, **kw)
    torch.cuda.synchronize()
    assert o.guards_intact() and lse.guards_intact()
    return o.tensors, lse.tensors


def check(q, k, v, o, lse, scale, **kw):
    for r in range(len(q)):
        if q[r].numel() == 0:
            continue
        want, z, a = forward(q[r], k[r], v[r], scale, **kw)
        u = HALF_STEP[q[r].dtype]
        tiny = k[r].shape[1] * 2.0 ** -25 * 8 if q[r].dtype == torch.float16 else 0.0
        tol = u * want.abs() + (u + 1e-4) * a + tiny + 2.0 ** -24
        err = (o[r].double() - want).abs()
        assert not (err > tol).any() and not o[r].isnan().any(), \
            f"rank {r}: {int((err > tol).sum())} off, worst {float((err - tol).max())}"
        empty = z == -math.inf
        assert torch.equal(lse[r] == -math.inf, empty)
        assert bool((o[r].transpose(1, 2)[empty] == 0).all())
        fin = ~empty
        le = (lse[r].double() - z)[fin].abs()
        assert not (le > 3e-5 + 2.0 ** -22 * z[fin].abs()).any(), float(le.max())


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


SHAPES = [
    # W, b, sq, skv, kv heads, group, d
    (1, 1, 1, 1, [1], 1, 64),
    (1, 1, 128, 128, [1], 1, 128),
    (1, 1, 256, 256, [1], 1, 64),
    (2, 2, 333, 517, [2, 1], 1, 128),
    (3, 1, 200, 129, [1, 0, 2], 1, 64),
    (1, 3, 65, 1000, [2], 1, 72),
    (2, 1, 129, 640, [1, 2], 4, 128),
    (1, 2, 100, 300, [2], 3, 80),        # three heads share: a tile holds 42 tokens
    (1, 1, 17, 260, [1], 64, 64),        # two tokens a tile
    (1, 2, 300, 77, [3], 1, 8),
    (1, 1, 140, 200, [1], 5, 120),
    (8, 1, 515, 515, [1] * 8, 2, 96),
    (1, 1, 1, 5000, [2], 8, 128),        # one token: the keys are split
    (2, 3, 1, 4100, [1, 1], 1, 64),
    (1, 2, 7, 3001, [1], 4, 72),
    (1, 1, 1500, 40, [2], 1, 40),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("shape", SHAPES, ids=["x".join(map(str, (s[0], s[1], s[2], s[3], s[5], s[6]))) for s in SHAPES])
def test_matches_definition(shape, causal, dtype):
    W, b, sq, skv, kv_heads, g, d = shape
    qp, kp = plans(*shape, dtype)
    q, k, v = inputs(*shape, dtype)
    scale = d ** -0.5
    kw = {}
    if causal and sq < skv:  # the rows are the last of the sequence
        kw = {"causal": True, "q_start": i32(*[skv - sq] * b)}
    elif causal:
        kw = {"causal": True}
    o, lse = attend(qp, kp, q, k, v, scale, **kw)
    check(q, k, v, o, lse, scale, **kw)


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("shape", [(2, 4, 150, 300, [1, 2], 2, 64), (1, 4, 1, 3000, [2], 4, 128),
                                   (1, 4, 129, 270, [1], 1, 72)], ids=["tiles", "token", "odd"])
def test_ragged_keys_and_what_lies_past_them(shape, causal):
    """Lengths of zero, one, at and inside a block, past the tensor; NaN and infinity past them."""
    dtype = torch.bfloat16
    W, b, sq, skv, kv_heads, g, d = shape
    qp, kp = plans(*shape, dtype)
    q, k, v = inputs(*shape, dtype, seed=4)
    for lens in ((0, 1, 128, skv + 9), (skv, 129, -3, 255)):
        n = i32(*lens)
        for t in (k, v):
            for x in t:
                for bb, m in enumerate(lens):
                    x[bb, max(0, m):] = math.nan if bb % 2 else math.inf
        kw = {"kv_lens": n}
        if causal:
            kw |= {"causal": True, "q_start": n - sq}  # negative where the rows outnumber the keys
        o, lse = attend(qp, kp, q, k, v, 0.2, **kw)
        kw["kv_lens"] = n.clamp(0, skv)
        check(q, [torch.nan_to_num(x, 0, 0, 0) for x in k], [torch.nan_to_num(x, 0, 0, 0) for x in v],
              o, lse, 0.2, **kw)
        q, k, v = inputs(*shape, dtype, seed=5)


@pytest.mark.parametrize("ctas", [1, 3, 0])
@pytest.mark.parametrize("shape", [(2, 6, 300, 1300, [1, 2], 2, 64), (1, 6, 1, 2600, [3], 2, 128)],
                         ids=["tiles", "token"])
def test_many_ragged_units_on_few_ctas(shape, ctas):
    """Each CTA runs through many units of different lengths, its ring of stages round many times,
    with NaN past the keys of every batch element."""
    W, b, sq, skv, kv_heads, g, d = shape
    qp, kp = plans(*shape, torch.bfloat16)
    B.ulysses_plan_set_max_ctas(qp, ctas)
    for seed, lens in enumerate(((1300, 100, 5, 900, 0, 1299), (640, 1280, 1, 2, 130, 129))):
        q, k, v = inputs(*shape, torch.bfloat16, seed=seed)
        n = i32(*lens)
        for t in (k, v):
            for x in t:
                for bb, m in enumerate(lens):
                    x[bb, m:] = math.nan
        for kw in ({"kv_lens": n}, {"kv_lens": n, "causal": True}):
            o, lse = attend(qp, kp, q, k, v, 0.2, **kw)
            check(q, [torch.nan_to_num(x, 0, 0, 0) for x in k],
                  [torch.nan_to_num(x, 0, 0, 0) for x in v], o, lse, 0.2, **kw)


def test_causal_start_beyond_and_before_the_keys():
    shape = (1, 4, 40, 200, [1], 1, 64)
    qp, kp = plans(*shape, torch.bfloat16)
    q, k, v = inputs(*shape, torch.bfloat16, seed=6)
    for start in (i32(-40, -39, 0, 2 ** 31 - 1), i32(-2 ** 31, 160, 199, 500)):
        o, lse = attend(qp, kp, q, k, v, 0.125, causal=True, q_start=start)
        check(q, k, v, o, lse, 0.125, causal=True, q_start=start.long())


def test_growing_and_falling_scores():
    """Scores that grow block by block (each block rescales the output), fall, and are large."""
    shape = (1, 1, 200, 1000, [1], 1, 64)
    qp, kp = plans(*shape, torch.float16)
    q, k, v = inputs(*shape, torch.float16, seed=7)
    ramp = torch.linspace(-40, 40, 1000, device="cuda")[None, :, None]
    for sign in (1, -1):
        q[0][..., 0] = 8.0
        k[0][..., 0] = (sign * ramp).half()
        o, lse = attend(qp, kp, q, k, v, 0.125)
        # scores reach 40, so their fp32 sums are off by up to 2^-22 * 330 * scale: 1e-5
        check(q, k, v, o, lse, 0.125)


def test_same_bytes_every_time_and_on_another_stream():
    shape = (2, 2, 300, 2500, [1, 2], 2, 128)
    qp, kp = plans(*shape, torch.bfloat16)
    q, k, v = inputs(*shape, torch.bfloat16, seed=8)
    o, lse = attend(qp, kp, q, k, v, 0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2, lse2 = attend(qp, kp, q, k, v, 0.1)
    B.ulysses_plan_set_max_ctas(qp, 7)
    o3, lse3 = attend(qp, kp, q, k, v, 0.1)
    for x, y, z in zip(o + lse, o2 + lse2, o3 + lse3):
        assert torch.equal(x, y)
    check(q, k, v, o3, lse3, 0.1)


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes: a token near its end, and the elements there."""
    skv, m, d = 2_200_000, 8, 128
    qp = B.ulysses_plan(1, 1, [2], [m], d, "bfloat16")
    kp = B.ulysses_plan(1, 1, [skv], [m], d, "bfloat16")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    q = [torch.randn((1, 2, m, d), generator=gen, device="cuda").bfloat16()]
    k = [torch.randn((1, skv, m, d), generator=gen, device="cuda", dtype=torch.bfloat16)]
    v = [torch.randn((1, skv, m, d), generator=gen, device="cuda", dtype=torch.bfloat16)]
    k[0][:, -5:] = 4 * q[0][:, :1]  # the last keys draw the first token's weight
    o, lse = attend(qp, kp, q, k, v, d ** -0.5)
    check(q, k, v, o, lse, d ** -0.5)
