"""Attention shapes that take the kernels' other ways: ragged keys in the long layout above d = 64, ragged
keys under 33 to 128 rows of one tile, more units of single tokens than CTAs without key counts, and
gradients away from unit scale. Tolerances as in test_gpu_attention.py and
test_gpu_attention_backward.py."""
import math

import pytest
import torch

import test_gpu_attention as fwd
import test_gpu_attention_backward as bwd
from test_gpu_attention import attend, i32, inputs, plans
from ulysses_sequence_all_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_timeout():
    yield
    assert B.ulysses_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("shape", [
    (1, 4, 300, 900, [1], 1, 128),     # long layout, d = 128
    (2, 4, 260, 1500, [1, 1], 2, 96),
    (1, 4, 17, 2600, [2], 4, 128),     # 68 rows
    (2, 4, 9, 3000, [1, 1], 4, 64),    # 36 rows
    (1, 4, 16, 1300, [1], 8, 72),      # 128 rows
    (1, 4, 33, 700, [2], 1, 8),
], ids=lambda s: "x".join(map(str, (s[2], s[3], s[5], s[6]))))
def test_ragged_keys(shape, causal, dtype):
    W, b, sq, skv, kv_heads, g, d = shape
    qp, kp = plans(*shape, dtype)
    for seed, lens in enumerate(((0, 1, 128, skv), (skv - 1, 129, skv // 2, 513))):
        q, k, v = inputs(*shape, dtype, seed=seed)
        n = i32(*lens)
        for t in (k, v):
            for x in t:
                for bb, m in enumerate(lens):
                    x[bb, m:] = math.nan if bb % 2 else math.inf
        kw = {"kv_lens": n}
        if causal:
            kw |= {"causal": True, "q_start": n - sq}
        o, lse = attend(qp, kp, q, k, v, 0.2, **kw)
        zero = lambda t: [torch.nan_to_num(x, 0, 0, 0) for x in t]
        fwd.check(q, zero(k), zero(v), o, lse, 0.2, **kw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("skv", [77, 256, 384, 500, 513])
@pytest.mark.parametrize("b", [1, 3])
def test_padded_text(b, skv, dtype):
    """Few key blocks with key counts at d = 128, in either layout: more units than CTAs, of all lengths."""
    shape = (2, b, 4100, skv, [4, 3], 1, 128)
    qp, kp = plans(*shape, dtype)
    for part in (1.0, 0.6, 0.3):
        q, k, v = inputs(*shape, dtype, seed=9)
        lens = [max(1, int(skv * part) - 40 * i) for i in range(b)]
        for t in (k, v):
            for x in t:
                for bb, m in enumerate(lens):
                    x[bb, m:] = math.nan
        o, lse = attend(qp, kp, q, k, v, 0.1, kv_lens=i32(*lens))
        zero = lambda t: [torch.nan_to_num(x, 0, 0, 0) for x in t]
        fwd.check(q, zero(k), zero(v), o, lse, 0.1, kv_lens=i32(*lens))


@pytest.mark.parametrize("shape", [(1, 200, 1, 700, [1], 1, 64), (2, 90, 1, 400, [1, 2], 8, 128),
                                   (1, 170, 5, 520, [1], 16, 128)],
                         ids=lambda s: "x".join(map(str, (s[1], s[2], s[3], s[5], s[6]))))
def test_more_single_tokens_than_ctas(shape):
    W, b, sq, skv, kv_heads, g, d = shape
    assert b * sum(kv_heads) > 152
    qp, kp = plans(*shape, torch.bfloat16)
    q, k, v = inputs(*shape, torch.bfloat16, seed=2)
    for kw in ({}, {"causal": True, "q_start": i32(*[skv - sq - i for i in range(b)])}):
        o, lse = attend(qp, kp, q, k, v, 0.15, **kw)
        fwd.check(q, k, v, o, lse, 0.15, **kw)


@pytest.mark.parametrize("size", [1e-3, 1e3])
def test_gradients_of_another_scale(size):
    shape = (2, 2, 200, 333, [1, 2], 2, 128)
    qp, kp = plans(*shape, torch.bfloat16)
    q, k, v = inputs(*shape, torch.bfloat16, seed=3)
    o, lse, go = bwd.given(q, k, v, 0.1, causal=True)
    go = [(size * x.float()).bfloat16() for x in go]
    got = bwd.gradients(qp, kp, q, k, v, o, lse, go, 0.1, causal=True)
    bwd.check(got, q, k, v, o, lse, go, 0.1, causal=True)
