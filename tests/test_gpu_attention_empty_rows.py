"""Causal rows that see no key (negative q_start: a batch padded at its start) may hold anything, and so may
their gradient.

Tolerances as in test_gpu_attention.py and test_gpu_attention_backward.py."""
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
@pytest.mark.parametrize("shape,starts", [((1, 4, 300, 200, [2], 2, 64), (-150, -299, -64, -400)),
                                          ((2, 4, 130, 700, [1, 2], 3, 128), (-1, -129, 3, -50)),
                                          ((1, 4, 1000, 150, [1], 1, 72), (-900, -129, -1, -511))],
                         ids=["shared", "three", "long"])
def test_rows_that_see_no_key(shape, starts, dtype):
    """Zero output and dq, and nothing of them in dk and dv."""
    W, b, sq, skv, kv_heads, g, d = shape
    qp, kp = plans(*shape, dtype)
    q, k, v = inputs(*shape, dtype, seed=12)
    kw = {"causal": True, "q_start": i32(*starts)}
    o, lse, go = bwd.given(q, k, v, 0.2, **kw)
    dirty_q, dirty_go = [x.clone() for x in q], [x.clone() for x in go]
    for i, t in enumerate((dirty_q, dirty_go)):
        for x in t:
            for bb, s in enumerate(starts):
                x[bb, :max(0, -s)] = math.nan if (bb + i) % 2 else math.inf
    o1, lse1 = attend(qp, kp, dirty_q, k, v, 0.2, **kw)
    fwd.check(q, k, v, o1, lse1, 0.2, **kw)
    got = bwd.gradients(qp, kp, dirty_q, k, v, o, lse, dirty_go, 0.2, **kw)
    bwd.check(got, q, k, v, o, lse, go, 0.2, **kw)
    for x in got[0]:
        for bb, s in enumerate(starts):
            assert bool((x[bb, :max(0, -s)] == 0).all())
