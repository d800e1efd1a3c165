"""Keys and values that no row sees may hold anything, also without key counts: causal calls on a cache
with room left (q_start, or fewer queries than keys).

Tolerances as in test_gpu_attention.py and test_gpu_attention_backward.py, against the definition with
zeros in place of what is hidden."""
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


def zero(t):
    return [torch.nan_to_num(x, 0, 0, 0) for x in t]


CACHES = [
    # W, b, sq, skv, kv heads, group, d; the starts
    ((1, 3, 1, 3000, [2], 4, 128), (1700, 0, 2998)),       # one token: parts of the keys
    ((2, 3, 7, 2100, [1, 1], 8, 64), (1000, 5, 2093)),     # a few: 56 rows
    ((1, 3, 200, 900, [1], 2, 128), (300, -20, 640)),      # tiles, over more than a ring of blocks
    ((2, 3, 150, 300, [1, 2], 2, 72), (0, 100, 140)),
    ((1, 2, 140, 500, [2], 1, 64), None),                  # no start: keys past the last row
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("shape,starts", CACHES, ids=[f"{s[0][2]}x{s[0][3]}x{s[0][6]}" for s in CACHES])
def test_keys_that_no_row_sees(shape, starts, dtype):
    W, b, sq, skv, kv_heads, g, d = shape
    qp, kp = plans(*shape, dtype)
    q, k, v = inputs(*shape, dtype, seed=11)
    kw = {"causal": True}
    if starts is not None:
        kw["q_start"] = i32(*starts)
    for t in (k, v):
        for x in t:
            for bb in range(b):
                x[bb, max(0, (starts[bb] if starts else 0) + sq):] = math.inf if bb % 2 else math.nan
    o, lse = attend(qp, kp, q, k, v, 0.2, **kw)
    fwd.check(q, zero(k), zero(v), o, lse, 0.2, **kw)
    o, lse, go = bwd.given(q, zero(k), zero(v), 0.2, **kw)
    got = bwd.gradients(qp, kp, q, k, v, o, lse, go, 0.2, **kw)
    bwd.check(got, q, zero(k), zero(v), o, lse, go, 0.2, **kw)
    for t in got[1:]:
        for x in t:
            for bb in range(b):
                assert bool((x[bb, max(0, (starts[bb] if starts else 0) + sq):] == 0).all())
