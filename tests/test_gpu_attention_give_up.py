"""The attention kernels' failure path, without a fault: with a wait limit of nothing, CTAs whose units take
longer than one look give up, finish what they have in flight, say so in the status word and return; the
device works on, and the same calls with the usual limit are right. And a limit that is short against a
unit, but long against a step of it, stops nothing: it counts only time in which nothing moves."""
import time

import pytest
import torch

from test_gpu_attention import inputs, plans
from ulysses_sequence_all_gb300 import binding as B

pytestmark = pytest.mark.gpu

DEFAULT = 2_000_000

# W, b, sq, skv, kv heads, group, d, CTA cap: more units a CTA than it knows ahead, each of some 100 us
FORWARD = [((1, 1, 3000, 40_000, [1], 1, 128), 1), ((1, 1, 3000, 40_000, [1], 1, 64), 1),
           ((1, 6, 1, 120_000, [1], 1, 128), 1), ((1, 6, 20, 120_000, [1], 4, 64), 1),
           ((1, 1, 40_000, 40_000, [8], 1, 128), 0)]
IDS = ["long128", "long64", "token", "paired", "stealing"]


@pytest.fixture(autouse=True)
def usual_limit():
    assert B.ulysses_device_status() == 0
    yield
    B.ulysses_selftest_attention_wait_limit(DEFAULT)
    assert B.ulysses_device_status() == 0


def make(shape, cap, dtype):
    qp, kp = plans(*shape, dtype)
    B.ulysses_plan_set_max_ctas(qp, cap)
    q, k, v = inputs(*shape, dtype, seed=1)
    o = [torch.zeros_like(x) for x in q]
    lse = [torch.zeros((x.shape[0], x.shape[2], x.shape[1]), device="cuda") for x in q]
    need = B.ulysses_attention_workspace(qp, kp)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda") if need else None
    return qp, kp, q, k, v, o, lse, ws


def limited(limit, fn):
    """(status word, seconds) of a call under a limit."""
    torch.cuda.synchronize()
    B.ulysses_selftest_attention_wait_limit(limit)
    t0 = time.perf_counter()
    fn()
    status = B.ulysses_device_status()
    B.ulysses_selftest_attention_wait_limit(DEFAULT)
    return status, time.perf_counter() - t0


@pytest.mark.parametrize("shape,cap", FORWARD, ids=IDS)
def test_forward_gives_up_and_works_again(shape, cap):
    qp, kp, q, k, v, o, lse, ws = make(shape, cap, torch.bfloat16)
    call = lambda: B.ulysses_attention(qp, kp, q, k, v, o, lse, scale=0.1, workspace=ws)
    call()
    assert B.ulysses_device_status() == 0
    want = [x.clone() for x in o + lse]
    status, seconds = limited(0, call)
    assert status == 1 and seconds < 1.0, (status, seconds)  # no wait for a copy ran out behind it
    call()
    assert B.ulysses_device_status() == 0
    assert all(torch.equal(x, y) for x, y in zip(want, o + lse))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("ragged", [False, True], ids=["full", "ragged"])
@pytest.mark.parametrize("shape,cap", [((1, 2, 20_000, 20_000, [1], 1, 128), 2),
                                       ((1, 2, 20_000, 20_000, [1], 1, 64), 2),
                                       ((1, 2, 20_000, 20_000, [4], 1, 128), 0)],
                         ids=["128", "64", "stealing"])
def test_backward_gives_up_and_works_again(shape, cap, ragged, dtype):
    qp, kp, q, k, v, o, lse, ws = make(shape, cap, dtype)
    kw = {"scale": 0.1}
    if ragged:
        kw |= {"kv_lens": torch.tensor([19_990, 15_001], dtype=torch.int32, device="cuda"),
               "causal": True,
               "q_start": torch.tensor([-7, 300], dtype=torch.int32, device="cuda")}
    B.ulysses_attention(qp, kp, q, k, v, o, lse, workspace=ws, **kw)
    grads = [[torch.zeros_like(x) for x in t] for t in (q, k, v)]
    bws = torch.empty(B.ulysses_attention_backward_workspace(qp, kp), dtype=torch.uint8,
                      device="cuda")
    call = lambda: B.ulysses_attention_backward(qp, kp, *grads, q, k, v, o, lse, o, workspace=bws, **kw)
    call()
    assert B.ulysses_device_status() == 0
    want = [x.clone() for t in grads for x in t]
    status, seconds = limited(0, call)
    assert status == 1 and seconds < 1.0, (status, seconds)
    call()
    assert B.ulysses_device_status() == 0
    assert all(torch.equal(x, y) for x, y in zip(want, [x for t in grads for x in t]))


def test_a_limit_counts_only_time_in_which_nothing_moves():
    """Units of several ms, and runs of units without work of more, under a limit of 1 ms."""
    qp, kp, q, k, v, o, lse, ws = make((1, 1, 700, 600_000, [1], 64, 64), 4, torch.bfloat16)
    assert ws is None  # not split: a unit walks all keys
    status, seconds = limited(1000, lambda: B.ulysses_attention(qp, kp, q, k, v, o, lse, scale=0.1))
    assert status == 0 and seconds > 0.05, (status, seconds)

    qp, kp, q, k, v, o, lse, ws = make((1, 1, 600, 1_000_000, [2], 1, 64), 1, torch.bfloat16)
    grads = [[torch.zeros_like(x) for x in t] for t in (q, k, v)]
    bws = torch.empty(B.ulysses_attention_backward_workspace(qp, kp), dtype=torch.uint8,
                      device="cuda")
    few = torch.full((1,), 1000, dtype=torch.int32, device="cuda")
    for lens in (None, few):
        status, seconds = limited(1000, lambda: B.ulysses_attention_backward(
            qp, kp, *grads, q, k, v, o, lse, o, scale=0.1, workspace=bws, kv_lens=lens))
        assert status == 0 and seconds > 0.005, (status, seconds)


def test_limits_are_checked():
    with pytest.raises(B.UlyssesError) as e:
        B.ulysses_selftest_attention_wait_limit(DEFAULT + 1)
    assert e.value.status == B.ULY_EINVAL
