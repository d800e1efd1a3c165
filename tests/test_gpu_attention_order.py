"""The backward's kernels overlap: the last one starts before the one in front of it has ended. One
workspace serving calls on other values in turn, each over what the last call left in it, with nothing
between them: the bits of every call are those that it gives alone."""
import pytest
import torch

from test_gpu_attention import inputs, plans
from test_gpu_attention_backward import given
from ulysses_sequence_all_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("shape", [(1, 2, 700, 500, [3], 2, 128), (2, 1, 64, 130, [1, 1], 1, 64),
                                   (1, 4, 2000, 2000, [8], 1, 64)], ids=["medium", "small", "large"])
def test_one_workspace_for_calls_in_turn(shape, dtype):
    qp, kp = plans(*shape, dtype)
    sets = []
    for seed in (1, 2, 3):
        q, k, v = inputs(*shape, dtype, seed=seed)
        o, lse, go = given(q, k, v, 0.1, seed)
        sets.append((q, k, v, o, lse, go))
    need = B.ulysses_attention_backward_workspace(qp, kp)

    def call(which, ws):
        q, k, v, o, lse, go = sets[which]
        g = [[torch.empty_like(x) for x in t] for t in (q, k, v)]
        B.ulysses_attention_backward(qp, kp, *g, q, k, v, o, lse, go, scale=0.1, workspace=ws)
        return [x for t in g for x in t]

    alone = []
    for i in range(3):
        torch.cuda.synchronize()
        alone.append(call(i, torch.full((need,), 255, dtype=torch.uint8, device="cuda")))
    torch.cuda.synchronize()
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(8):
        got = [call(i, ws) for i in (0, 1, 2, 0, 2, 1)]
        for i, g in zip((0, 1, 2, 0, 2, 1), got):
            assert all(torch.equal(x, y) for x, y in zip(alone[i], g))
    assert B.ulysses_device_status() == 0
