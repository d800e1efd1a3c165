"""A plan's CTA cap (ulysses_plan_set_max_ctas) on the attention calls: every kernel they launch stays
within it, and it changes no bit of the results."""
import ctypes

import pytest
import torch

from test_gpu_attention import attend, inputs, plans
from test_gpu_attention_backward import given, gradients
from ulysses_sequence_all_gb300 import binding as B

pytestmark = pytest.mark.gpu

# W, b, sq, skv, kv heads, group, d: rows whose keys are split and joined; single tokens; many units
SHAPES = [(2, 2, 300, 2500, [1, 2], 2, 128), (1, 3, 1, 5000, [2], 4, 64),
          (1, 2, 1500, 900, [4], 1, 64)]
IDS = ["tiles", "token", "units"]


@pytest.fixture(autouse=True)
def no_timeout():
    yield
    assert B.ulysses_device_status() == 0


class KernelNode(ctypes.Structure):
    """The start of the driver's CUDA_KERNEL_NODE_PARAMS, with room for the rest."""
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3),
                ("smem", ctypes.c_uint), ("rest", ctypes.c_void_p * 8)]


def launches(fn):
    """CTAs of each kernel that fn queues, from a capture of its stream that is not replayed."""
    cu = ctypes.CDLL("libcuda.so.1")
    side = torch.cuda.Stream()
    raw = ctypes.c_void_p(side.cuda_stream)
    graph, n = ctypes.c_void_p(), ctypes.c_size_t()
    torch.cuda.synchronize()
    assert cu.cuStreamBeginCapture_v2(raw, 2) == 0  # relaxed
    try:
        with torch.cuda.stream(side):
            fn()
    finally:
        assert cu.cuStreamEndCapture(raw, ctypes.byref(graph)) == 0
    assert cu.cuGraphGetNodes(graph, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cu.cuGraphGetNodes(graph, nodes, ctypes.byref(n)) == 0
    out = []
    for node in nodes:
        kind, p = ctypes.c_int(), KernelNode()
        assert cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        if kind.value == 0:
            assert cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)) == 0
            out.append(p.grid[0] * p.grid[1] * p.grid[2])
    cu.cuGraphDestroy(graph)
    return out


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_every_launch_stays_within_the_cap(shape):
    qp, kp = plans(*shape, torch.bfloat16)
    q, k, v = inputs(*shape, torch.bfloat16)
    o, lse = [torch.empty_like(x) for x in q], None
    lse = [torch.empty((x.shape[0], x.shape[2], x.shape[1]), device="cuda") for x in q]
    grads = [[torch.empty_like(x) for x in t] for t in (q, k, v)]
    bws = torch.empty(B.ulysses_attention_backward_workspace(qp, kp), dtype=torch.uint8,
                      device="cuda")

    def calls(ws):
        B.ulysses_attention(qp, kp, q, k, v, o, lse, scale=0.1, workspace=ws)
        B.ulysses_attention_backward(qp, kp, *grads, q, k, v, o, lse, q, scale=0.1, workspace=bws)

    for cap in (0, 1, 3, 200):
        B.ulysses_plan_set_max_ctas(qp, cap)
        need = B.ulysses_attention_workspace(qp, kp)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
        calls(ws)  # (kernels are loaded before the capture)
        got = launches(lambda: calls(ws))
        assert len(got) == (5 if need else 4)
        if cap:
            assert max(got) <= cap, got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_a_cap_changes_no_bit(shape, dtype):
    qp, kp = plans(*shape, dtype)
    q, k, v = inputs(*shape, dtype, seed=8)
    o, lse, go = given(q, k, v, 0.1)
    runs = []
    for cap in (0, 1, 7, 151, 500):
        B.ulysses_plan_set_max_ctas(qp, cap)
        a = attend(qp, kp, q, k, v, 0.1)
        b = gradients(qp, kp, q, k, v, o, lse, go, 0.1)
        runs.append([*a[0], *a[1], *b[0], *b[1], *b[2]])
    for other in runs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(runs[0], other))
