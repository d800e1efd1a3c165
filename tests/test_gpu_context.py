"""The calls leave the thread's CUDA context as they find it: a caller's own stays current, and a thread
without one gets the device's."""
import ctypes
import threading

import pytest
import torch

from ulysses_sequence_all_gb300 import binding as B

pytestmark = pytest.mark.gpu


def in_thread(fn):
    out = []

    def body():
        try:
            out.append((True, fn()))
        except BaseException as e:  # carried over to the test's thread
            out.append((False, e))

    t = threading.Thread(target=body)
    t.start()
    t.join()
    ok, value = out[0]
    if not ok:
        raise value
    return value


def current(cu):
    ctx = ctypes.c_void_p()
    assert cu.cuCtxGetCurrent(ctypes.byref(ctx)) == 0
    return ctx.value


def test_a_context_of_the_caller_stays_current():
    torch.cuda.synchronize()  # the device's own context is there
    cu = ctypes.CDLL("libcuda.so.1")
    plan = B.ulysses_plan(1, 1, [300], [2], 64, "bfloat16")

    def body():
        ctx = ctypes.c_void_p()
        assert cu.cuCtxCreate_v2(ctypes.byref(ctx), 0, 0) == 0
        try:
            assert current(cu) == ctx.value
            B.ulysses_attention_workspace(plan, plan)
            B.ulysses_plan_auto_engine(plan)
            return current(cu) == ctx.value
        finally:
            cu.cuCtxDestroy_v2(ctx)

    assert in_thread(body)


def test_a_thread_without_a_context_gets_one():
    plan = B.ulysses_plan(1, 1, [300], [2], 64, "bfloat16")
    q = torch.randn(1, 300, 2, 64, device="cuda").bfloat16()
    o, lse = torch.empty_like(q), torch.empty(1, 2, 300, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    in_thread(lambda: B.ulysses_attention(plan, plan, [q], [q], [q], [o], [lse], scale=0.125,
                                          workspace=None, stream=stream))
    torch.cuda.synchronize()
    assert bool(o.isfinite().all()) and B.ulysses_device_status() == 0
