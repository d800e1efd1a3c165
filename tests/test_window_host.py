"""Refusals of attention with a window, which need no GPU."""
import ctypes

import pytest
import torch

from ulysses_sequence_all_gb300 import autograd as A
from ulysses_sequence_all_gb300 import binding as B

BASE = [0x10000000 * i for i in range(1, 13)]
N, S = 0x2_00000000, 0x2_00100000


def plan(b=2, s=300, heads=(4, 2), d=64, dtype="bfloat16"):
    W = len(heads)
    return B.ulysses_plan(W, b, [s] + [0] * (W - 1), list(heads), d, dtype)


def at(base, step=0x100000):
    return (ctypes.c_void_p * 2)(base, base + step)


def forward(q=None, kv=None, window=10, sinks=0, scale=0.125, lens=N, start=S, ptrs=None, ws=BASE[6],
            ws_bytes=1 << 28):
    p = [at(x) for x in BASE[:5]]
    for i, x in (ptrs or {}).items():
        p[i] = x
    return B.library().ulysses_attention_window(q or plan(), kv or plan(heads=(2, 1)), *p, lens, start, window,
                                                sinks, scale, ws, ws_bytes, None)


BAD = {
    "no window": dict(window=0), "a window below 0": dict(window=-3), "sinks below 0": dict(sinks=-1),
    "scale 0": dict(scale=0.0), "another batch": dict(kv=plan(b=3, heads=(2, 1))),
    "another d": dict(kv=plan(heads=(2, 1), d=72)), "d above 128": dict(q=plan(d=136), kv=plan(heads=(2, 1), d=136)),
    "fp32": dict(q=plan(dtype="float32"), kv=plan(heads=(2, 1), dtype="float32")),
    "heads that no group makes": dict(q=plan(heads=(3, 3))), "no queries": dict(ptrs={0: None}),
}


@pytest.mark.parametrize("rows", [300, 1], ids=["many", "few"])
@pytest.mark.parametrize("what", BAD)
def test_refuses(what, rows):
    kw = dict(BAD[what])
    if rows == 1 and "q" not in kw:
        kw["q"] = plan(s=1)
    assert forward(**kw) == B.ULY_EINVAL


@pytest.mark.parametrize("rows", [300, 1], ids=["many", "few"])
def test_refuses_misaligned_and_overlap(rows):
    q = plan(s=rows)
    assert forward(q=q, lens=N + 2) == B.ULY_EALIGN
    assert forward(q=q, ptrs={1: at(BASE[1] + 8)}) == B.ULY_EALIGN
    assert forward(q=q, ptrs={3: at(BASE[0])}) == B.ULY_EOVERLAP
    assert forward(q=q, lens=BASE[3]) == B.ULY_EOVERLAP


def test_backward_refuses():
    call = lambda window=10, sinks=0, scale=0.125: B.library().ulysses_attention_window_backward(
        plan(), plan(heads=(2, 1)), *[at(x) for x in BASE[:9]], N, S, window, sinks, scale, BASE[9], 1 << 28, None)
    for kw in (dict(window=0), dict(window=-1), dict(sinks=-1), dict(scale=-1.0)):
        assert call(**kw) == B.ULY_EINVAL


def test_workspace_refuses():
    n = ctypes.c_size_t()
    for name in ("ulysses_attention_window_workspace", "ulysses_attention_window_backward_workspace"):
        fn = getattr(B.library(), name)
        for q in (plan(), plan(s=1)):
            assert fn(q, plan(heads=(2, 1)), 0, 0, ctypes.byref(n)) == B.ULY_EINVAL
            assert fn(q, plan(heads=(2, 1)), 5, -1, ctypes.byref(n)) == B.ULY_EINVAL
            assert fn(q, plan(b=1, heads=(2, 1)), 5, 0, ctypes.byref(n)) == B.ULY_EINVAL
            assert fn(q, None, 5, 0, ctypes.byref(n)) == B.ULY_EINVAL
            assert fn(q, plan(heads=(2, 1)), 5, 0, None) == B.ULY_EINVAL


def test_first_tokens_without_a_window():
    p = plan()
    with pytest.raises(ValueError, match="sinks"):
        A.attention(p, p, [], [], [], sinks=4)
    with pytest.raises(ValueError, match="kv_lens"):
        B.ulysses_attention_window(p, p, [], [], [], [], [], 1.0, 5, kv_lens=torch.zeros(2, dtype=torch.int32))
