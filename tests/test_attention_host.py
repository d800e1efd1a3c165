"""Refusals of the attention calls: every check that comes before the device is touched, with
addresses that are never read (host only)."""
import os

import pytest

from ulysses_sequence_all_gb300 import binding as B
from ulysses_sequence_all_gb300 import build as build_mod


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(B.LIBRARY):
        build_mod.build_library()


def plans(q=(1, 2, [64], [4], 64, "bfloat16"), kv=(1, 2, [128], [2], 64, "bfloat16")):
    return B.ulysses_plan(*q), B.ulysses_plan(*kv)


MB = 1 << 20


def status(qp, kp, **kw):
    """Status of a call with distinct made-up addresses, overridden by kw."""
    W = qp.W
    at = {name: [(16 * i + r + 1) * MB for r in range(W)]
          for i, name in enumerate(("q", "k", "v", "out", "lse"))}
    args = dict(at, scale=0.125, causal=False, kv_lens=None, q_start=None)
    args.update(kw)
    try:
        B.ulysses_attention(qp, kp, args.pop("q"), args.pop("k"), args.pop("v"), args.pop("out"),
                            args.pop("lse"), stream=0, **args)
    except B.UlyssesError as e:
        return e.status
    return B.ULY_OK


@pytest.mark.parametrize("change", [
    {"kv": (1, 2, [128], [3], 64, "bfloat16")},             # 4 query heads over 3
    {"kv": (1, 2, [128], [8], 64, "bfloat16")},             # more key heads than query heads
    {"kv": (1, 2, [128], [2], 72, "bfloat16")},             # other head dimension
    {"kv": (1, 3, [128], [2], 64, "bfloat16")},             # other batch
    {"kv": (1, 2, [128], [2], 64, "float16")},              # other type
    {"kv": (2, 2, [64, 64], [1, 1], 64, "bfloat16")},       # other rank count
    {"q": (1, 2, [64], [4], 64, "float32"), "kv": (1, 2, [64], [4], 64, "float32")},
    {"q": (1, 2, [64], [4], 64, "float8_e4m3fn"), "kv": (1, 2, [64], [4], 64, "float8_e4m3fn")},
    {"q": (1, 2, [64], [4], 136, "bfloat16"), "kv": (1, 2, [64], [4], 136, "bfloat16")},
    {"q": (1, 2, [64], [65], 64, "bfloat16"), "kv": (1, 2, [64], [1], 64, "bfloat16")},
    {"q": (2, 1, [9, 9], [4, 2], 64, "bfloat16"), "kv": (2, 1, [9, 9], [1, 2], 64, "bfloat16")},
    {"kv": (1, 2, [2 ** 31], [2], 64, "bfloat16")},         # past tensor-map coordinates
    {"kv": (1, 2, [2 ** 26 + 1], [2], 64, "bfloat16")},     # more keys than a unit walks
    {"q": (1, 2, [2 ** 25 + 1], [4], 64, "bfloat16")},      # more rows: two heads share keys
])
def test_plans_that_do_not_go_together(change):
    assert status(*plans(**change)) == B.ULY_EINVAL


@pytest.mark.parametrize("kw,want", [
    ({"scale": 0.0}, B.ULY_EINVAL),
    ({"scale": -1.0}, B.ULY_EINVAL),
    ({"scale": float("nan")}, B.ULY_EINVAL),
    ({"scale": float("inf")}, B.ULY_EINVAL),
    ({"causal": 2}, B.ULY_EINVAL),
    ({"q_start": 90 * MB}, B.ULY_EINVAL),                    # a start without the causal mask
    ({"q_start": 90 * MB + 2, "causal": True}, B.ULY_EALIGN),
    ({"kv_lens": 90 * MB + 1}, B.ULY_EALIGN),
    ({"q": [MB + 8]}, B.ULY_EALIGN),
    ({"lse": [90 * MB + 4]}, B.ULY_EALIGN),
    ({"q": [None]}, B.ULY_EINVAL),
    ({"v": [None]}, B.ULY_EINVAL),
    ({"out": [None]}, B.ULY_EINVAL),
    ({"lse": [None]}, B.ULY_EINVAL),
    ({"out": [MB]}, B.ULY_EOVERLAP),                         # the queries' own place
    ({"lse": [49 * MB + 256]}, B.ULY_EOVERLAP),              # inside the output
    ({"kv_lens": 49 * MB + 256}, B.ULY_EOVERLAP),
])
def test_refused_arguments(kw, want):
    assert status(*plans(), **kw) == want


def test_null_plans_and_workspace_query():
    qp, kp = plans()
    import ctypes
    lib, n = B.library(), ctypes.c_size_t()
    ptrs = B._ptrs([MB])
    for a, b in ((None, kp), (qp, None)):
        assert lib.ulysses_attention(a, b, ptrs, ptrs, ptrs, ptrs, ptrs, None, None, 0, 0.125, None,
                                     0, None) == B.ULY_EINVAL
        assert lib.ulysses_attention_workspace(a, b, ctypes.byref(n)) == B.ULY_EINVAL
    assert lib.ulysses_attention_workspace(qp, kp, None) == B.ULY_EINVAL
    assert lib.ulysses_attention(qp, kp, None, ptrs, ptrs, ptrs, ptrs, None, None, 0, 0.125, None, 0,
                                 None) == B.ULY_EINVAL


def backward_status(qp, kp, **kw):
    """The same for the backward, with a workspace that is long enough unless overridden."""
    import ctypes
    at = {name: [(16 * i + 1) * MB]
          for i, name in enumerate(("q", "k", "v", "o", "lse", "go", "dq", "dk", "dv"))}
    a = dict(at, scale=0.125, causal=0, kv_lens=0, q_start=0, ws=200 * MB,
             ws_bytes=B.ulysses_attention_backward_workspace(qp, kp))
    a.update(kw)
    ptr = lambda x: None if a[x] is None else B._ptrs(a[x])
    return B.library().ulysses_attention_backward(
        qp, kp, *map(ptr, ("dq", "dk", "dv", "q", "k", "v", "o", "lse", "go")),
        ctypes.c_void_p(a["kv_lens"]), ctypes.c_void_p(a["q_start"]), a["causal"], a["scale"],
        ctypes.c_void_p(a["ws"]), a["ws_bytes"], None)


@pytest.mark.parametrize("kw,want", [
    ({"scale": 0.0}, B.ULY_EINVAL),
    ({"causal": -1}, B.ULY_EINVAL),
    ({"q_start": 300 * MB}, B.ULY_EINVAL),
    ({"kv_lens": 300 * MB + 2}, B.ULY_EALIGN),
    ({"ws": 0}, B.ULY_EINVAL),
    ({"ws_bytes": 64}, B.ULY_EINVAL),
    ({"ws": 200 * MB + 4}, B.ULY_EALIGN),
    ({"ws": MB}, B.ULY_EOVERLAP),
    ({"go": [None]}, B.ULY_EINVAL),
    ({"dk": None}, B.ULY_EINVAL),
    ({"lse": [None]}, B.ULY_EINVAL),
    ({"o": [MB + 2]}, B.ULY_EALIGN),
    ({"dq": [MB]}, B.ULY_EOVERLAP),                          # the queries' own place
    ({"dv": [113 * MB + 16]}, B.ULY_EOVERLAP),               # inside dk
])
def test_backward_refused_arguments(kw, want):
    assert backward_status(*plans(), **kw) == want


def test_backward_plans_that_do_not_go_together():
    qp, kp = plans(kv=(1, 2, [128], [3], 64, "bfloat16"))
    with pytest.raises(B.UlyssesError) as e:
        B.ulysses_attention_backward_workspace(qp, kp)
    assert e.value.status == B.ULY_EINVAL
    assert B.library().ulysses_attention_backward(*(None,) * 13, 0, 0.125, None, 0, None) == B.ULY_EINVAL
