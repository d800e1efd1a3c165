"""Refusals of the paged cache's calls, which need no GPU."""
import ctypes

import pytest
import torch

from ulysses_sequence_all_gb300 import binding as B

Q, K, V, O, L, WS = (0x10000000 * i for i in range(1, 7))
T, N, S = 0x80000000, 0x80100000, 0x80200000


def plan(b=2, s=1, heads=(4, 2), d=64, dtype="bfloat16"):
    W = len(heads)
    return B.ulysses_plan(W, b, [s] + [0] * (W - 1), list(heads), d, dtype)


def at(base, W=2, step=0x100000):
    return (ctypes.c_void_p * W)(*[base + r * step for r in range(W)])


def paged(q=None, cache=None, ptrs=None, table=T, pages=4, lens=N, start=S, window=0, sinks=0, scale=0.125,
          ws=WS, ws_bytes=1 << 30):
    q = q or plan()
    cache = cache or plan(b=8, s=16, heads=(2, 1))
    p = dict(q=at(Q), k=at(K), v=at(V), o=at(O), lse=at(L))
    p.update(ptrs or {})
    return B.library().ulysses_attention_paged(q, cache, p["q"], p["k"], p["v"], p["o"], p["lse"], table,
                                               pages, lens, start, window, sinks, scale, ws, ws_bytes, None)


def append(new=None, cache=None, ptrs=None, table=T, pages=4, starts=N, counts=S):
    new = new or plan(heads=(2, 1))
    cache = cache or plan(b=8, s=16, heads=(2, 1))
    p = dict(k=at(K), v=at(V), kc=at(Q), vc=at(O))
    p.update(ptrs or {})
    return B.library().ulysses_cache_append(new, cache, p["k"], p["v"], p["kc"], p["vc"], table, pages,
                                            starts, counts, None)


PAGED = {
    "another d": dict(q=plan(d=72)), "another dtype": dict(q=plan(dtype="float16")),
    "fp32": dict(q=plan(dtype="float32"), cache=plan(b=8, s=16, heads=(2, 1), dtype="float32")),
    "d above 128": dict(q=plan(d=136), cache=plan(b=8, s=16, heads=(2, 1), d=136)),
    "ranks": dict(q=plan(heads=(4,))), "heads that no group makes": dict(q=plan(heads=(3, 3))),
    "a rank without its keys": dict(q=plan(heads=(2, 4))), "a page of 12": dict(cache=plan(b=8, s=12, heads=(2, 1))),
    "groups of 65": dict(q=plan(heads=(130, 65))), "no table": dict(table=None),
    "a table of nothing": dict(pages=0), "room past 2^29": dict(pages=2 ** 29 // 16 + 1),
    "no lengths": dict(lens=None), "a window below 0": dict(window=-1), "sinks below 0": dict(sinks=-1),
    "scale 0": dict(scale=0.0), "scale inf": dict(scale=float("inf")), "scale nan": dict(scale=float("nan")),
    "no queries": dict(ptrs=dict(q=None)), "a null rank": dict(ptrs=dict(k=(ctypes.c_void_p * 2)(K, None))),
}


@pytest.mark.parametrize("what", PAGED)
def test_paged_refuses(what):
    assert paged(**PAGED[what]) == B.ULY_EINVAL


@pytest.mark.parametrize("kw", [dict(table=T + 2), dict(lens=N + 1), dict(start=S + 3),
                                dict(ptrs=dict(v=at(V + 8))), dict(ptrs=dict(lse=at(L + 4)))])
def test_paged_refuses_misaligned(kw):
    assert paged(**kw) == B.ULY_EALIGN


@pytest.mark.parametrize("kw", [dict(ptrs=dict(o=at(Q))), dict(ptrs=dict(o=at(K + 0x40))), dict(table=O),
                                dict(lens=L), dict(ptrs=dict(lse=at(O)))])
def test_paged_refuses_overlap(kw):
    assert paged(**kw) == B.ULY_EOVERLAP


APPEND = {
    "another d": dict(new=plan(heads=(2, 1), d=72)), "another dtype": dict(new=plan(heads=(2, 1), dtype="float16")),
    "other heads": dict(new=plan(heads=(1, 2))), "ranks": dict(new=plan(heads=(2,))),
    "a page of 12": dict(cache=plan(b=8, s=12, heads=(2, 1))), "no table": dict(table=None),
    "no starts": dict(starts=None), "a table of nothing": dict(pages=0),
    "room past 2^29": dict(pages=2 ** 29 // 16 + 1), "no keys": dict(ptrs=dict(k=None)),
}


@pytest.mark.parametrize("what", APPEND)
def test_append_refuses(what):
    assert append(**APPEND[what]) == B.ULY_EINVAL


def test_append_refuses_misaligned_and_overlap():
    assert append(table=T + 2) == B.ULY_EALIGN
    assert append(counts=S + 2) == B.ULY_EALIGN
    assert append(ptrs=dict(kc=at(Q + 8))) == B.ULY_EALIGN
    assert append(ptrs=dict(kc=at(K))) == B.ULY_EOVERLAP
    assert append(ptrs=dict(vc=at(Q))) == B.ULY_EOVERLAP
    assert append(starts=Q) == B.ULY_EOVERLAP


def test_null_plans():
    n = ctypes.c_size_t()
    lib = B.library()
    assert lib.ulysses_attention_paged_workspace(None, plan(), ctypes.byref(n)) == B.ULY_EINVAL
    assert lib.ulysses_attention_paged_workspace(plan(), plan(heads=(2, 1)), None) == B.ULY_EINVAL
    assert lib.ulysses_cache_append(None, plan(), None, None, None, None, None, 0, None, None, None) == B.ULY_EINVAL


@pytest.mark.parametrize("table", [torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3)])
def test_the_binding_looks_at_the_table(table):
    with pytest.raises(ValueError, match="page_table"):
        B.ulysses_cache_append(plan(heads=(2, 1)), plan(b=8, s=16, heads=(2, 1)), [], [], [], [], table, None)
