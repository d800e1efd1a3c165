"""Lists that have fewer tensors than the plan has ranks are refused by the binding: the library reads one
address a rank from them."""
import pytest

from ulysses_sequence_all_gb300 import binding as B

W = 3


def plan(heads=2, s=16):
    return B.ulysses_plan(W, 2, [s] + [0] * (W - 1), [heads] * W, 64, "bfloat16")


def lists(n, short):
    """n lists of W addresses, one of them an entry short."""
    return [[0x1000000 * (W * i + r + 1) for r in range(W - (i == short))] for i in range(n)]


CALLS = {  # lists, the call that takes them
    "a2a": (2, lambda p, x: B.ulysses_a2a_4d(p, 0, *x, stream=0)),
    "engine": (2, lambda p, x: B.ulysses_a2a_4d_engine(p, 0, B.ULY_ENGINE_TMA, *x, stream=0)),
    "qk fused": (4, lambda p, x: B.ulysses_a2a_4d_qk_fused(p, *x, 16, 1e-6, 1e4, stream=0)),
    "qkv fused": (4, lambda p, x: B.ulysses_a2a_4d_qkv_fused(p, *x, 16, 1e-6, 1e4, stream=0)),
    "packed fused": (4, lambda p, x: B.ulysses_a2a_4d_packed_fused(p, 3, 0, 1, 384, x[0], x[1:], 16, 1e-6, 1e4,
                                                                   stream=0)),
    "attention": (5, lambda p, x: B.ulysses_attention(p, p, *x, 0.1, stream=0)),
    "attention backward": (9, lambda p, x: B.ulysses_attention_backward(p, p, *x, 0.1, stream=0)),
    "window": (5, lambda p, x: B.ulysses_attention_window(p, p, *x, 0.1, 8, stream=0)),
    "window backward": (9, lambda p, x: B.ulysses_attention_window_backward(p, p, *x, 0.1, 8, stream=0)),
    "host": (4, lambda p, x: B.ulysses_a2a_4d_host(p, 0, *x, stream=0)),
}


@pytest.mark.parametrize("what", CALLS)
def test_short_lists_are_refused(what):
    n, call = CALLS[what]
    for short in range(n):
        with pytest.raises(ValueError, match="ranks"):
            call(plan(), lists(n, short))


@pytest.mark.parametrize("short", range(5))
def test_short_lists_over_pages(short, monkeypatch):
    monkeypatch.setattr(B, "_page_table", lambda x, b: (0x10, 4))
    monkeypatch.setattr(B, "_counts", lambda x, b, what: 0x10)
    with pytest.raises(ValueError, match="ranks"):
        B.ulysses_attention_paged(plan(), plan(), *lists(5, short), None, None, 0.1, stream=0)
    if short < 4:
        with pytest.raises(ValueError, match="ranks"):
            B.ulysses_cache_append(plan(), plan(), *lists(4, short), None, None, stream=0)
