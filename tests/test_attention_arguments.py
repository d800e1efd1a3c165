"""What the Python forms of the attention calls refuse before anything is launched, so that no kernel
gets an address or a length that it cannot read (host only: the tensors here are no device's, or claim to
be one)."""
import os

import pytest
import torch

from ulysses_sequence_all_gb300 import autograd as A
from ulysses_sequence_all_gb300 import binding as B
from ulysses_sequence_all_gb300 import build as build_mod

b, W = 3, 2


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(B.LIBRARY):
        build_mod.build_library()


@pytest.fixture
def plan():
    return B.ulysses_plan(W, b, [4, 5], [2, 1], 64, "bfloat16")


class Device:
    """A tensor of the host that says it is the device's."""

    def __init__(self, t):
        self.t = t
        self.is_cuda, self.device = True, "cuda:0"

    def __getattr__(self, name):
        return getattr(self.t, name)


COUNTS = [torch.zeros(b, dtype=torch.int32),                      # on the host
          Device(torch.zeros(b, dtype=torch.int64)),              # pairs of int32 to the kernels
          Device(torch.zeros(b, dtype=torch.float32)),
          Device(torch.zeros(b - 1, dtype=torch.int32)),          # read past its end
          Device(torch.zeros(b + 1, dtype=torch.int32)),
          Device(torch.zeros(2 * b, dtype=torch.int32)[::2])]
IDS = ["host", "int64", "float", "short", "long", "strided"]


@pytest.mark.parametrize("counts", COUNTS, ids=IDS)
@pytest.mark.parametrize("which", ["kv_lens", "q_start"])
def test_counts_that_the_binding_refuses(plan, counts, which):
    MB = 1 << 20
    at = [[(16 * i + r + 1) * MB for r in range(W)] for i in range(9)]
    kw = {which: counts, "causal": True, "scale": 0.125}
    with pytest.raises(ValueError, match=which):
        B.ulysses_attention(plan, plan, *at[:5], stream=0, **kw)
    with pytest.raises(ValueError, match=which):
        B.ulysses_attention_backward(plan, plan, *at, stream=0, **kw)


def test_counts_of_the_differentiable_form():
    """Taken from the host, from lists and in other whole types; refused when there are not b."""
    cpu = torch.device("cpu")
    assert A._counts(None, b, cpu, "kv_lens") is None
    for given in ([1, 2, 3], torch.tensor([1, 2, 3]), torch.tensor([1, 2, 3], dtype=torch.uint8),
                  torch.tensor([1, 0, 2, 0, 3, 0])[::2]):
        x = A._counts(given, b, cpu, "kv_lens")
        assert x.dtype == torch.int32 and x.is_contiguous() and x.tolist() == [1, 2, 3]
    far = A._counts(torch.tensor([2 ** 40, -2 ** 40, 7]), b, cpu, "q_start")
    assert far.tolist() == [2 ** 31 - 1, -2 ** 31, 7]
    for bad in ([1, 2], torch.zeros(b + 1, dtype=torch.int32), torch.zeros(b), 5):
        with pytest.raises(ValueError, match="kv_lens"):
            A._counts(bad, b, cpu, "kv_lens")


def heads(dtype=torch.bfloat16, S=9, n=(2, 1), d=64):
    return [Device(torch.zeros(b, S, m, d, dtype=dtype)) for m in n]


@pytest.mark.parametrize("bad", [[torch.zeros(b, 9, m, 64, dtype=torch.bfloat16) for m in (2, 1)],
                                 heads(S=8), heads(dtype=torch.float16), heads(n=(1, 2)),
                                 heads(n=(2,)), heads(d=72)],
                         ids=["host", "short", "type", "ranks", "missing", "d"])
@pytest.mark.parametrize("which", [0, 1, 2])
def test_tensors_that_the_differentiable_form_refuses(plan, bad, which):
    args = [heads(), heads(), heads()]
    args[which] = bad
    with pytest.raises(ValueError, match="qkv"[which]):
        A.attention(plan, plan, *args)
