"""Gradients of gradients through the differentiable forms: the relayout's is the relayout again; the others
have a first derivative only, and differentiating it raises instead of leaving out what went through them."""
import pytest
import torch

from ulysses_sequence_all_gb300 import autograd as A
from ulysses_sequence_all_gb300 import binding as B

pytestmark = pytest.mark.gpu

W, b, d = 2, 1, 64
SEQ, HEADS = [9, 8], [1, 2]
N, S = 3, 17


def leaves(*shapes):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    return [torch.randn(s, generator=gen, device="cuda").bfloat16().requires_grad_() for s in shapes]


def seq(*mid):
    return leaves(*[(b, s, *mid, N, d) for s in SEQ])


def heads():
    return leaves(*[(b, S, n, d) for n in HEADS])


def rms():
    return torch.ones(2, d, device="cuda", requires_grad=True)


FORMS = {
    "qk_fused": (lambda plan, x: A.qk_fused(plan, x, x, rms(), 1e-6, 1e4)[0], seq),
    "qkv_fused": (lambda plan, x: A.qkv_fused(plan, x, rms(), 1e-6, 1e4)[0], lambda: seq(3)),
    "packed_fused": (lambda plan, x: A.packed_fused(plan, x, 4, 0, 1, rms(), 1e-6, 1e4)[0],
                     lambda: seq(4)),
    "attention": (lambda plan, x: A.attention(plan, plan, x, x, x), heads),
}


@pytest.mark.parametrize("form", FORMS)
def test_a_second_derivative_raises(form):
    fn, make = FORMS[form]
    plan = B.ulysses_plan(W, b, SEQ, HEADS, d, "bfloat16")
    xs = make()
    ys = fn(plan, xs)
    first = torch.autograd.grad([y.float().square().sum() for y in ys], xs, create_graph=True)
    loss = sum(g.float().square().sum() + x.float().square().sum() for g, x in zip(first, xs))
    with pytest.raises(RuntimeError, match="once_differentiable"):
        loss.backward()


@pytest.mark.parametrize("mode", [0, 1])
def test_the_relayout_can_be_differentiated_again(mode):
    """y = P x: the gradient of |y|^2 is 2 x, that of |2 x|^2 + |x|^2 is 8 x + 2 x."""
    plan = B.ulysses_plan(W, b, SEQ, HEADS, d, "bfloat16")
    xs = seq() if mode == 0 else heads()
    ys = A.a2a_4d(plan, xs, mode)
    first = torch.autograd.grad([y.float().square().sum() for y in ys], xs, create_graph=True)
    sum(g.float().square().sum() + x.float().square().sum() for g, x in zip(first, xs)).backward()
    for x, g in zip(xs, first):
        assert torch.equal(g.detach(), 2 * x.detach())
        assert torch.allclose(x.grad.float(), 10 * x.detach().float(), rtol=2.0 ** -8, atol=0)
