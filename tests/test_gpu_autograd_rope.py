"""The fused forms' gradient is taken with the rotation of their forward: a plan whose pair layout or position
axes were changed in between is refused, one whose settings are back as they were is not."""
import pytest
import torch

from ulysses_sequence_all_gb300 import autograd as A
from ulysses_sequence_all_gb300 import binding as B

pytestmark = pytest.mark.gpu

W, b, d = 2, 1, 64
SEQ, HEADS = [9, 8], [1, 2]
N = 3

FORMS = {
    "qk_fused": ((), lambda plan, x, w: A.qk_fused(plan, x, x, w, 1e-6, 1e4)[0]),
    "qkv_fused": ((3,), lambda plan, x, w: A.qkv_fused(plan, x, w, 1e-6, 1e4)[0]),
    "packed_fused": ((4,), lambda plan, x, w: A.packed_fused(plan, x, 4, 0, 1, w, 1e-6, 1e4)[0]),
}
CHANGES = {
    "grid": lambda plan: B.ulysses_plan_set_rope_grid(plan, [4, 4], [16, 16]),
    "first": lambda plan: B.ulysses_plan_set_rope_grid(plan, [2, 8], [16, 16], 1),
    "off": lambda plan: B.ulysses_plan_set_rope_grid(plan, [], []),
    "pairs": lambda plan: B.ulysses_plan_set_rope_pairs(plan, B.ULY_ROPE_HALF),
}


def start(plan):
    B.ulysses_plan_set_rope_pairs(plan, B.ULY_ROPE_ADJACENT)
    B.ulysses_plan_set_rope_grid(plan, [2, 8], [16, 16])


def once(form, change=None, back=False):
    mid, fn = FORMS[form]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    plan = B.ulysses_plan(W, b, SEQ, HEADS, d, "bfloat16")
    start(plan)
    xs = [torch.randn((b, s, *mid, N, d), generator=gen, device="cuda").bfloat16().requires_grad_()
          for s in SEQ]
    w = torch.ones(2, d, device="cuda", requires_grad=True)
    loss = sum(y.float().square().mul(torch.arange(d, device="cuda")).sum() for y in fn(plan, xs, w))
    if change:
        change(plan)
    if back:
        start(plan)
    loss.backward()
    return [x.grad for x in xs]


@pytest.mark.parametrize("change", CHANGES)
@pytest.mark.parametrize("form", FORMS)
def test_settings_changed_in_between(form, change):
    with pytest.raises(RuntimeError, match="RoPE settings"):
        once(form, CHANGES[change])
    same = once(form, CHANGES[change], back=True)
    assert all(torch.equal(x, y) for x, y in zip(same, once(form)))
