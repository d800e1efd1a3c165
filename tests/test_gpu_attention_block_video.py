"""The library's attention block (positions of three axes, attention, both relayouts, all of them
the library's) against the block written in plain torch without ranks, forward and gradients.

The two differ in rounding only: bf16 after the norm and rotation, of the probabilities, of the
attention output and of each gradient on the way back, each 2^-9 of the value on average over sums
of random sign. Four of them in a row and the outputs' own stay below 2e-2 of the largest value; a
wrong head, position, axis or rank anywhere gives errors of order 1."""
import pytest
import torch

from ulysses_sequence_all_gb300 import binding as B
from ulysses_sequence_all_gb300.attention_block import attention_block, axis_pairs, main

pytestmark = pytest.mark.gpu

EPS, THETA, TOL = 1e-6, 1e4, 2e-2
W, b, d = 3, 2, 64
GRID, TEXT = (4, 7, 9), 5                      # a clip with text tokens in front
SEQ, HEADS = [90, 0, 167], [2, 3, 1]           # uneven ranks, one without tokens
N, S = sum(HEADS), sum(SEQ)


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    B.library()
    yield
    assert B.ulysses_device_status() == 0, "a kernel recorded a wait timeout"


def plain_block(qkv, w, causal, lens):
    p = torch.arange(S, device="cuda") - TEXT
    on = p >= 0
    coords = [(p // 63) * on, (p // 9 % 7) * on, (p % 9) * on]
    ang = torch.cat([c[:, None].double() * THETA ** (-torch.arange(m, device="cuda").double() / m)
                     for c, m in zip(coords, axis_pairs(d, 3))], 1)
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]

    def turn(x, weight):
        x = x.float()
        y = x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + EPS) * weight
        e, o = y[..., 0::2], y[..., 1::2]
        return torch.stack((e * cos - o * sin, e * sin + o * cos), -1).flatten(-2)

    q, k, v = turn(qkv[:, :, 0], w[0]), turn(qkv[:, :, 1], w[1]), qkv[:, :, 2].float()
    s = torch.einsum("bind,bjnd->bnij", q, k) * d ** -0.5
    j = torch.arange(S, device="cuda")
    hide = j[None, None, :] >= lens[:, None, None]
    if causal:
        hide = hide | (j[None, None, :] > j[None, :, None])
    s = s.masked_fill(hide[:, None], float("-inf"))
    return torch.einsum("bnij,bjnd->bind", s.softmax(-1), v)


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
def test_block_matches_plain_block(causal):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    whole = torch.randn((b, S, 3, N, d), generator=gen, device="cuda").bfloat16()
    w0 = 1.0 + 0.1 * torch.randn((2, d), generator=gen, device="cuda")
    gy = torch.randn((b, S, N, d), generator=gen, device="cuda").bfloat16()
    lens = torch.tensor([S, 130], device="cuda", dtype=torch.int32)
    plan = B.ulysses_plan(W, b, SEQ, HEADS, d, "bfloat16")
    B.ulysses_plan_set_rope_grid(plan, GRID, axis_pairs(d, 3), first=TEXT)
    x1, w1 = whole.clone().requires_grad_(), w0.clone().requires_grad_()
    x2, w2 = whole.clone().requires_grad_(), w0.clone().requires_grad_()
    y1 = torch.cat(attention_block(plan, list(x1.split(SEQ, 1)), w1, EPS, THETA, causal=causal,
                                   kv_lens=lens), 1)
    y2 = plain_block(x2, w2, causal, lens)
    y1.backward(gy)
    y2.backward(gy.float())
    for name, got, want in (("out", y1, y2), ("qkv", x1.grad, x2.grad), ("rms_w", w1.grad, w2.grad)):
        err = (got.double() - want.double()).abs().max() / want.double().abs().max()
        assert err < TOL, (name, float(err))


def test_command_runs(capsys):
    main(["--grid", "3", "5", "8", "--heads", "2", "--ranks", "2", "--d", "64", "--backward"])
    assert "forward and backward" in capsys.readouterr().out
