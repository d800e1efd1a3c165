"""fp16 attention away from unit scale: many keys (probabilities far below fp16's smallest normal number),
small and large gradients, rows of very different ones.

Bounds, u = 2^-11. A gradient is a sum of products, one factor of each held in fp16: off by u of itself,
each its own way, so the sum is off by u sqrt(sum (ds k)^2) in the root mean square (the same for dk with
q, dv with P and go), where the factors' own range does not matter. The result is rounded: u of it, or
2^-25 where it is subnormal itself. In fp32 on the way: probabilities to 1e-4 (as in
test_gpu_attention_backward.py), dP and D to 2^-20 of the magnitudes that they sum up."""
import pytest
import torch

from attention_reference import forward
from test_gpu_attention_backward import check, given, gradients, plans
from ulysses_sequence_all_gb300 import binding as B

pytestmark = pytest.mark.gpu

U = 2.0 ** -11


@pytest.fixture(autouse=True)
def no_timeout():
    yield
    assert B.ulysses_device_status() == 0


def rms(x):
    return x.square().mean().sqrt().item()


def reference(q, k, v, o, lse, go, scale):
    """Per gradient: the value, sqrt of the sum of squared products, the same of the magnitudes that
    fp32 sums up (of one rank, no mask)."""
    g = q.shape[2] // k.shape[2]
    new = lambda: [torch.zeros(x.shape, dtype=torch.float64, device="cuda") for x in (q, k, v)]
    val, sq, mag = new(), new(), new()
    for bb in range(q.shape[0]):
        for h in range(q.shape[2]):
            qq, kk, vv = q[bb, :, h].double(), k[bb, :, h // g].double(), v[bb, :, h // g].double()
            gg, oo = go[bb, :, h].double(), o[bb, :, h].double()
            p = torch.exp(qq @ kk.T * scale - lse[bb, h].double()[:, None])
            ds = p * (gg @ vv.T - (gg * oo).sum(-1, keepdim=True))
            m = p * (gg.abs() @ vv.abs().T + (gg * oo).abs().sum(-1, keepdim=True))
            val[0][bb, :, h] = scale * ds @ kk
            sq[0][bb, :, h] = scale ** 2 * ds.square() @ kk.square()
            mag[0][bb, :, h] = scale ** 2 * m.square() @ kk.square()
            val[1][bb, :, h // g] += scale * ds.T @ qq
            sq[1][bb, :, h // g] += scale ** 2 * ds.square().T @ qq.square()
            mag[1][bb, :, h // g] += scale ** 2 * m.square().T @ qq.square()
            val[2][bb, :, h // g] += p.T @ gg
            sq[2][bb, :, h // g] += p.square().T @ gg.square()
    return zip(val, [x.sqrt() for x in sq], [x.sqrt() for x in mag])


def compare(got, q, k, v, o, lse, go, scale, rows=None):
    for r in range(len(q)):
        for name, x, (y, s, m) in zip(("dq", "dk", "dv"), (t[r] for t in got),
                                      reference(q[r], k[r], v[r], o[r], lse[r], go[r], scale)):
            x = x.double()
            if rows is not None and name == "dq":
                x, y, s, m = (t[:, rows] for t in (x, y, s, m))
            assert bool(x.isfinite().all()), (r, name)
            bound = (U + 1e-4) * (rms(y) + rms(s)) + 2.0 ** -25 + 2.0 ** -20 * rms(m)
            err = rms(x - y)
            assert err <= bound, (r, name, err / rms(y), bound / rms(y))


def rand(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return lambda size, *s: (size * torch.randn(s, generator=gen, device="cuda")).half()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [1e-4, 1e-3, 1.0, 30.0])
@pytest.mark.parametrize("q_size", [1.0, 64.0])
def test_many_keys(d, size, q_size):
    """q larger and k smaller by the same factor brings dk, in place of dq, into fp16's range."""
    shape = (1, 1, 40, 100_000, [1], 2, d)
    qp, kp = plans(*shape, torch.float16)
    rnd = rand(1)
    q, k, v = [rnd(q_size, 1, 40, 2, d)], [rnd(1 / q_size, 1, 100_000, 1, d)], [rnd(1.0, 1, 100_000, 1, d)]
    scale = d ** -0.5
    o, lse, _ = given(q, k, v, scale)
    go = [rnd(size, 1, 40, 2, d)]
    got = gradients(qp, kp, q, k, v, o, lse, go, scale)
    compare(got, q, k, v, o, lse, go, scale)


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size,v_size", [(1e-6, 1.0), (300.0, 30.0), (4000.0, 30.0)])
def test_few_keys_and_gradients_of_any_size(d, size, v_size, causal):
    """dS itself beyond fp16's largest number, the gradients within it; and all of them subnormal."""
    shape = (2, 2, 40, 21, [1, 2], 2, d)
    qp, kp = plans(*shape, torch.float16)
    rnd = rand(2)
    q = [rnd(0.05, 2, 40, 2 * m, d) for m in (1, 2)]
    k = [rnd(0.05, 2, 21, m, d) for m in (1, 2)]
    v = [rnd(v_size, 2, 21, m, d) for m in (1, 2)]
    kw = {"causal": True} if causal else {}
    o, lse, _ = given(q, k, v, 0.125, **kw)
    go = [rnd(size, *x.shape) for x in q]
    got = gradients(qp, kp, q, k, v, o, lse, go, 0.125, **kw)
    check(got, q, k, v, o, lse, go, 0.125, **kw)
    if not causal:
        compare(got, q, k, v, o, lse, go, 0.125)


@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_different_sizes(d):
    """Every other row's gradient 2,000 times smaller: its own dq keeps its digits."""
    shape = (1, 1, 150, 4000, [1], 2, d)
    qp, kp = plans(*shape, torch.float16)
    rnd = rand(3)
    q, k, v = [rnd(1.0, 1, 150, 2, d)], [rnd(1.0, 1, 4000, 1, d)], [rnd(1.0, 1, 4000, 1, d)]
    go = [rnd(20.0, 1, 150, 2, d)]
    go[0][:, ::2] *= 0.0005
    o, lse, _ = given(q, k, v, 0.125)
    got = gradients(qp, kp, q, k, v, o, lse, go, 0.125)
    compare(got, q, k, v, o, lse, go, 0.125, rows=slice(0, None, 2))
    compare(got, q, k, v, o, lse, go, 0.125, rows=slice(1, None, 2))


@pytest.mark.parametrize("lead", [17.5, 18.5])
@pytest.mark.parametrize("d", [64, 128])
def test_forward_small_weights_together(d, lead):
    """One key with most of the weight and 60,000 with about e^-lead of it each, all under one running
    maximum: together they are the output, although fp16 rounds each to nothing beside a 1. Bound: half
    a step for the result and for each probability, 1e-4 for scores and sums, 1e-4 for what the roundings
    of probabilities at 2^-18 leave on average; and the tensor cores cut their fp32 sums off instead of
    rounding them, by less than 2^-23 of the sum for every 16 keys."""
    n, sq, g = 60_000, 700, 64
    qp, kp = plans(1, 1, sq, n, [1], g, d, torch.float16)
    rnd = rand(7)
    q, k, v = rnd(0.2, 1, sq, g, d), rnd(0.2, 1, n, 1, d), 1 + rnd(0.1, 1, n, 1, d)
    q[..., 0], k[..., 0] = 8.0, 0.0
    k[:, 1000], v[:, 1000] = 0.0, 0.0
    k[:, 1000, :, 0] = lead / 8
    assert B.ulysses_attention_workspace(qp, kp) == 0  # not split: the parts would have maxima of their own
    o, lse = torch.empty_like(q), torch.empty(1, g, sq, device="cuda")
    B.ulysses_attention(qp, kp, [q], [k], [v], [o], [lse], scale=1.0)
    want, z, _ = forward(q[:, :3], k, v, 1.0)
    assert 3e-4 < want.mean() < 3e-3
    err = ((o[:, :3].double() - want).abs() / want.abs()).max().item()
    assert err <= 2 * U + 2e-4 + n / 16 * 2.0 ** -23, err
    assert (lse[:, :, :3].double() - z).abs().max() < 3e-5 + 2.0 ** -22 * 20
