"""A step of decoding captured once and replayed token by token: the new token appended at the sequences' ends, the
lengths counted up on the device, its attention over the pages. A second graph, of a few drafted tokens a sequence,
shares the workspace and is replayed in between. Against the definition in 64 bits (tolerances: each output rounded
once, each probability once, fp32 parts 1e-4)."""
import math

import pytest
import torch

import window_reference as R
from ulysses_sequence_all_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    B.library()
    yield
    assert B.ulysses_device_status() == 0


@pytest.mark.parametrize("window, sinks", [(0, 0), (50, 3)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_captured_steps(dtype, window, sinks):
    W, heads, g, d, page, b = 2, [1, 2], 4, 64, 16, 3
    first, steps, drafted = [0, 15, 130], [1, 4, 1, 1, 4, 1, 4] * 3, 4
    u = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[dtype]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(11)
    most = max(first) + sum(steps)
    rnd = lambda n, m: torch.randn((b, n, m, d), generator=gen, device="cuda").to(dtype)
    q, k, v = ([rnd(most, x * m) for m in heads] for x in (g, 1, 1))
    name = str(dtype).split(".")[1]
    plan = lambda n, hs, batch=b: B.ulysses_plan(W, batch, [n] + [0] * (W - 1), hs, d, name)
    per = -(-most // page)
    table = torch.randperm(b * per, generator=gen, device="cuda").to(torch.int32).view(b, per)
    cp = plan(page, heads, b * per)
    pools = [[torch.full((b * per, page, m, d), math.nan, device="cuda").to(dtype) for m in heads] for _ in range(2)]
    lens = torch.tensor(first, dtype=torch.int32, device="cuda")
    B.ulysses_cache_append(plan(most, heads), cp, k, v, *pools, table, torch.zeros_like(lens), counts=lens)
    qps = {n: plan(n, [g * m for m in heads]) for n in (1, drafted)}
    ws = torch.empty(max(B.ulysses_attention_paged_workspace(p, cp) for p in qps.values()), dtype=torch.uint8,
                     device="cuda")
    graphs = {}
    for n, qp in qps.items():
        new = [[torch.zeros((b, n, x * m, d), device="cuda", dtype=dtype) for m in heads] for x in (g, 1, 1)]
        out, lse = [torch.empty_like(x) for x in new[0]], [torch.empty((b, g * m, n), device="cuda") for m in heads]
        kp, tokens = plan(n, heads), torch.zeros_like(lens)  # (none yet: the call before the capture changes nothing)

        def step():
            B.ulysses_cache_append(kp, cp, new[1], new[2], *pools, table, lens, counts=tokens)
            lens.add_(tokens)
            B.ulysses_attention_paged(qp, cp, new[0], *pools, out, lse, table, lens, scale=d ** -0.5, window=window,
                                      sinks=sinks, workspace=ws)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        tokens.fill_(n)
        graphs[n] = graph, new, out, lse, tokens
    at = list(first)
    for n in steps:
        graph, new, out, lse, _ = graphs[n]
        for xs, whole in zip(new, (q, k, v)):
            for x, y in zip(xs, whole):
                for bb in range(b):
                    x[bb] = y[bb, at[bb]:at[bb] + n]
        graph.replay()
        see = torch.cat([R.visible(1, n, most, window, sinks, [at[bb] + n], [at[bb]]) for bb in range(b)])
        for r in range(W):
            want, z, a = R.forward(new[0][r], k[r], v[r], d ** -0.5, see)
            tiny = most * 2.0 ** -25 * 8 if dtype == torch.float16 else 0.0
            err = (out[r].double() - want).abs()
            assert not (err > u * want.abs() + (u + 1e-4) * a + tiny + 2.0 ** -24).any() and out[r].isfinite().all()
            assert not ((lse[r].double() - z).abs() > 3e-5 + 2.0 ** -22 * z.abs()).any()
        at = [x + n for x in at]
    assert lens.tolist() == at
