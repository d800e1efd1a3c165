"""The paged cache and windows where arithmetic could run out: pools past 2^32 bytes, starts at the ends of int32,
windows and first tokens beyond every position, many rows under CTA caps, two calls at a time. Tolerances as in
test_gpu_attention_paged and test_gpu_attention_window, whose cases these are."""
import math

import pytest
import torch

import test_gpu_attention_paged as P
import test_gpu_attention_window as Win
import window_reference as R
from test_gpu_attention_paged import i32
from ulysses_sequence_all_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    B.library()


@pytest.fixture(autouse=True)
def status():
    yield
    assert B.ulysses_device_status() == 0


def bits(xs):
    return [x.view(torch.uint8) for t in xs for x in t]


@pytest.mark.parametrize("sq", [1, 20, 40], ids=["few", "pairs", "many"])
def test_a_pool_past_four_gigabytes(sq):
    """Pages at the end of a pool of 4.6 GB for the keys and as much for the values: written by the append,
    read by the attention."""
    b, m, g, d, page, pages, n = 2, 4, 2, 128, 64, 70_000, 300
    assert pages * page * m * d * 2 > 2 ** 32
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()
    q, k, v = rnd(b, sq, g * m, d), rnd(b, n, m, d), rnd(b, n, m, d)
    pools = [torch.empty(pages, page, m, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    per = -(-n // page)
    at = [pages - 1 - 7 * i for i in range(b * per)]
    table = i32(at).view(b, per)
    for x in pools:
        x[at] = math.nan
    plan = lambda batch, tokens, heads: B.ulysses_plan(1, batch, [tokens], [heads], d, "bfloat16")
    cp, qp = plan(pages, page, m), plan(b, sq, g * m)
    B.ulysses_cache_append(plan(b, n, m), cp, [k], [v], [pools[0]], [pools[1]], table, i32([0] * b))
    for x, y in zip((k, v), pools):
        got = y[at].view(b, per * page, m, d)
        assert torch.equal(got[:, :n], x) and bool(got[:, n:].isnan().all())
    o, lse = torch.empty_like(q), torch.empty(b, g * m, sq, device="cuda")
    need = B.ulysses_attention_paged_workspace(qp, cp)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    B.ulysses_attention_paged(qp, cp, [q], [pools[0]], [pools[1]], [o], [lse], table, i32([n] * b),
                              scale=d ** -0.5, workspace=ws)
    want, z, a = R.forward(q, k, v, d ** -0.5, R.visible(b, sq, n, q_start=[n - sq] * b))
    err = (o.double() - want).abs()
    assert not (err > 2.0 ** -8 * want.abs() + (2.0 ** -8 + 1e-4) * a).any()
    assert not ((lse.double() - z).abs() > 3e-5 + 2.0 ** -22 * z.abs()).any()


@pytest.mark.parametrize("sq", [2, 30, 50], ids=["few", "pairs", "many"])
@pytest.mark.parametrize("window, sinks", [(0, 0), (1, 0), (60, 3), (2 ** 62, 2 ** 62)])
def test_starts_at_the_ends_of_int32(sq, window, sinks):
    starts = [-2 ** 31, -2 ** 31 + 1, -1, 2 ** 30, 2 ** 31 - 1 - sq, 2 ** 31 - 1, 130]
    c = P.Case(2, sq, [150] * 7, [1, 1], 2, 64, 16, window=min(window, 2 ** 40), sinks=min(sinks, 200),
               q_start=starts)
    c.window, c.sinks = window, sinks
    c.check(*c.run())
    if window:
        c = Win.Case(1, 7, sq, 150, [1], 2, 64, min(window, 2 ** 40), min(sinks, 200), q_start=starts)
        c.window, c.sinks = window, sinks
        o, lse = c.forward()
        c.check(o, lse)
        c.check_backward(o, lse, c.backward(o, lse))


@pytest.mark.parametrize("sq, window, sinks", [(40, 0, 0), (40, 100, 70), (300, 90, 5), (20, 0, 0)])
def test_many_rows_have_the_same_bits_under_a_cap(sq, window, sinks):
    c = P.Case(2, sq, [700, 300, 1, 520], [1, 2], 2, 64, 16, window=window, sinks=sinks)
    want = c.run()
    c.check(*want)
    for cap in (1, 5, 300):
        B.ulysses_plan_set_max_ctas(c.qp, cap)
        for x, y in zip(bits(c.run()), bits(want)):
            assert torch.equal(x, y)


@pytest.mark.parametrize("page", [8, 24, 48, 128, 200, 1024])
@pytest.mark.parametrize("window, sinks", [(0, 0), (33, 9), (150, 65), (400, 4)])
def test_prompts_over_pages_of_every_kind(page, window, sinks):
    """Rows that fill tiles, behind a cache: first tokens that share a block and those that have their own."""
    for g, d in ((1, 128), (3, 72)):
        c = P.Case(1, 270, [270, 900, 100, 777], [2], g, d, page, window=window, sinks=sinks, seed=page)
        c.check(*c.run())


def test_two_calls_at_a_time():
    """On two streams, each with a workspace of its own."""
    cases = [P.Case(1, 1, [3000, 500], [2], 4, 128, 16, seed=1), P.Case(1, 45, [2000, 60, 900], [1], 1, 64, 32,
                                                                    window=700, sinks=2, seed=2)]
    streams = [torch.cuda.Stream() for _ in cases]
    runs = []
    for c in cases:
        out = [torch.empty_like(x) for x in c.q]
        lse = [torch.empty(x.shape[0], x.shape[2], x.shape[1], device="cuda") for x in c.q]
        need = B.ulysses_attention_paged_workspace(c.qp, c.cp)
        runs.append((out, lse, torch.empty(need, dtype=torch.uint8, device="cuda"), i32(c.lens)))
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, (out, lse, ws, lens) in zip(cases, streams, runs):
            B.ulysses_attention_paged(c.qp, c.cp, c.q, c.k_pages, c.v_pages, out, lse, c.table, lens,
                                      scale=c.scale, window=c.window, sinks=c.sinks, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for c, (out, lse, _, _) in zip(cases, runs):
        c.check(out, lse)


def test_a_workspace_in_turn():
    """Calls of other shapes on one stream leave the workspace as it comes."""
    cases = [P.Case(1, 1, [3000, 500], [2], 4, 128, 16, seed=1), P.Case(1, 45, [2000, 60, 900], [1], 1, 64, 32, seed=2),
             P.Case(2, 3, [5000] + [7] * 30, [1, 1], 8, 128, 64, seed=3)]
    ws = torch.empty(max(B.ulysses_attention_paged_workspace(c.qp, c.cp) for c in cases), dtype=torch.uint8,
                     device="cuda")
    for c in cases * 2:
        out = [torch.empty_like(x) for x in c.q]
        lse = [torch.empty(x.shape[0], x.shape[2], x.shape[1], device="cuda") for x in c.q]
        B.ulysses_attention_paged(c.qp, c.cp, c.q, c.k_pages, c.v_pages, out, lse, c.table, i32(c.lens),
                                  scale=c.scale, workspace=ws)
        c.check(out, lse)


def test_a_short_workspace_is_refused():
    c = P.Case(1, 1, [300], [1], 1, 64, 16)
    need = B.ulysses_attention_paged_workspace(c.qp, c.cp)
    out, lse = [torch.empty_like(x) for x in c.q], [torch.empty(1, 1, 1, device="cuda")]
    for ws in (None, torch.empty(need - 1, dtype=torch.uint8, device="cuda")):
        with pytest.raises(B.UlyssesError, match="invalid argument"):
            B.ulysses_attention_paged(c.qp, c.cp, c.q, c.k_pages, c.v_pages, out, lse, c.table, i32(c.lens),
                                      scale=1.0, workspace=ws)
