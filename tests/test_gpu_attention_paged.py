"""Attention of the last tokens over a paged cache (ulysses_attention_paged) against the definition in 64
bits, and the writing of tokens into the pages (ulysses_cache_append), which is exact.

Tolerances: those of attention over contiguous keys, for the same roundings. The output is rounded once (u,
half a step: bf16 2^-8, fp16 2^-11), each probability by u p_j, which moves the output by at most
u sum_j p_j |v_j| =: u a; scores, exponentials, sums and the joining of parts in fp32: 1e-4 a covers
them tenfold. fp16 probabilities below 2^-14 are off by 2^-25 each, relative to a maximum that may lag but
never lead, times 2^7: keys 2^-25 max|v|, with max|v| < 8, covers them. lse is fp32: 2^-22 of its size plus
the score's error, 3e-5."""
import math
import random

import pytest
import torch

import window_reference as R
from gpu_util import GuardedOutputs
from ulysses_sequence_all_gb300 import binding as B

pytestmark = pytest.mark.gpu
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    B.library()


@pytest.fixture(autouse=True)
def status():
    yield
    assert B.ulysses_device_status() == 0


def split(total, W):
    return [total // W + (r < total % W) for r in range(W)]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    """Sequences of `lens` tokens, their last `sq` as queries, in shuffled pages; what no row sees and
    every page that no row needs holds `fill`, and the table -1 where no page is needed."""

    def __init__(self, W, sq, lens, kv_heads, g, d, page, window=0, sinks=0, dtype=torch.bfloat16, seed=0,
                 q_start=None, fill=math.nan, spare=3):
        b = len(lens)
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dtype)
        self.lens, self.window, self.sinks, self.page = [max(0, n) for n in lens], window, sinks, page
        self.q_start, self.dtype, self.scale = q_start, dtype, d ** -0.5
        most = max(1, max(self.lens))
        per = -(-most // page)
        starts = [n - sq for n in self.lens] if q_start is None else q_start
        self.see = R.visible(b, sq, most, window, sinks, self.lens, starts)
        self.q = [rnd(b, sq, g * m, d) for m in kv_heads]
        self.k = [rnd(b, most, m, d) for m in kv_heads]
        self.v = [rnd(b, most, m, d) for m in kv_heads]
        rng = random.Random(seed)
        need = [[bool(self.see[bb, :, p * page:(p + 1) * page].any()) for p in range(per)] for bb in range(b)]
        self.pages = sum(map(sum, need)) + spare
        order = rng.sample(range(self.pages), self.pages)
        table = [[order.pop() if x else -1 for x in row] for row in need]
        self.table_cpu = torch.tensor(table)
        self.table = i32(table)
        some = self.see.any(1)[:, :, None, None]
        hide = lambda x: torch.where(some, x, torch.full_like(x, fill))
        pool = lambda x: R.paged(hide(x), self.lens, page, self.table_cpu, self.pages, fill)
        self.k_pages, self.v_pages = [pool(x) for x in self.k], [pool(x) for x in self.v]
        name = str(dtype).split(".")[1]
        self.qp = B.ulysses_plan(W, b, split(sq, W), [g * m for m in kv_heads], d, name)
        self.cp = B.ulysses_plan(W, self.pages, split(page, W), kv_heads, d, name)

    def run(self, stream=None):
        o = GuardedOutputs([x.shape for x in self.q], self.dtype)
        lse = GuardedOutputs([(x.shape[0], x.shape[2], x.shape[1]) for x in self.q], torch.float32)
        ws = torch.full((B.ulysses_attention_paged_workspace(self.qp, self.cp),), 255, dtype=torch.uint8,
                        device="cuda")
        B.ulysses_attention_paged(self.qp, self.cp, self.q, self.k_pages, self.v_pages, o.tensors,
                                  lse.tensors, self.table, i32(self.lens), scale=self.scale,
                                  q_start=None if self.q_start is None else i32(self.q_start),
                                  window=self.window, sinks=self.sinks, workspace=ws, stream=stream)
        torch.cuda.synchronize()
        assert o.guards_intact() and lse.guards_intact()
        return o.tensors, lse.tensors

    def check(self, o, lse):
        u = HALF_STEP[self.dtype]
        for r in range(len(self.q)):
            if self.q[r].numel() == 0:
                continue
            want, z, a = R.forward(self.q[r], self.k[r], self.v[r], self.scale, self.see)
            tiny = self.k[r].shape[1] * 2.0 ** -25 * 8 if self.dtype == torch.float16 else 0.0
            err = (o[r].double() - want).abs()
            tol = u * want.abs() + (u + 1e-4) * a + tiny + 2.0 ** -24
            assert not (err > tol).any() and not o[r].isnan().any(), \
                f"rank {r}: {int((err > tol).sum())} off, worst {float((err - tol).max())}"
            empty = z == -math.inf
            assert torch.equal(lse[r] == -math.inf, empty)
            assert bool((o[r].transpose(1, 2)[empty] == 0).all())
            le = (lse[r].double() - z)[~empty].abs()
            assert not (le > 3e-5 + 2.0 ** -22 * z[~empty].abs()).any(), float(le.max())


SHAPES = [
    # W, new tokens, lengths, kv heads, group, d, page
    (1, 1, [1], [1], 1, 64, 8),
    (1, 1, [16], [1], 1, 128, 16),
    (2, 1, [65, 1, 64], [1, 1], 1, 64, 16),
    (1, 1, [1000], [2], 8, 128, 16),
    (3, 1, [0, 333, 17, 130], [1, 0, 2], 4, 128, 32),
    (1, 1, [777, 5], [2], 3, 72, 24),
    (2, 4, [100, 3, 4, 900], [2, 1], 2, 64, 8),
    (1, 4, [513, 129], [1], 8, 128, 64),        # 32 rows
    (1, 3, [200, 91], [1], 5, 80, 48),          # 15 rows
    (1, 7, [300, 40], [2], 9, 96, 16),          # 63 rows: two passes, the last one not full
    (1, 150, [150, 400], [1], 1, 120, 128),     # five passes
    (1, 1, [20000], [1], 8, 128, 64),           # one head on every CTA
    (8, 1, [50] * 40 + [2000], [1] * 8, 2, 8, 40),
    (1, 1, [3000, 1, 700], [1], 64, 64, 256),   # 64 heads share
]
IDS = ["x".join(map(str, (s[0], s[1], max(s[2]), s[4], s[5], s[6]))) for s in SHAPES]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_matches_definition(shape, dtype):
    c = Case(*shape, dtype=dtype)
    c.check(*c.run())


@pytest.mark.parametrize("window, sinks", [(1, 0), (1, 1), (17, 4), (64, 16), (100, 0), (300, 70), (5000, 3)])
@pytest.mark.parametrize("shape", [s for s in SHAPES if max(s[2]) > 90],
                         ids=[i for i, s in zip(IDS, SHAPES) if max(s[2]) > 90])
def test_window(shape, window, sinks):
    """Pages that no row sees are given back (-1) or hold NaN; a window before, at and past the start."""
    c = Case(*shape, window=window, sinks=sinks, seed=3)
    c.check(*c.run())


@pytest.mark.parametrize("fill", [math.nan, math.inf, 0.0])
def test_starts_of_their_own(fill):
    """Queries that begin before the first key, inside, at the end and past what the cache holds."""
    c = Case(2, 6, [200, 200, 200, 200, 0, 30], [1, 2], 2, 64, 16, q_start=[-3, 60, 194, 400, 5, -9],
             fill=fill)
    c.check(*c.run())
    c = Case(2, 6, [200, 200, 200, 200, 0, 30], [1, 2], 2, 64, 16, q_start=[-3, 60, 194, 400, 5, -9],
             window=20, sinks=2, fill=fill)
    c.check(*c.run())


def test_the_same_bits_under_a_cap_and_again():
    c = Case(2, 1, [5000, 130, 77, 1, 2600], [1, 2], 4, 128, 16, window=0)
    want = c.run()
    for cap in (0, 1, 7, 200):
        B.ulysses_plan_set_max_ctas(c.qp, cap)
        for x, y in zip(c.run(), want):
            for s, t in zip(x, y):
                assert torch.equal(s.view(torch.uint8), t.view(torch.uint8))


def test_shared_pages_and_lengths_past_the_table():
    """Two sequences with one beginning; a length beyond what the table has room for is what it has."""
    c = Case(1, 1, [96, 96], [2], 2, 64, 16)
    table = c.table_cpu.clone()
    table[1, :4] = table[0, :4]
    for x in c.k + c.v:
        x[1, :64] = x[0, :64]
    c.table = i32(table.tolist())
    c.check(*c.run())
    c.lens = [5000, 96]
    c.q_start = [95, 95]
    c.check(*c.run())


def test_needed_pages_outside_the_pool_are_reported():
    c = Case(1, 1, [64, 64], [1], 1, 64, 16, fill=0.0)
    table = c.table_cpu.clone()
    for bad in (-1, c.pages, 2 ** 31 - 1, -2 ** 31):
        table[1, 2] = bad
        c.table = i32(table.tolist())
        o, lse = c.run()
        assert B.ulysses_device_status() == 4
        c.v[0][1, 32:48], c.k[0][1, 32:48] = 0, 0  # read as zeros
        c.check(o, lse)


def test_graph_streams_and_new_lengths():
    """A captured call replayed after the lengths, the table and the pages changed; another stream."""
    c = Case(1, 1, [500, 40, 7], [2], 4, 128, 16, fill=0.0, spare=40)
    lens = i32(c.lens)
    out = [torch.empty_like(x) for x in c.q]
    lse = [torch.empty(3, 8, 1, device="cuda")]
    ws = torch.empty(B.ulysses_attention_paged_workspace(c.qp, c.cp), dtype=torch.uint8, device="cuda")
    call = lambda: B.ulysses_attention_paged(c.qp, c.cp, c.q, c.k_pages, c.v_pages, out, lse, c.table, lens,
                                             scale=c.scale, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    c.check(out, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    lens.copy_(i32([33, 0, 7]))
    for x in c.q:
        x.mul_(-1)
    graph.replay()
    torch.cuda.synchronize()
    c.lens = [33, 0, 7]
    c.see = R.visible(3, 1, 500, 0, 0, c.lens, [32, -1, 6])
    c.check(out, lse)


# ---- append ---------------------------------------------------------------------------------------

APPENDS = [
    # W, tokens, starts, counts, kv heads, d, page, dtype
    (1, 1, [0], None, [1], 64, 8, torch.bfloat16),
    (2, 1, [0, 15, 16, 700], None, [2, 1], 128, 16, torch.float16),
    (3, 9, [0, 3, 40], [9, 0, 4], [1, 0, 2], 72, 24, torch.bfloat16),
    (1, 300, [0, 77], [300, 123], [3], 8, 64, torch.float32),
    (8, 5, list(range(30)), [i % 7 - 1 for i in range(30)], [1] * 8, 16, 8, torch.uint8),
    (2, 64, [128], [99], [1, 1], 120, 32, torch.bfloat16),
]


@pytest.mark.parametrize("W, tokens, starts, counts, heads, d, page, dtype", APPENDS)
def test_append(W, tokens, starts, counts, heads, d, page, dtype):
    b = len(starts)
    ends = [s + (tokens if counts is None else min(tokens, max(0, counts[i]))) for i, s in enumerate(starts)]
    per = max(1, -(-max(ends) // page))
    pages = b * per + 2
    rng = random.Random(1)
    order = rng.sample(range(pages), pages)
    table = [[order.pop() if p * page < ends[bb] else 10 ** 9 for p in range(per)] for bb in range(b)]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    rnd = lambda *s: (torch.randn(s, generator=gen, device="cuda") * 50).to(dtype)
    k, v = ([rnd(b, tokens, m, d) for m in heads] for _ in range(2))
    pools = [GuardedOutputs([(pages, page, m, d) for m in heads], dtype) for _ in range(2)]
    want = []
    for new, pool in zip((k, v), pools):
        for x, y in zip(new, pool.tensors):
            z = y.clone()
            for bb in range(b):
                for i in range(ends[bb] - starts[bb]):
                    j = starts[bb] + i
                    z[table[bb][j // page], j % page] = x[bb, i]
            want.append(z)
    name = str(dtype).split(".")[1]
    kp = B.ulysses_plan(W, b, split(tokens, W), heads, d, name)
    cp = B.ulysses_plan(W, pages, split(page, W), heads, d, name)
    B.ulysses_cache_append(kp, cp, k, v, pools[0].tensors, pools[1].tensors, i32(table), i32(starts),
                           counts=None if counts is None else i32(counts))
    torch.cuda.synchronize()
    for got, z in zip(pools[0].tensors + pools[1].tensors, want):
        assert torch.equal(got.view(torch.uint8), z.view(torch.uint8))
    assert pools[0].guards_intact() and pools[1].guards_intact()


def test_append_writes_nothing_without_a_place():
    kp = B.ulysses_plan(1, 4, [3], [1], 64, "bfloat16")
    cp = B.ulysses_plan(1, 6, [8], [1], 64, "bfloat16")
    k, v = ([torch.ones(4, 3, 1, 64, device="cuda").bfloat16()] for _ in range(2))
    pools = [[torch.zeros(6, 8, 1, 64, device="cuda").bfloat16()] for _ in range(2)]
    table = i32([[0, 1], [-1, 2], [6, 3], [4, 2 ** 31 - 1]])
    B.ulysses_cache_append(kp, cp, k, v, *pools, table, i32([-2, 6, 6, 15]))
    assert B.ulysses_device_status() == 4
    rows = torch.zeros(6, 8, dtype=torch.bool)
    rows[0, 0] = True                 # of -2, -1, 0
    rows[2, 0] = rows[3, 0] = True    # of 6, 7, 8 with a bad first page
    for p in pools:
        assert torch.equal((p[0] != 0).all(-1).all(-1).cpu(), rows)
        assert torch.equal((p[0] != 0).any(-1).any(-1).cpu(), rows)


@pytest.mark.parametrize("cap", [1, 3, 1000])
def test_append_under_a_cap(cap):
    kp = B.ulysses_plan(2, 2, [50, 50], [2, 1], 64, "bfloat16")
    cp = B.ulysses_plan(2, 30, [8, 8], [2, 1], 64, "bfloat16")
    B.ulysses_plan_set_max_ctas(kp, cap)
    new = [torch.randn(2, 100, m, 64, device="cuda").bfloat16() for m in (2, 1)]
    pools = [[torch.zeros(30, 16, m, 64, device="cuda").bfloat16() for m in (2, 1)] for _ in range(2)]
    table = torch.arange(30, dtype=torch.int32, device="cuda").view(2, 15)
    B.ulysses_cache_append(kp, cp, new, new, *pools, table, i32([4, 100]))
    for pool in pools:
        for x, y in zip(new, pool):
            flat = y.view(2, 240, *y.shape[2:])
            assert torch.equal(flat[0, 4:104], x[0]) and torch.equal(flat[1, 100:200], x[1])


def test_a_prompt_then_token_by_token():
    """A prompt attends and is appended; each new token is appended and attends over the pages: the same as
    causal attention over the whole sequence, within the rounding of both (two half steps of each)."""
    W, b, S, new, heads, g, d, page = 2, 2, 90, 5, [1, 2], 2, 64, 16
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    rnd = lambda n, m: torch.randn((b, n, m, d), generator=gen, device="cuda").bfloat16()
    T = S + new
    q, k, v = [rnd(T, g * m) for m in heads], [rnd(T, m) for m in heads], [rnd(T, m) for m in heads]
    plan = lambda n, hs, batch=b: B.ulysses_plan(W, batch, split(n, W), hs, d, "bfloat16")
    per = -(-T // page)
    pages = b * per
    table = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32).view(b, per)
    kc, vc = ([torch.full((pages, page, m, d), math.nan, device="cuda").bfloat16() for m in heads]
              for _ in range(2))
    cp = plan(page, heads, pages)
    see = R.visible(b, T, T)
    want = [R.forward(x, y, z, d ** -0.5, see) for x, y, z in zip(q, k, v)]
    at = i32([0] * b)
    lens = i32([0] * b)
    for first, n in [(0, S)] + [(S + i, 1) for i in range(new)]:
        rows = slice(first, first + n)
        part = lambda xs: [x[:, rows].contiguous() for x in xs]
        qp, kp = plan(n, [g * m for m in heads]), plan(n, heads)
        B.ulysses_cache_append(kp, cp, part(k), part(v), kc, vc, table, at)
        lens += n
        out = [torch.empty_like(x) for x in part(q)]
        lse = [torch.empty(b, g * m, n, device="cuda") for m in heads]
        ws = torch.empty(B.ulysses_attention_paged_workspace(qp, cp), dtype=torch.uint8, device="cuda")
        B.ulysses_attention_paged(qp, cp, part(q), kc, vc, out, lse, table, lens, scale=d ** -0.5,
                                  workspace=ws)
        at += n
        for o, (x, _, a) in zip(out, want):
            err = (o.double() - x[:, rows]).abs()
            assert not (err > 2.0 ** -8 * x[:, rows].abs() + (2.0 ** -8 + 1e-4) * a[:, rows]).any()
