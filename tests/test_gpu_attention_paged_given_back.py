"""Attention of many rows over pages of which those between the first tokens and the windows were given back:
their entries hold -1, and a call that needs none of them reports no bad page (bit 4 of the status word), wherever
the first tokens end against the blocks that they take."""
import random

import pytest
import torch

from test_gpu_attention_paged import Case
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


# new tokens, lengths, group, d, page, window, first tokens: the latter rounded up to whole blocks reach the window
CASES = [(40, [200], 1, 64, 8, 61, 70), (12, [330], 4, 128, 16, 100, 140), (100, [1000, 930], 1, 128, 8, 270, 600),
         (64, [400, 1, 380], 2, 80, 8, 215, 100), (300, [700], 1, 64, 32, 180, 130)]


@pytest.mark.parametrize("case", CASES, ids=["x".join(map(str, (c[0], max(c[1]), *c[2:]))) for c in CASES])
def test_pages_between_first_tokens_and_window(case):
    sq, lens, g, d, page, window, sinks = case
    c = Case(2, sq, lens, [1, 2], g, d, page, window=window, sinks=sinks)
    assert max(lens) < 700 or (c.table_cpu[0] < 0).any()
    c.check(*c.run())
    assert B.ulysses_device_status() == 0


@pytest.mark.parametrize("seed", range(24))
def test_any_window_and_first_tokens(seed):
    rng = random.Random(seed)
    g = rng.choice([1, 2, 3, 8])
    sq = rng.randint(33, 300) // g + 1
    lens = [rng.randint(max(1, sq - 5), 700) for _ in range(rng.randint(1, 3))]
    c = Case(1, sq, lens, [2], g, rng.choice([64, 128]), rng.choice([8, 16, 24, 40, 64, 128]),
             window=rng.randint(1, 300), sinks=rng.randint(0, 400), seed=seed)
    c.check(*c.run())
    assert B.ulysses_device_status() == 0
