"""The failure path of attention over pages and of few rows with a window, without a fault: under a wait limit of
nothing the kernels give up, say so in the status word and return, and the same call with the usual limit is what
it was, to the bit."""
import time

import pytest
import torch

from test_gpu_attention_paged import Case as Paged
from test_gpu_attention_window import Case as Window
from ulysses_sequence_all_gb300 import binding as B

pytestmark = pytest.mark.gpu

DEFAULT = 2_000_000


@pytest.fixture(autouse=True)
def usual_limit():
    B.library()
    assert B.ulysses_device_status() == 0
    yield
    B.ulysses_selftest_attention_wait_limit(DEFAULT)
    assert B.ulysses_device_status() == 0


def gives_up(run):
    want = [x.clone() for t in run() for x in t]
    assert B.ulysses_device_status() == 0
    for _ in range(3):
        B.ulysses_selftest_attention_wait_limit(0)
        t0 = time.perf_counter()
        run()
        status = B.ulysses_device_status()
        seconds = time.perf_counter() - t0
        B.ulysses_selftest_attention_wait_limit(DEFAULT)
        assert status == 1 and seconds < 1.0, (status, seconds)  # no wait for a copy ran out behind it
        got = [x for t in run() for x in t]
        assert B.ulysses_device_status() == 0
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(want, got))


# one CTA with a share after the other, hundreds of blocks; and all of them
@pytest.mark.parametrize("cap", [1, 0])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sq, g", [(1, 1), (1, 8), (2, 8), (4, 8)], ids=["1row", "8rows", "16rows", "32rows"])
def test_few_rows_over_pages(sq, g, d, cap):
    c = Paged(2, sq, [30000, 500, 0, 9000], [1, 1], g, d, 16, fill=0.0)
    B.ulysses_plan_set_max_ctas(c.qp, cap)
    gives_up(c.run)


@pytest.mark.parametrize("d", [64, 128])
def test_many_rows_over_pages(d):
    c = Paged(1, 1500, [20000, 3000], [1], 1, d, 16, fill=0.0)
    B.ulysses_plan_set_max_ctas(c.qp, 1)  # more units a CTA than it knows ahead
    gives_up(c.run)


@pytest.mark.parametrize("sq, g", [(1, 1), (2, 8)], ids=["1row", "16rows"])
def test_few_rows_with_a_window(sq, g):
    c = Window(2, 3, sq, 20000, [1, 1], g, 128, 9000, 4, q_start=[20000 - sq, 500, 12000], fill=0.0)
    B.ulysses_plan_set_max_ctas(c.qp, 1)
    gives_up(c.forward)
