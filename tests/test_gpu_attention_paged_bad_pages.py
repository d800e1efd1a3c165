"""A needed page outside the pool, with as many query rows as each kernel over pages takes: reported by bit 4 of the
status word, its keys and values read as zeros, every other page as it is; the next call reports nothing."""
import pytest
import torch

from test_gpu_attention_paged import Case, i32
from ulysses_sequence_all_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    B.library()


# new tokens, group, d, page: 2, 16, 32 and 60, 600 rows a key head
@pytest.mark.parametrize("window, sinks", [(0, 0), (100, 40), (100, 90)])
@pytest.mark.parametrize("sq, g, d, page", [(1, 2, 64, 16), (2, 8, 128, 16), (4, 8, 64, 24), (60, 1, 128, 16),
                                            (60, 10, 64, 8)])
def test_bad_pages(sq, g, d, page, window, sinks):
    c = Case(2, sq, [300, 300], [1, 1], g, d, page, window=window, sinks=sinks, fill=0.0)
    want = c.run()
    assert B.ulysses_device_status() == 0
    c.check(*want)
    table = c.table_cpu.clone()
    at = (0, 299 // page)  # (with a window the first is needed for its first tokens)
    whole = [x.clone() for x in c.k + c.v]
    for p in at if sinks or not window else at[1:]:
        for bad in (-1, c.pages, 2 ** 31 - 1, -2 ** 31):
            broken = table.clone()
            broken[1, p] = bad
            c.table = i32(broken.tolist())
            for x, y in zip(c.k + c.v, whole):
                x.copy_(y)
                x[1, p * page:(p + 1) * page] = 0
            o, lse = c.run()
            assert B.ulysses_device_status() == 4
            c.check(o, lse)
    c.table = i32(table.tolist())
    for got, w in zip(c.run(), want):
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(got, w))
    assert B.ulysses_device_status() == 0
