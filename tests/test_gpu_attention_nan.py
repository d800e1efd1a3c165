"""NaN where a row sees it is never lost: a query of NaN gives NaN in its own output and log-sum-exp, and in
no other row's bits; visible keys of NaN give NaN in every row that sees them. Whatever kernel a call's rows
and keys take: few rows over pages or contiguous keys, whole or shared by several CTAs, or many rows."""
import math

import pytest
import torch

import window_reference as R
from test_gpu_attention_paged import Case as Paged
from test_gpu_attention_window import Case as Window
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


def bits(x):
    return x.contiguous().view(torch.uint8)


# new tokens, lengths, group, d, page: 1, 16 and 32 rows a key head; one CTA, several, most of them; many rows
PAGED = [(1, [40], 1, 64, 8), (1, [300, 70], 1, 128, 16), (1, [20000], 8, 128, 64), (2, [500, 9000], 8, 128, 32),
         (4, [200, 6000], 8, 128, 16), (4, [100, 4000], 8, 64, 24), (150, [400, 3000], 1, 128, 32)]
PAGED_IDS = ["x".join(map(str, (s[0], max(s[1]), s[2], s[3]))) for s in PAGED]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("window, sinks", [(0, 0), (100, 3)])
@pytest.mark.parametrize("shape", PAGED, ids=PAGED_IDS)
def test_a_query_of_nan_over_pages(shape, window, sinks, dtype):
    sq, lens, g, d, page = shape
    c = Paged(2, sq, lens, [1, 2], g, d, page, window=window, sinks=sinks, dtype=dtype)
    o, lse = c.run()
    c.check(o, lse)
    bb, tok, head = len(lens) - 1, sq - 1, g - 1
    c.q[1][bb, tok, head, d // 2] = math.nan
    o2, lse2 = c.run()
    assert o2[1][bb, tok, head].isnan().all() and lse2[1][bb, head, tok].isnan()
    o2[1][bb, tok, head] = o[1][bb, tok, head]
    lse2[1][bb, head, tok] = lse[1][bb, head, tok]
    for x, y in zip(o + lse, o2 + lse2):
        assert torch.equal(bits(x), bits(y))


@pytest.mark.parametrize("shape", PAGED, ids=PAGED_IDS)
@pytest.mark.parametrize("first, n", [(16, 16), (0, 1), (32, 64)])
def test_keys_of_nan_over_pages(shape, first, n):
    """Those of one warp's tile of keys, a single one, a stretch: in one sequence and one key head."""
    sq, lens, g, d, page = shape
    c = Paged(2, sq, lens, [1, 2], g, d, page)
    o, lse = c.run()
    bb, n = len(lens) - 1, min(n, lens[-1] - sq + 1 - first)  # (seen by every row)
    for j in range(first, first + n):
        c.k_pages[1][int(c.table_cpu[bb, j // page]), j % page, 1] = math.nan
    if n <= 0:
        return
    o2, lse2 = c.run()
    assert o2[1][bb, :, g:].isnan().all() and lse2[1][bb, g:].isnan().all()
    o2[1][bb, :, g:] = o[1][bb, :, g:]
    lse2[1][bb, g:] = lse[1][bb, g:]
    for x, y in zip(o + lse, o2 + lse2):
        assert torch.equal(bits(x), bits(y))


@pytest.mark.parametrize("sq, g, keys", [(1, 1, 60), (1, 8, 5000), (2, 8, 700), (3, 8, 700), (200, 2, 700)],
                         ids=["1row", "8rows", "16rows", "24rows", "prompt"])
def test_a_query_of_nan_with_a_window(sq, g, keys):
    c = Window(2, 2, sq, keys, [2, 1], g, 128, 50, 2, q_start=[keys - sq] * 2)
    o, lse = c.forward()
    c.check(o, lse)
    c.q[0][1, sq - 1, 0] = math.nan
    o2, lse2 = c.forward()
    assert o2[0][1, sq - 1, 0].isnan().all() and lse2[0][1, 0, sq - 1].isnan()
    o2[0][1, sq - 1, 0] = o[0][1, sq - 1, 0]
    lse2[0][1, 0, sq - 1] = lse[0][1, 0, sq - 1]
    for x, y in zip(o + lse, o2 + lse2):
        assert torch.equal(bits(x), bits(y))


@pytest.mark.parametrize("sq, g, keys", [(1, 1, 60), (1, 8, 5000), (2, 8, 700), (200, 2, 700)],
                         ids=["1row", "8rows", "16rows", "prompt"])
def test_keys_of_nan_with_a_window(sq, g, keys):
    """A first token of NaN, which every row sees; and all that a row sees."""
    c = Window(2, 2, sq, keys, [2, 1], g, 128, 50, 2, q_start=[keys - sq] * 2)
    o, lse = c.forward()
    c.k[0][1, 1, 1] = math.nan
    o2, lse2 = c.forward()
    assert o2[0][1, :, g:].isnan().all() and lse2[0][1, g:].isnan().all()
    o2[0][1, :, g:] = o[0][1, :, g:]
    lse2[0][1, g:] = lse[0][1, g:]
    for x, y in zip(o + lse, o2 + lse2):
        assert torch.equal(bits(x), bits(y))
    c.k[1][0] = math.nan
    o2, lse2 = c.forward()
    assert o2[1][0].isnan().all() and lse2[1][0].isnan().all()
