"""Appends to the 8-bit cache at the edges of what the interface promises: blocks whose
earlier codes are not numbers, and rows with many skipped ones among and behind them
(needs a GB300)."""
import math

import pytest
import torch

import kv8_util as k8
from exact_attention_57_gb300 import fa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,bs", [(1, 16), (1, 128), (40, 64), (100, 128)])
def test_codes_under_a_scale_that_is_no_positive_number_count_as_zeros(dtype, rows, bs):
    """Whatever a block held, NaN codes among it, is zero once a token behind it is
    written, if the block's scale was not a positive number."""
    old = [math.nan, -3.0, 0.0, -0.0, -math.inf]
    n, d, first = len(old), 32, 9
    codes = torch.arange(n * bs * d).reshape(n, 1, bs, d).to(torch.uint8)  # every code
    codes[:, :, 3], codes[:, :, 4] = 0x7F, 0xFF
    scales = torch.tensor(old)[:, None]
    cache = k8.on([codes.clone(), scales.clone(), codes.clone(), scales.clone()], DEV)
    x = torch.ones(n * rows, 1, d).to(DT[dtype]).to(DEV)
    off = first + torch.arange(rows)
    slots = (torch.arange(n)[:, None] * bs + off).flatten().to(DEV)
    fa.kv8_append(x, x, slots, *cache)
    for c, s in (cache[:2], cache[2:]):
        c = c.view(torch.uint8).cpu()
        assert s.flatten().tolist() == [2.0 ** -8] * n  # 448 / 2^8 = 1.75
        assert (c[:, :, :first] & 127 == 0).all()
        assert (k8.numbers(c[:, :, off]) == 256).all()
        assert torch.equal(c[:, :, first + rows:], codes[:, :, first + rows:])
