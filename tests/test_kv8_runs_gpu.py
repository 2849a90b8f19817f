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


def appended(rows, slots, T, Hk, d, bs, blocks, seed, dtype=torch.bfloat16):
    """Rows at `rows` of T, the others skipped: what the library and the plain reference
    make of them."""
    g = torch.Generator().manual_seed(seed)
    before = k8.random_store(blocks, Hk, bs, d, g) + k8.random_store(blocks, Hk, bs, d, g)
    x = torch.randn(len(rows), 2 * Hk, d, generator=g) * 2.0 ** torch.randint(-4, 4, (len(rows), 1, 1),
                                                                           generator=g)
    x = x.to(dtype)
    at = torch.tensor(rows)
    sent = torch.full((T,), -1, dtype=torch.long)
    sent[at] = torch.tensor(slots)
    wide = torch.full((T, 2 * Hk, d), math.nan, dtype=dtype, device=DEV)
    wide[at.to(DEV)] = x.to(DEV)
    cache = k8.on(before, DEV)
    fa.kv8_append(wide[:, :Hk], wide[:, Hk:], sent.to(DEV), *cache)
    want = k8.append(x[:, :Hk], torch.tensor(slots), *before[:2]) + \
        k8.append(x[:, Hk:], torch.tensor(slots), *before[2:])
    return [c.cpu().view(torch.uint8) if c.dtype == torch.float8_e4m3fn else c.cpu() for c in cache], want


GAPS = [0, 1, 7, 31, 32, 100, 119, 120, 223, 224, 246, 247, 248, 249, 255, 256, 257, 2047, 2048, 2049,
        4087, 4096, 4103, 9001]


@pytest.mark.parametrize("gap", GAPS)
@pytest.mark.parametrize("bs,Hk,d", [(16, 1, 64), (64, 2, 128), (128, 1, 16)])
@pytest.mark.parametrize("more", [False, True])
def test_skipped_rows_of_any_number(gap, bs, Hk, d, more):
    """Skipped rows ahead of, inside and behind the rows of a block, in batches of either
    side of 4096 rows; `more`: another block's rows follow, or none."""
    lens = [3, bs - 2, 1, bs]  # rows of four blocks, the first begun before
    rows, slots, t = [], [], gap
    ids = [5, 2, 9, 0]
    for b, n in zip(ids, lens):
        for i in range(n):
            rows.append(t)
            slots.append(b * bs + (1 if n == bs - 2 else 0) + i)
            t += 1 + (gap if i == n // 2 else 0)
        t += gap if b == 2 else 0
    if more:
        rows.append(t + gap)
        slots.append(7 * bs + 5)
    T = rows[-1] + 1 + gap
    got, want = appended(rows, slots, T, Hk, d, bs, 11, gap)
    for i in range(4):
        a, b = got[i], want[i]
        if i % 2 == 0:  # -0 and +0 are one value
            a, b = torch.where(a == 128, 0, a), torch.where(b == 128, 0, b)
        assert torch.equal(a, b)


@pytest.mark.parametrize("bs", [16, 128])
def test_a_row_here_and_there(bs):
    """Each row far from the next: rows of one block on either side of every gap, or of
    two."""
    step = 700
    rows = list(range(0, 40 * step, step))
    slots = [(t // 5) * bs + 2 * (t % 5) + 1 for t in range(len(rows))]  # five rows a block
    got, want = appended(rows, slots, rows[-1] + step, 2, 64, bs, 8, bs)
    for i in range(4):
        a, b = got[i], want[i]
        if i % 2 == 0:
            a, b = torch.where(a == 128, 0, a), torch.where(b == 128, 0, b)
        assert torch.equal(a, b)


def microseconds(call, n=10, turns=5):
    """Of one call in a row of n, the least of a few turns (events)."""
    best = math.inf
    for _ in range(turns):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        call()
        torch.cuda.synchronize()
        a.record()
        for _ in range(n):
            call()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 1000 / n)
    return best


@pytest.mark.parametrize("T,where", [(4096, "ahead"), (65536, "ahead"), (65536, "ends"), (65536, "inside")])
def test_a_padded_batch_costs_no_walk_along_its_skipped_rows(T, where):
    """64 rows of as many requests and skipped ones behind them (a captured step's
    capacity), ahead of some of them, or inside a block: within a few times of a batch of
    skipped rows alone of that length, which reads the same slots.  One warp that looks
    at 32 skipped rows after another takes 0.2 us for each 32 of them at the very least
    (a load that depends on the loop): 400 us for 65536, and several times that for
    each head; what is read side by side takes under 20."""
    bs, Hk, d, blocks = 16, 8, 128, 70
    cache = fa.kv8_cache(blocks, Hk, bs, d, device=DEV)
    x = torch.randn(T, 2 * Hk, d, device=DEV, dtype=torch.bfloat16)
    none = torch.full((T,), -1, dtype=torch.long, device=DEV)
    slots = none.clone()
    if where == "ahead":
        slots[:64] = bs * torch.arange(64, device=DEV) + 3
    elif where == "ends":
        slots[:32] = bs * torch.arange(32, device=DEV) + 3
        slots[-32:] = bs * torch.arange(32, 64, device=DEV) + 3
    else:
        slots[0], slots[-1] = 3, 4
    off = {}
    for name, s in (("none", none), ("some", slots)):
        off[name] = microseconds(lambda: fa.kv8_append(x[:, :Hk], x[:, Hk:], s, *cache))
    assert off["some"] <= 10 * off["none"], off
