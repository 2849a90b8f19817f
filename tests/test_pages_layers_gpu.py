"""Forks and compactions of the arrays of many layers, in one call and in several
(needs a GB300)."""
import random

import pytest
import torch

import kv8_util as k8
from exact_attention_57_gb300 import fa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
MOST = 256  # arrays of one call


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def layers(n, blocks, seed):
    """n arrays of pages of codes and scales, in turn, of one or several pieces."""
    g = torch.Generator().manual_seed(seed)
    sizes = [(4096, 32, 20000, 8)[i % 4] + 16 * (i % 3) for i in range(n)]
    return [torch.randint(0, 256, (blocks, s), dtype=torch.uint8, generator=g) for s in sizes]


def requests(seed, B=9, width=6, bs=16):
    """Ragged rows over shuffled blocks, some blocks in two rows, and blocks to spare."""
    r = random.Random(seed)
    lens = [r.randrange(0, width * bs + 1) for _ in range(B)]
    blocks = sum(-(-n // bs) for n in lens) + 12
    ids = list(range(blocks))
    r.shuffle(ids)
    table = []
    for n in lens:
        need = -(-n // bs)
        table.append(ids[:need] + [-1] * (width - need))
        ids = ids[need:]
    table[3][0] = table[0][0] if lens[0] and lens[3] > bs else table[3][0]
    return table, lens, ids, blocks


def moved(arrays, moves):
    out = [x.clone() for x in arrays]
    for x, y in zip(arrays, out):
        for s, d in moves:
            y[d] = x[s]
    return out


@pytest.mark.parametrize("n", [13, 128, 256, 320])
@pytest.mark.parametrize("end", [False, True])
def test_fork_of_layers(n, end):
    """More arrays than a call takes: several calls with the same inputs, which write the
    same tables."""
    table, lens, free, blocks = requests(n)
    parents = [0, 4, 4, 7, 2, 2, 2, 8]
    arrays = layers(n, blocks, n)
    dev = [x.to(DEV) for x in arrays]
    want = k8.fork(table, lens, parents, free, 0, 16, blocks, end)
    for i in range(0, n, MOST):
        got = fa.kv_fork(ints(table), ints(lens), ints(parents), ints(free), 16, dev[i:i + MOST],
                         parents_end=end)
        assert [x.tolist() for x in got] == list(want[:3])
    assert want[3]
    for x, y in zip(moved(arrays, want[3]), dev):
        assert torch.equal(x, y.cpu())


@pytest.mark.parametrize("n", [13, 128, 256, 320])
def test_compact_of_layers(n):
    """Likewise, with a table beside the old one; in place in the last call."""
    table, lens, _, blocks = requests(n + 1)
    arrays = layers(n, blocks, n)
    dev = [x.to(DEV) for x in arrays]
    want = k8.compact(table, lens, 16, blocks)
    t, l = ints(table), ints(lens)
    for i in range(0, n, MOST):
        out = None
        if i + MOST >= n:
            out = (t, torch.empty(blocks, dtype=torch.int32, device=DEV), ints([0, 0]))
        got = fa.kv_compact(t, l, dev[i:i + MOST], 16, out=out)
        assert [x.tolist() for x in got] == list(want[:3])
    assert want[3]
    for x, y in zip(moved(arrays, want[3]), dev):
        assert torch.equal(x, y.cpu())
