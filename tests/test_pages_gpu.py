"""Pages of a cache on the GPU against plain references: copied, forked, collected and
compacted, and a server's steps with all of them (needs a GB300)."""
import random

import pytest
import torch

import kv8_util as k8
from exact_attention_57_gb300 import fa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device=DEV)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def bytes_of(blocks, sizes, seed):
    """Arrays of `blocks` pages of so many bytes, any contents (CPU)."""
    g = gen(seed)
    return [torch.randint(0, 256, (blocks, n), dtype=torch.uint8, generator=g) for n in sizes]


SIZES = [
    (16,), (4096, 32, 4096, 32), (1, 3, 4), (20, 16384), (16400, 40000), (65536, 32, 65536, 32),
    (7,) * 9, (48,) * 256,
]


# ------------------------------------------------------------------ copy
@pytest.mark.parametrize("sizes", SIZES, ids=[str(i) for i in range(len(SIZES))])
@pytest.mark.parametrize("n", [1, 37])
def test_copy(sizes, n):
    """Within a cache and to another of another size; ids outside skip their pair."""
    blocks, others = 2 * n + 5, n + 9
    a = bytes_of(blocks, sizes, n)
    ids = torch.randperm(blocks, generator=gen(1)).int()
    src, dst = ids[:n].clone(), ids[n:2 * n].clone()
    if n > 4:
        src[1], dst[2], src[3] = -1, blocks, 2 ** 31 - 1
    ok = [(s, d) for s, d in zip(src.tolist(), dst.tolist()) if 0 <= s < blocks and 0 <= d < blocks]
    dev = [x.to(DEV) for x in a]
    assert fa.kv_copy(src.to(DEV), dst.to(DEV), dev) is None
    for x, y in zip(a, dev):
        for s, d in ok:
            x[d] = x[s]
        assert torch.equal(x, y.cpu())
    b = bytes_of(others, sizes, n + 1)
    dev2 = [x.to(DEV) for x in b]
    to = torch.randperm(others, generator=gen(2)).int()[:n]
    to[0] = others - 1
    if n > 4:
        to[1:] = torch.tensor([i for i in to[1:].tolist() if i != others - 1] + [0])[:n - 1]
        to[4] = -5
        to = torch.unique(to, sorted=False)
        to = torch.cat([to, torch.full((n - to.numel(),), -1)]).int()
    fa.kv_copy(src.to(DEV), to.to(DEV), dev, to=dev2)
    for x, y, z in zip(a, b, dev2):
        for s, d in zip(src.tolist(), to.tolist()):
            if 0 <= s < blocks and 0 <= d < others:
                y[d] = x[s]
        assert torch.equal(y, z.cpu())


def test_copy_of_pages_beyond_32_bit_offsets_and_off_alignment():
    big = torch.empty(70000, 70000, dtype=torch.uint8, device=DEV)  # 4.9 GB
    one = torch.randint(0, 256, (70000,), dtype=torch.uint8, generator=gen(3))
    big[69999] = one.to(DEV)
    fa.kv_copy(ints([69999, 69999]), ints([65000, 2]), [big])
    assert torch.equal(big[65000].cpu(), one) and torch.equal(big[2].cpu(), one)
    buf = torch.randint(0, 256, (4 * 32 + 1,), dtype=torch.uint8, generator=gen(4))
    dev = buf.to(DEV)
    fa.kv_copy(ints([0]), ints([3]), [dev[1:].view(4, 32)])
    buf[1 + 96:] = buf[1:33]
    assert torch.equal(dev.cpu(), buf)


# ------------------------------------------------------------------ fork
def tables(B, width, bs, seed, blocks=None, share=False):
    """Ragged rows over distinct blocks (or, shared, any), wild behind their blocks; the
    blocks left."""
    r = random.Random(seed)
    lens = [r.choice([0, r.randrange(0, width * bs + 1), bs * r.randrange(0, width + 1)])
            for _ in range(B)]
    lens[0] = width * bs
    need = [-(-n // bs) for n in lens]
    blocks = blocks or sum(need) + 7
    ids = list(range(blocks))
    r.shuffle(ids)
    table = []
    for n in need:
        row = [r.randrange(blocks) for _ in range(n)] if share else ids[:n]
        ids = ids[0 if share else n:]
        table.append(row + [r.choice([-1, 2 ** 31 - 1, 0, -9]) for _ in range(width - n)])
    return table, lens, ids, blocks


def run_fork(table, lens, parents, free, head, bs, blocks, end, arrays):
    t, l, counts = fa.kv_fork(ints(table), ints(lens), ints(parents), ints(free), bs, arrays,
                              num_blocks=blocks, free_head=ints([head]) if head else None,
                              parents_end=end)
    return t.tolist(), l.tolist(), counts.tolist()


@pytest.mark.parametrize("B,n,width,bs,sizes", [
    (1, 1, 1, 16, (64,)), (3, 7, 4, 16, (4096, 32, 4096, 32)), (5, 256, 3, 32, (20, 48)),
    (40, 257, 9, 64, (16400, 8)), (7, 1000, 33, 16, (1, 256)), (600, 600, 2, 128, (16,) * 12),
    (2, 5, 300, 16, ()), (9, 70, 5, 16, (70000, 64)),
])
@pytest.mark.parametrize("end", [False, True])
def test_fork(B, n, width, bs, sizes, end):
    r = random.Random(B + n)
    table, lens, ids, blocks = tables(B, width, bs, seed=n)
    extra = n + 3  # blocks for the children's copies
    free = [blocks + i for i in range(extra)]
    r.shuffle(free)
    blocks += extra
    parents = [r.choice([r.randrange(B), 0, -1, B, B - 1]) for _ in range(n)]
    for head, cut, lens_ in ((0, len(free), lens), (2, max(3, n // 2), lens),
                             (0, 0, [-3 if b == 1 else 10 ** 9 if b == 2 else x
                                     for b, x in enumerate(lens)])):
        # (a length of 10^9 in a row with wild entries: its last block is whatever stands there)
        arrays = bytes_of(blocks, sizes, B)
        dev = [x.to(DEV) for x in arrays]
        got = run_fork(table, lens_, parents, free[:cut], head, bs, blocks, end, dev)
        want = k8.fork(table, lens_, parents, free[:cut], head, bs, blocks, end)
        assert got[0] == want[0] and got[1] == want[1] and got[2] == want[2]
        for x, y in zip(arrays, dev):
            before = x.clone()
            for s, d in want[3]:
                x[d] = before[s]
            assert torch.equal(x, y.cpu())


def test_fork_of_wild_entries_and_a_bad_free_list():
    """A parent's last entry outside the cache makes its children's -1; so does an id
    of the free list outside it, which is used up all the same."""
    table = [[4, 99], [1, -7], [2, 3]]
    a = torch.arange(8, dtype=torch.uint8)[:, None].expand(8, 16).contiguous()
    for end in (False, True):
        dev = a.to(DEV)
        got = run_fork(table, [20, 20, 20], [0, 1, 2, 2, 2], [6, 8, -1, 7], 0, 16, 8, end, [dev])
        want = k8.fork(table, [20, 20, 20], [0, 1, 2, 2, 2], [6, 8, -1, 7], 0, 16, 8, end)
        assert (got[0], got[1], got[2]) == want[:3]
        b = a.clone()
        for s, d in want[3]:
            b[d] = a[s]
        assert torch.equal(dev.cpu(), b)


def test_fork_of_many():
    """The most children and rows, alone their tables."""
    B = n = 65535
    lens = torch.randint(0, 40, (B,), generator=gen(5)).int()
    table = torch.randint(0, 1000, (B, 3), generator=gen(6)).int()
    parents = torch.randint(0, B, (n,), generator=gen(7)).int()
    free = torch.arange(70000).int() % 1000
    for end in (False, True):
        got = fa.kv_fork(table.to(DEV), lens.to(DEV), parents.to(DEV), free.to(DEV), 16,
                         num_blocks=1000, parents_end=end)
        want = k8.fork(table.tolist(), lens.tolist(), parents.tolist(), free.tolist(), 0, 16, 1000, end)
        assert got[0].tolist() == want[0] and got[1].tolist() == want[1]
        assert got[2].tolist() == want[2]


# ------------------------------------------------------------------ free
@pytest.mark.parametrize("B,width,bs,blocks", [
    (1, 1, 16, 1), (1, 1, 16, 2), (4, 5, 16, 31), (4, 5, 16, 33), (70, 9, 32, 1500), (300, 7, 16, 5000),
    (9, 1000, 64, 32768), (9, 1000, 64, 32769), (33, 260, 128, 100001), (3, 4, 16, 1 << 23),
    (2000, 30, 16, 40000),
])
@pytest.mark.parametrize("share", [False, True])
def test_free(B, width, bs, blocks, share):
    if not share and B * width > blocks:
        width = max(1, blocks // B)
    table, lens, _, _ = tables(B, width, bs, seed=B, blocks=blocks, share=share)
    r = random.Random(B)
    ended = [r.random() < 0.3 for _ in range(B)]
    if B > 2:
        lens[1], lens[2] = -5, 2 ** 31 - 1
        table[2][0] = table[0][0]
    for end in (None, ended):
        l = ints(lens)
        free, head = fa.kv_free(ints(table), l, blocks, bs,
                                ended=None if end is None else torch.tensor(end, device=DEV))
        want, L = k8.free_list(table, lens, bs, blocks, end)
        assert head.tolist() == [L] and torch.equal(free.cpu(), torch.tensor(want).int())
        assert l.tolist() == [0 if end and e else x for x, e in zip(lens, ended)]


def test_free_list_feeds_the_plan():
    table, lens, _, blocks = tables(6, 8, 16, seed=2)
    lens = [min(n, 100) for n in lens]
    free, head = fa.kv_free(ints(table), ints(lens), blocks + 50, 16)
    t = ints(table)
    slots, *_, counts = fa.kv_plan(ints(lens), ints([9] * 6), free, t, 16, 54, free_head=head)
    have = k8.held(table, lens, 16, blocks + 50)
    fresh = [i for row, n in zip(t.tolist(), lens) for i in row[-(-n // 16):-(-(n + 9) // 16)]]
    assert len(fresh) == counts[0] and not set(fresh) & have and (slots >= 0).all()
    assert fresh == [i for i in range(blocks + 50) if i not in have][:len(fresh)]


# ------------------------------------------------------------------ compact
@pytest.mark.parametrize("B,width,bs,blocks,sizes", [
    (1, 1, 16, 1, (16,)), (1, 1, 16, 2, (16,)), (4, 5, 16, 31, (4096, 32)), (4, 5, 16, 64, (1, 20, 16400)),
    (70, 9, 32, 1500, (256, 4)), (9, 300, 64, 32768, (16,)), (9, 300, 64, 32769, (48, 1)),
    (20, 100, 128, 100001, (16,) * 10), (3, 4, 16, 1 << 23, ()),
])
@pytest.mark.parametrize("share", [False, True])
def test_compact(B, width, bs, blocks, sizes, share):
    if not share and B * width > blocks:
        width = max(1, blocks // B)
    table, lens, _, _ = tables(B, width, bs, seed=B + 1, blocks=blocks, share=share)
    if B > 2:
        lens[1], lens[2] = -5, 2 ** 31 - 1
    arrays = bytes_of(blocks, sizes, B)
    want = k8.compact(table, lens, bs, blocks)
    moved = [x.clone() for x in arrays]
    for x, y in zip(arrays, moved):
        for s, d in want[3]:
            y[d] = x[s]
    for place in (False, True):
        dev = [x.to(DEV) for x in arrays]
        t = ints(table)
        out = None
        if place:
            out = (t, torch.empty(blocks, dtype=torch.int32, device=DEV), ints([0, 0]))
        got, new, counts = fa.kv_compact(t, ints(lens), dev, bs, num_blocks=blocks, out=out)
        assert got.tolist() == want[0] and counts.tolist() == want[2]
        assert torch.equal(new.cpu(), torch.tensor(want[1]).int())
        for x, y in zip(moved, dev):
            assert torch.equal(x, y.cpu())
        if not place:
            assert t.tolist() == table
    # compact again: nothing moves
    held = [b for b in range(B) if lens[b] > 0]
    again, new, counts = fa.kv_compact(got, ints(lens), dev, bs, num_blocks=blocks)
    assert counts.tolist() == [want[2][0], 0] and (not held or torch.equal(again, got))


@pytest.mark.parametrize("op", ["copy", "fork", "free", "compact"])
def test_captured_and_on_a_stream_of_its_own(op):
    """Captured, replayed with other contents of the same tensors, and run on a stream
    given by its handle: the results of plain calls."""
    bs, width, B = 16, 6, 5
    blocks = 64
    data = bytes_of(blocks, (4096, 32, 20), 9)
    side = torch.cuda.Stream()
    cases = []
    for seed in (3, 4):
        table, lens, ids, _ = tables(B, width, bs, seed=seed, blocks=blocks)
        r = random.Random(seed)
        ids = ids + [blocks] * 40
        cases.append([ints(table), ints(lens), ints([r.randrange(B) for _ in range(9)]), ints(ids[:9]),
                      torch.tensor([r.random() < 0.5 for _ in range(B)], device=DEV)])

    def run(s, arrays, stream=None):
        t, l, p, f, e = s
        if op == "copy":
            fa.kv_copy(t[0], f[:width], arrays, stream=stream)
            return []
        if op == "fork":
            return list(fa.kv_fork(t, l, p, f, bs, arrays, parents_end=True, stream=stream))
        if op == "free":
            return [l, *fa.kv_free(t, l, blocks, bs, ended=e, stream=stream)]
        return list(fa.kv_compact(t, l, arrays, bs, stream=stream))

    want = []
    for s in cases:
        a = [x.to(DEV) for x in data]
        want.append([x.clone() for x in run([x.clone() for x in s], a)] + a)
    held = [x.clone() for x in cases[0]]
    a = [x.to(DEV) for x in data]
    cg = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(cg, stream=side):
        got = run(held, a)
    for s, w in list(zip(cases, want)) * 2:
        for x, y in zip(held, s):
            x.copy_(y)
        for x, y in zip(a, data):
            x.copy_(y)
        cg.replay()
        torch.cuda.synchronize()
        for x, y in zip(got + a, w):
            assert torch.equal(x, y)
    a = [x.to(DEV) for x in data]
    s = [x.clone() for x in cases[1]]
    torch.cuda.synchronize()
    got = run(s, a, side.cuda_stream)
    torch.full((1 << 20,), 9.0, device=DEV)  # would take freed memory of the current stream
    torch.cuda.synchronize()
    for x, y in zip(got + a, want[1]):
        assert torch.equal(x, y)


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("kind", ["kv4", "kv8"])
@pytest.mark.parametrize("graph", [False, True])
def test_a_beam_search_step_by_step(kind, graph):
    """Two prompts, four beams each: every step forks the beams, collects the blocks that
    nobody holds, plans one token more, writes it and attends; the cache has no room for
    copies that were not collected.  Against the same steps with every beam's tokens kept
    apart and written into a cache of their own.  In the end requests end, the cache is
    compacted in place, and the attention is as before bit for bit."""
    Hq, Hk, d, bs, width, beams, steps = 8, 2, 64, 16, 6, 8, 12
    g = gen(31)
    blocks = beams * width + beams
    make, append, attend = {"kv4": (fa.kv4_cache, fa.kv4_append, fa.attention_kv4),
                            "kv8": (fa.kv8_cache, fa.kv8_append, fa.attention_kv8)}[kind]
    layers = [make(blocks, Hk, bs, d, device=DEV) for _ in range(2)]
    arrays = [x for layer in layers for x in layer]
    lens0, first = [37, 20], [0, 1]
    table = torch.full((2, width), -1, dtype=torch.int32, device=DEV)
    lens = ints([0, 0])
    free, head = fa.kv_free(table, lens, blocks, bs)
    assert head.item() == 0 and free.tolist() == list(range(blocks))
    new = torch.randn(sum(lens0), 2, 2, Hk, d, generator=g).bfloat16()  # token, layer, k or v
    slots, _, _, lens, counts = fa.kv_plan(lens, ints(lens0), free, table, bs, sum(lens0),
                                           free_head=head)
    for i, layer in enumerate(layers):
        append(new[:, i, 0].contiguous().to(DEV), new[:, i, 1].contiguous().to(DEV), slots, *layer)
    history = [[new[t] for t in range(37)], [new[t] for t in range(37, 57)]]
    state = [torch.full((beams, width), -1, dtype=torch.int32, device=DEV), ints([0] * beams)]
    state[0][:2], state[1][:2] = table, lens
    parents, tok = ints([0] * beams), torch.zeros(beams, 2, 2, Hk, d, dtype=torch.bfloat16, device=DEV)
    q = torch.zeros(beams, Hq, d, dtype=torch.bfloat16, device=DEV)

    def step():
        free, head = fa.kv_free(*state, blocks, bs)
        t, l, c = fa.kv_fork(*state, parents, free, bs, arrays, free_head=head, parents_end=True)
        slots, _, _, l2, _ = fa.kv_plan(l, ints([1] * beams) if not graph else one, free, t, bs, beams,
                                        free_head=c[1:])
        out = []
        for i, layer in enumerate(layers):
            append(tok[:, i, 0].contiguous(), tok[:, i, 1].contiguous(), slots, *layer)
            out.append(attend(q, *layer, t, l2, width * bs))
        state[0].copy_(t)
        state[1].copy_(l2)
        return out, slots

    one = ints([1] * beams)
    cg, kept = None, None
    if graph:
        save = [x.clone() for x in state + arrays]
        step()  # warm-up
        for x, y in zip(state + arrays, save):
            x.copy_(y)
        torch.cuda.synchronize()
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            kept = step()
        for x, y in zip(state + arrays, save):
            x.copy_(y)
    r = random.Random(5)
    for s in range(steps):
        n = 2 if s == 0 else beams
        choice = [0] * 4 + [1] * 4 if s == 0 else sorted(r.randrange(n) for _ in range(beams))
        parents.copy_(ints(choice))
        tok.copy_(torch.randn(tok.shape, generator=g).bfloat16())
        q.copy_(torch.randn(q.shape, generator=g).bfloat16())
        history = [history[p] + [tok[i].cpu()] for i, p in enumerate(choice)]
        if graph:
            cg.replay()
            out, slots = kept
        else:
            out, slots = step()
        assert (slots >= 0).all() and state[1].tolist() == [len(h) for h in history]
        have = k8.held(state[0].tolist(), state[1].tolist(), bs, blocks)
        assert all(0 <= i < blocks for i in have)
        # the same in a cache of each beam's own, written token by token as here
        own = make(beams * width, Hk, bs, d, device=DEV)
        flat = ints([[b * width + j for j in range(width)] for b in range(beams)])
        for i in range(2):
            prompts = [lens0[0] if len(h) > 0 and torch.equal(h[0], new[0]) else lens0[1] for h in history]
            x = [h[:p] for h, p in zip(history, prompts)]
            at = torch.cat([torch.arange(p) + b * width * bs for b, p in enumerate(prompts)]).to(DEV)
            rows = torch.stack([y for h in x for y in h])[:, i].to(DEV)
            append(rows[:, 0].contiguous(), rows[:, 1].contiguous(), at, *own)
            for t in range(s + 1):
                rows = torch.stack([h[p + t] for h, p in zip(history, prompts)])[:, i].to(DEV)
                at = ints([b * width * bs + p + t for b, p in enumerate(prompts)], torch.int64)
                append(rows[:, 0].contiguous(), rows[:, 1].contiguous(), at, *own)
            want = attend(q, *own, flat, state[1], width * bs)
            assert torch.equal(out[i][0], want[0]) and torch.equal(out[i][1], want[1])
    ended = torch.tensor([b % 3 == 1 for b in range(beams)], device=DEV)
    free, head = fa.kv_free(*state, blocks, bs, ended=ended)
    before = [attend(q, *layer, *state, width * bs) for layer in layers]
    t, new_ids, counts = fa.kv_compact(*state, arrays, bs, out=(state[0], torch.empty_like(free),
                                                               ints([0, 0])))
    assert counts[0] == head[0]
    for layer, (o, lse) in zip(layers, before):
        small = [x[:int(counts[0])].contiguous() for x in layer]  # the rest can be given back
        got = attend(q, *small, *state, width * bs)
        assert torch.equal(got[0], o) and torch.equal(got[1], lse)
        assert (o[ended] == 0).all() and (o[~ended] != 0).any()


def test_wrapper_refusals():
    table, lens, ids, blocks = tables(4, 5, 16, seed=8, blocks=40)
    t, l, p, f = ints(table), ints(lens), ints([0, 1]), ints(ids[:4] or [0])
    a = torch.zeros(40, 64, dtype=torch.uint8, device=DEV)

    def refused(f, *args, **kw):
        with pytest.raises((ValueError, TypeError, fa.FaError)):
            f(*args, **kw)

    fa.kv_copy(p, p + 2, [a])
    for bad in ((p.long(), p, [a]), (p, p[:1], [a]), (p, p, []), (p, p, [a, a]), (p, p, [a.t()]),
                (p, p, [a.cpu()]), (p, p, [a, a[:20].clone()]), (p, p, [a, 3]), (p.cpu(), p.cpu(), [a]),
                (p, p, 3), (a[0, :8].view(torch.int32), p, [a]), (p[:0], p[:0], [a])):
        refused(fa.kv_copy, *bad)
    refused(fa.kv_copy, p, p, [a], to=[a[:, :32].contiguous()])
    refused(fa.kv_copy, p, p, [a[:20]], to=[a[10:]])
    refused(fa.kv_copy, p, p, [torch.zeros(40, 1, device=DEV) for _ in range(257)])
    fa.kv_fork(t, l, p, f, 16, [a])
    for bad in ((t.long(), l, p, f, 16, [a]), (t, l[:2], p, f, 16, [a]), (t, l, p.long(), f, 16, [a]),
                (t, l, p, f.cpu(), 16, [a]), (t, l, p, f, 24, [a]), (t, l, p[:0], f, 16, [a]),
                (t, l, p, f, 16), (t.t(), l, p, f, 16, [a]), (t, l, p, f, 16, [t])):
        refused(fa.kv_fork, *bad)
    refused(fa.kv_fork, t, l, p, f, 16, [a], num_blocks=41)
    refused(fa.kv_fork, t, l, p, f, 16, num_blocks=0)
    refused(fa.kv_fork, t, l, p, f, 16, [a], free_head=p.long())
    good = fa.kv_fork(t, l, p, f, 16, [a])
    assert fa.kv_fork(t, l, p, f, 16, [a], out=good) is good
    for i in range(3):
        bad = list(good)
        bad[i] = bad[i][:-1]
        refused(fa.kv_fork, t, l, p, f, 16, [a], out=bad)
    refused(fa.kv_fork, t, l, p, f, 16, [a], out=(t[:2], good[1], good[2]))  # on its own input
    fa.kv_free(t, l, 40, 16)
    for bad in ((t.long(), l, 40, 16), (t, l.cpu(), 40, 16), (t, l, 0, 16), (t, l, 40, 17),
                (t, l, (1 << 23) + 1, 16), (t, l, -1, 16)):
        refused(fa.kv_free, *bad)
    refused(fa.kv_free, t, l, 40, 16, ended=ints([0, 1, 0, 1]))
    refused(fa.kv_free, t, l, 40, 16, ended=torch.zeros(3, dtype=torch.bool, device=DEV))
    got = fa.kv_free(t, l, 40, 16)
    assert fa.kv_free(t, l, 40, 16, out=got) is got
    refused(fa.kv_free, t, l, 40, 16, out=(got[0][:-1], got[1]))
    refused(fa.kv_free, t, l, 40, 16, out=(t.flatten()[:20], got[1]))
    fa.kv_compact(t, l, [a], 16)
    for bad in ((t.long(), l, [a], 16), (t, l[:3], [a], 16), (t, l, [a], 8), (t, l, [], 16),
                (t, l, [a, a], 16)):
        refused(fa.kv_compact, *bad)
    refused(fa.kv_compact, t, l, [a], 16, num_blocks=39)
    refused(fa.kv_compact, t, l, [], 16, num_blocks=(1 << 23) + 1)
    refused(fa.kv_compact, t, l, [a], 16, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    refused(fa.kv_compact, t, l, [a], 16, workspace=a)
