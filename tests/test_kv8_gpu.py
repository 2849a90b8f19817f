"""The 8-bit cache and attention over it on the GPU against 64-bit references
(needs a GB300)."""
import math

import pytest
import torch

import kv8_util as k8
import serve_util as ref
from exact_attention_57_gb300 import fa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
F8 = torch.float8_e4m3fn


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device=DEV)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def raw(cache):
    return [c.cpu().view(torch.uint8) if c.dtype == F8 else c.cpu() for c in cache]


def same_codes(a, b):
    """Equal, -0 and +0 being one value."""
    return torch.equal(torch.where(a == 128, 0, a), torch.where(b == 128, 0, b))


# ------------------------------------------------------------------ cache
def sequence_slots(table, spans, bs):
    """Slots of tokens [lo, hi) of each row, one row after the other."""
    return torch.tensor([row[t // bs] * bs + t % bs for row, (lo, hi) in zip(table, spans)
                         for t in range(lo, hi)], dtype=torch.long)


APPENDS = [
    # spans of tokens written a sequence, Hk, d, bs, dtype
    ([(0, 1)], 1, 16, 16, "bf16"), ([(5, 6), (0, 1), (15, 16)], 3, 64, 16, "fp16"),
    ([(0, 33), (7, 90)], 2, 128, 32, "bf16"), ([(100, 300), (64, 65), (3, 130)], 8, 128, 64, "fp16"),
    ([(1, 400)], 1, 256, 128, "fp32"), ([(130, 260), (0, 128)], 2, 80, 128, "fp32"),
    ([(i % 16, i % 16 + 1) for i in range(70)], 2, 48, 16, "bf16"),
    ([(i, i + 1 + i % 3) for i in range(130)], 4, 128, 64, "fp32"),
    ([(i % 40, i % 40 + 37) for i in range(40)], 1, 112, 32, "fp16"),
    ([(0, 5000)], 2, 64, 16, "bf16"), ([(17, 3000), (9, 3000)], 4, 256, 64, "bf16"),
]


@pytest.mark.parametrize("case", APPENDS, ids=[str(i) for i in range(len(APPENDS))])
@pytest.mark.parametrize("odd", [False, True])
def test_append_and_gather(case, odd):
    """Codes and scales bit for bit, of the rows written and of those ahead of them in
    their blocks, with old scales that are powers of two or not; the rest untouched."""
    spans, Hk, d, bs, dtype = case
    g = gen(len(spans) + d)
    blocks = sum(-(-hi // bs) for _, hi in spans) + 3
    ids = torch.randperm(blocks, generator=g).tolist()
    table = []
    for _, hi in spans:
        table.append(ids[:-(-hi // bs)])
        ids = ids[-(-hi // bs):]
    slots = sequence_slots(table, spans, bs)
    T = slots.numel()
    x = torch.randn(T, 3 * Hk, d, generator=g) * torch.rand(T, 3 * Hk, 1, generator=g) * \
        2.0 ** torch.randint(-6, 6, (T, 1, 1), generator=g)
    x[T // 2, 0, :16] = 0.0
    x = x.to(DT[dtype])
    before = k8.random_store(blocks, Hk, bs, d, g, odd=odd) + k8.random_store(blocks, Hk, bs, d, g)
    cache = k8.on(before, DEV)
    kv = x.to(DEV)
    k, v = kv[:, :Hk], kv[:, 2 * Hk:]
    # rows to skip among the others, behind and ahead
    sent = torch.full((2 * T + 3,), -1, dtype=torch.long)
    at = torch.randperm(2 * T, generator=g)[:T].sort().values + 1
    sent[at] = slots
    sent[0], sent[-1] = blocks * bs, -2 ** 62
    wide = torch.full((sent.numel(),) + kv.shape[1:], math.nan, dtype=kv.dtype, device=DEV)
    wide[at.to(DEV)] = kv
    want = k8.append(x[:, :Hk], slots, *before[:2]) + k8.append(x[:, 2 * Hk:], slots, *before[2:])
    for rows, n in (((k, v, slots), cache), ((wide[:, :Hk], wide[:, 2 * Hk:], sent), k8.on(before, DEV))):
        fa.kv8_append(rows[0], rows[1], rows[2].to(DEV), *n)
        got = raw(n)
        for i in (1, 3):
            assert torch.equal(got[i], want[i])
        for i in (0, 2):
            assert same_codes(got[i], want[i])
    # read back, with rows outside the cache
    back = torch.cat([torch.tensor([blocks * bs, -1]), torch.randint(0, blocks * bs, (77,), generator=g)])
    for out in DT.values():
        gk, gv = fa.kv8_gather(back.to(DEV), *cache, dtype=out)
        for y, (c, s) in ((gk, want[:2]), (gv, want[2:])):
            val = (k8.numbers(c)[back[2:] // bs, :, back[2:] % bs] *
                   s.double()[back[2:] // bs][..., None])
            assert torch.equal(y[2:].cpu(), val.float().to(out))
            assert (y[:2] == 0).all()


def test_append_grows_and_never_drifts():
    """Token by token into one block, each larger than the last: earlier tokens keep
    their values bit for bit (until they are below 2^-6 of the scale)."""
    bs, d = 16, 32
    cache = fa.kv8_cache(1, 1, bs, d, device=DEV)
    g = gen(3)
    x = torch.randn(bs, 1, d, generator=g).clamp(-4, 4)
    x += 0.25 * x.sign()
    x = (x * 2.0 ** (torch.arange(bs) / 3).floor()[:, None, None]).bfloat16()
    y = x.to(DEV)
    codes, scales = k8.append(x[:0], torch.zeros(0), *[c.cpu().view(torch.uint8) if c.dtype == F8 else
                                                        c.cpu() for c in cache[:2]])
    for t in range(bs):
        fa.kv8_append(y[t:t + 1], y[t:t + 1], ints([t], torch.int64), *cache)
        codes, scales = k8.append(x[t:t + 1], torch.tensor([t]), codes, scales)
        got = raw(cache)
        assert same_codes(got[0][:, :, :t + 1], codes[:, :, :t + 1]) and torch.equal(got[1], scales)
        assert same_codes(got[2][:, :, :t + 1], codes[:, :, :t + 1]) and torch.equal(got[3], scales)
    # every value within half a step of what went in: 2^-4 of it, and half of the smallest
    # step, 2^-10 of the scale
    got = k8.values(*raw(cache)[:2])[0].transpose(0, 1)
    tol = 2.0 ** -4 * x.double().abs() + 2.0 ** -10 * float(scales)
    assert ((got - x.double()).abs() <= tol).all()


def test_append_of_a_block_that_begins_anew():
    """Writing a block's first token forgets its scale; a later one does not, nor does
    a scale that is no positive number count."""
    cache = fa.kv8_cache(4, 1, 16, 16, device=DEV)
    for s in (cache[1], cache[3]):
        s[:, 0] = torch.tensor([1024.0, 1024.0, math.nan, -3.0])
    x = torch.ones(4, 1, 16, device=DEV)
    fa.kv8_append(x, x, ints([0, 16 + 1, 32 + 1, 48 + 5], torch.int64), *cache)
    one = 2.0 ** -8  # 448 / 2^8 = 1.75
    assert cache[1].flatten().tolist() == cache[3].flatten().tolist() == [one, 1024.0, one, one]
    k, _ = fa.kv8_gather(ints([0, 17, 33, 53, 32, 48], torch.int64), *cache, dtype=torch.float32)
    assert k[:, 0, 0].tolist() == [1.0, 0.0, 1.0, 1.0, 0.0, 0.0]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_append_of_what_is_not_finite(dtype):
    """NaNs and infinities do not count for the scale; they are stored as 448 times it."""
    x = torch.ones(3, 2, 32)
    x[0, 0, 3], x[0, 0, 4], x[1, 0, 20] = math.inf, -math.inf, math.nan
    x[:, 1] = math.nan
    x[2, 1, 5] = -math.inf
    y = x.to(DT[dtype]).to(DEV)
    cache = fa.kv8_cache(1, 2, 16, 32, device=DEV)
    fa.kv8_append(y, y, ints([1, 2, 7], torch.int64), *cache)
    k, v = fa.kv8_gather(ints([1, 2, 7], torch.int64), *cache, dtype=torch.float32)
    top, low = 448 * 2.0 ** -8, 448 * 2.0 ** -40
    want = torch.ones(3, 2, 32)
    want[0, 0, 3], want[0, 0, 4], want[1, 0, 20] = top, -top, top
    want[:, 1] = low
    want[2, 1, 5] = -low
    assert torch.equal(k.cpu(), want) and torch.equal(v.cpu(), want)
    assert all((c.view(torch.uint8) & 127 != 127).all() for c in (cache[0], cache[2]))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("none", [False, True])
def test_append_under_scales_of_any_size(dtype, rows, none):
    """Blocks whose old scales are powers of two from 2^-40 to 2^40, rows of numbers from
    the type's smallest to 448 times the scale, with a NaN among them or not."""
    exps = [-40, -24, -17, -16, -15, -14, -13, 0, 1, 8, 13, 14, 15, 16, 24, 40]
    bs, d = 64, 32
    g = gen(rows)
    before = k8.random_store(len(exps), 1, bs, d, g)
    before[1][:, 0] = torch.tensor([2.0 ** e for e in exps])
    x = torch.randn(len(exps), rows, 1, d, generator=g)
    x = x * 2.0 ** torch.randint(-12, 1, x.shape, generator=g) * 64 * before[1][:, None, :, None]
    x[:, 0, 0, :4] = torch.tensor([0.0, -0.0, 2.0 ** -24, -2.0 ** -133])
    top = torch.finfo(DT[dtype]).max
    x = x.clamp(-top, top).to(DT[dtype])
    if none:
        x[:, rows // 2, 0, 7] = math.nan
    slots = (torch.arange(len(exps))[:, None] * bs + 3 + torch.arange(rows)).flatten()
    want = k8.append(x.flatten(0, 1), slots, *before)
    cache = k8.on(before + before, DEV)
    y = x.flatten(0, 1).to(DEV)
    fa.kv8_append(y, y, slots.to(DEV), *cache)
    got = raw(cache)
    for i in (0, 2):
        assert same_codes(got[i], want[0]) and torch.equal(got[i + 1], want[1])


def test_append_of_the_smallest_and_largest_numbers():
    """Scales end at 2^-40 and 2^40: what lies outside becomes 0 or saturates."""
    x = torch.tensor([1e-38, 448 * 2.0 ** -40, 448 * 2.0 ** 40, 3e38, 0.0, 2.0 ** -50, 2.0 ** -49.0])
    y = x[:, None, None].expand(7, 1, 16).contiguous().to(DEV)
    cache = fa.kv8_cache(7, 1, 16, 16, device=DEV)
    fa.kv8_append(y, y, 16 * torch.arange(7, device=DEV), *cache)
    assert cache[1].flatten().tolist() == [2.0 ** e for e in (-40, -40, 40, 40, -40, -40, -40)]
    k, _ = fa.kv8_gather(16 * torch.arange(7, device=DEV), *cache, dtype=torch.float32)
    assert k[:, 0, 0].tolist() == [0.0, 448 * 2.0 ** -40, 448 * 2.0 ** 40, 448 * 2.0 ** 40, 0.0, 0.0,
                                   2.0 ** -49]


# ------------------------------------------------------------------ attention
def attention_tolerance(want, lse, a, big, code_sum, v_ratio, scale, d, dtype, lv):
    """|dO|, |dLSE| allowed.  Scores: a query of 11 significant bits times a code of
    four, exact in fp32, d of them added, each addition off by 2^-23 of the sum of
    magnitudes at most (the tensor cores truncate); times two factors and the V scale's
    logarithm added (2^-22 of the score, and of 40 at most: |lv|).  A query's element
    is off by 2^-11 of itself where it has more bits than fp16 keeps (`big` holds
    sum |q||k|: only elements below 2^-14 of a row's largest, 2^-25 of that; covered
    by d 2^-23).  A weight is off by e^(2 ds) times 2^-20 (exponential, sums, quotient,
    the scale's inverse) and, rounded to fp16, by 2^-11 of itself or 2^-25 where
    it is subnormal; weights are relative to a largest of at least 2^7, which is worth
    1 / vs of it in the sum: 2^-32 vs sum |code|.  O adds half a step."""
    ds = abs(scale) * ((d + 8) * 2.0 ** -23 + 2.0 ** -21) * big + 2.0 ** -21 + 2.0 ** -22 * lv
    w = (2 * ds.transpose(0, 1)[..., None] + 2.0 ** -11 + 2.0 ** -19) * a
    tol_o = HALF_STEP[dtype] * want.abs() + w * 1.01 + 2.0 ** -32 * v_ratio * code_sum + 2.0 ** -30 * a
    if dtype == torch.float16:
        tol_o = tol_o + 2.0 ** -25
    tol_l = ds + 2.0 ** -20 + 2.0 ** -22 * torch.nan_to_num(lse, neginf=0.0).abs()
    return tol_o, tol_l


def check_attention(q, cache, table, lens, nqs, bs, d, scale, causal, o, lse, dtype, max_k=None,
                    label=""):
    K, V = k8.values(*cache[:2]), k8.values(*cache[2:])
    blocks = K.shape[0]
    G = q.shape[1] // K.shape[1]
    row = 0
    o, lse = o.double().cpu(), lse.double().cpu()
    for b, (n, nq) in enumerate(zip(lens, nqs)):
        n = max(0, min(n, len(table[b]) * bs))
        if max_k is not None:
            n = min(n, max_k)
        ids = torch.tensor([table[b][j // bs] for j in range(n)], dtype=torch.long)
        ok = (ids >= 0) & (ids < blocks)
        at = ids.clamp(0, blocks - 1), torch.arange(n) % bs
        Kb, Vb = (torch.where(ok[:, None, None], x[at[0], :, at[1]], 0.0) for x in (K, V))
        want, wl, a, big = ref.attend(q[row:row + nq].double(), Kb, Vb, scale, causal, ok)
        vs = cache[3][at[0]][ok].double()
        ratio = float(vs.max() / vs.min()) if vs.numel() else 1.0
        lv = float(vs.log2().abs().max()) if vs.numel() else 0.0
        tol_o, tol_l = attention_tolerance(
            want, wl, a, big, Vb.abs().sum(0).repeat_interleave(G, 0), ratio, scale, d, dtype, lv)
        got, gl = o[row:row + nq], lse[:, row:row + nq]
        none = wl == -math.inf
        assert torch.equal(gl == -math.inf, none), f"{label} seq {b}: rows without keys"
        assert (got.transpose(0, 1)[none] == 0).all(), f"{label} seq {b}"
        off = (got - want).abs()
        assert (off <= tol_o).all(), \
            f"{label} seq {b} n={n} nq={nq}: O off by {off.max():.3e}, {(off / tol_o).max():.2f} of the bound"
        off = torch.where(none, 0.0, (gl - wl).abs())
        assert (off <= tol_l).all(), f"{label} seq {b} n={n} nq={nq}: LSE off by {off.max():.3e}"
        row += nq


def paged(lens, bs, blocks, g, more=1):
    """Block table rows (ids shuffled over the cache); entries behind a
    sequence's last block are wild."""
    ids = torch.randperm(blocks, generator=g).tolist()
    width = max(-(-n // bs) for n in lens) + more
    table = []
    for n in lens:
        need = -(-n // bs)
        table.append(ids[:need] + [-1, 2 ** 31 - 1, -2 ** 31][:width - need]
                     + [10 ** 9] * max(0, width - need - 3))
        ids = ids[need:]
    return table


def poison(cache, table, lens, bs):
    """NaN codes in every row that no sequence holds, NaN scales of every block."""
    blocks = cache[0].shape[0]
    used = torch.zeros(blocks, bs, dtype=torch.bool)
    for row, n in zip(table, lens):
        for j in range(min(n, len(row) * bs)):
            if 0 <= row[j // bs] < blocks:
                used[row[j // bs], j % bs] = True
    for c in (cache[0], cache[2]):
        c.transpose(1, 2)[~used] = 0xFF
    for s in (cache[1], cache[3]):
        s[~used.any(1)] = math.nan


ATTN_CASES = [
    # key lengths, query lengths (None: one each, no offsets), Hq, Hk, d, bs, dtype
    ([1], None, 1, 1, 64, 16, "bf16"),
    ([5, 0, 16, 17, 300], None, 8, 2, 128, 16, "bf16"),
    ([1023], None, 32, 8, 128, 16, "bf16"),
    ([1000, 31, 64, 2, 0, 777, 129], None, 5, 1, 64, 32, "fp16"),
    ([4097, 130], None, 16, 1, 128, 64, "fp16"),
    ([200, 513], None, 40, 2, 64, 128, "bf16"),
    ([200, 513], None, 40, 2, 128, 128, "bf16"),
    ([65, 257], None, 48, 1, 128, 16, "fp16"),
    ([40] * 70, None, 4, 4, 64, 16, "bf16"),
    ([100, 9, 0, 33, 2], [4, 1, 3, 0, 5], 16, 16, 64, 32, "fp16"),
    ([300, 1, 128], [2, 8, 3], 6, 2, 128, 16, "bf16"),
    ([64, 65], [8, 2], 8, 2, 128, 64, "bf16"),
    ([130, 70], [130, 1], 4, 1, 128, 16, "bf16"),
    ([300, 500, 20, 0], [129, 257, 60, 4], 6, 3, 64, 64, "fp16"),
    ([700, 1500], [200, 3], 8, 8, 128, 32, "bf16"),
    ([1000], [1000], 2, 1, 128, 128, "fp16"),
    ([513, 100], [64, 33], 20, 4, 64, 16, "bf16"),
    ([300, 129, 40], None, 128, 1, 64, 16, "bf16"),              # the largest group
    ([300, 140, 0, 7], [3, 20, 2, 9], 100, 1, 128, 16, "fp16"),  # a token a tile
    ([400, 390, 700], [90, 1, 2], 33, 1, 64, 32, "bf16"),
    ([17 * (i % 23) for i in range(300)], None, 8, 4, 64, 16, "fp16"),   # more than a CTA's threads
    ([17 * (i % 23) for i in range(400)], None, 8, 2, 128, 16, "fp16"),
    ([3 * (i % 50) for i in range(600)], [i % 4 for i in range(600)], 8, 1, 64, 16, "bf16"),
    ([5 + i % 40 for i in range(530)], [33 + (i == 7) for i in range(530)], 2, 2, 64, 16, "bf16"),
    ([2500, 2049], [700, 2049], 8, 2, 64, 16, "fp16"),
    # tiles of one and two steps: every ring of the pipeline runs far ahead
    ([5 + i % 140 for i in range(700)], [34] * 700, 2, 2, 128, 16, "bf16"),
    ([250, 3, 130, 0] * 20, [300, 260, 129, 131] * 20, 3, 3, 128, 32, "fp16"),
    ([1537], [1537], 4, 4, 128, 64, "bf16"),
]


@pytest.mark.parametrize("case", ATTN_CASES, ids=[str(i) for i in range(len(ATTN_CASES))])
@pytest.mark.parametrize("causal,odd", [(True, False), (False, True)])
def test_attention_matches_reference(case, causal, odd):
    lens, nqs, Hq, Hk, d, bs, dt = case
    g = gen(len(lens) + Hq + d)
    blocks = sum(-(-n // bs) for n in lens) + 2
    cache = k8.random_store(blocks, Hk, bs, d, g, odd=odd) + k8.random_store(blocks, Hk, bs, d, g, odd=odd)
    table = paged(lens, bs, blocks, g)
    poison(cache, table, lens, bs)
    total = len(lens) if nqs is None else sum(nqs) + 3  # rows behind the last sequence
    q = torch.randn(total, Hq, d, generator=g).to(DT[dt])
    scale = 1.0 / math.sqrt(d)
    o = torch.full((total, Hq, d), 7.0, dtype=DT[dt], device=DEV)
    lse = torch.full((Hq, total), 7.0, device=DEV)
    cu = None
    if nqs is not None:
        cu = ints([sum(nqs[:i]) for i in range(len(nqs) + 1)])
    fa.attention_kv8(q.to(DEV), *k8.on(cache, DEV), ints(table), ints(lens), max(max(lens), 1),
                     cu_seqlens_q=cu, max_seqlen_q=1 if nqs is None else max(nqs), scale=scale,
                     causal=causal, out=o, lse=lse)
    st, word = fa.fa_fwd_status(torch.cuda.current_stream().cuda_stream)
    assert st == fa.FA_OK, word
    nq = [1] * len(lens) if nqs is None else nqs
    check_attention(q, cache, table, lens, nq, bs, d, scale, causal, o, lse, DT[dt])
    assert (o[sum(nq):] == 7.0).all() and (lse[:, sum(nq):] == 7.0).all()


def small(seed, lens=(90, 33), nqs=(1, 1), Hq=8, Hk=2, d=128, bs=16, dt="bf16", spread=3):
    g = gen(seed)
    blocks = sum(-(-n // bs) for n in lens) + 2
    cache = k8.random_store(blocks, Hk, bs, d, g, spread) + k8.random_store(blocks, Hk, bs, d, g, spread)
    table = paged(lens, bs, blocks, g)
    q = torch.randn(sum(nqs), Hq, d, generator=g).to(DT[dt])
    cu = [sum(nqs[:i]) for i in range(len(nqs) + 1)]
    return q, cache, table, cu


def call(q, cache, table, lens, cu, nqs, max_k=None, **kw):
    return fa.attention_kv8(q.to(DEV), *k8.on(cache, DEV), ints(table), ints(list(lens)),
                            max(lens) if max_k is None else max_k, cu_seqlens_q=ints(cu),
                            max_seqlen_q=max(nqs), **kw)


@pytest.mark.parametrize("nqs", [(1, 1), (5, 40)])
@pytest.mark.parametrize("scale", [0.0, -0.2, 0.6])
def test_attention_scales(nqs, scale):
    lens = (90, 133)
    q, cache, table, cu = small(11, lens, nqs)
    s = scale / 8
    o, lse = call(q, cache, table, lens, cu, nqs, scale=s)
    check_attention(q, cache, table, lens, nqs, 16, 128, s, True, o, lse, torch.bfloat16)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("nqs", [(1, 1), (3, 1), (70, 90)])
def test_attention_of_blocks_of_very_different_scales(nqs, dt):
    """Values' scales 2^-12 .. 2^12 of one another within a sequence, neighbours among
    them: rows whose weight lies on the small ones keep their accuracy."""
    lens, d, bs = (700, 333), 64, 16
    g = gen(19)
    blocks = sum(-(-n // bs) for n in lens) + 2
    kc = k8.random_store(blocks, 2, bs, d, g, 1)
    vc = k8.random_store(blocks, 2, bs, d, g, 1)
    vc = (vc[0], 2.0 ** torch.randint(-14, -2, vc[1].shape, generator=g).float())
    table = paged(lens, bs, blocks, g)
    q = (2 * torch.randn(sum(nqs), 8, d, generator=g)).to(DT[dt])
    cu = [0, nqs[0], sum(nqs)]
    o, lse = call(q, kc + vc, table, lens, cu, nqs)
    check_attention(q, kc + vc, table, lens, nqs, bs, d, d ** -0.5, True, o, lse, DT[dt])


@pytest.mark.parametrize("nqs", [(1, 1), (50, 60)])
def test_attention_of_scales_that_count_otherwise(nqs):
    """A value's scale of zero counts as 2^-40, a key's scale that is not positive as 0:
    such a block (never written, or of zeros) has scores of 0 and values of nothing."""
    lens = (90, 133)
    q, cache, table, cu = small(23, lens, nqs)
    for b, j in ((0, 1), (1, 0), (1, 5)):
        for s in (cache[1], cache[3]):
            s[table[b][j]] = 0.0
    o, lse = call(q, cache, table, lens, cu, nqs)
    cache[3][cache[3] == 0] = 2.0 ** -40
    check_attention(q, cache, table, lens, nqs, 16, 128, 128 ** -0.5, True, o, lse, torch.bfloat16)


@pytest.mark.parametrize("nqs", [(1, 1), (4, 2), (70, 90)])
def test_attention_missing_pages_and_bounds(nqs):
    """Entries outside the cache in the middle of a sequence take their tokens
    out; lengths past the table, past max_seqlen_k or below zero are cut."""
    lens = (190, 160)
    q, cache, table, cu = small(12, lens, nqs, bs=32)
    table[0][2], table[1][0], table[1][4] = -1, len(cache[0]), -2 ** 31
    o, lse = call(q, cache, table, lens, cu, nqs)
    check_attention(q, cache, table, lens, nqs, 32, 128, 128 ** -0.5, True, o, lse, torch.bfloat16)
    q, cache, table, cu = small(13, lens, nqs, bs=32)
    o, lse = call(q, cache, table, (10 ** 9, 2 ** 31 - 1), cu, nqs, max_k=100)
    check_attention(q, cache, table, (100, 100), nqs, 32, 128, 128 ** -0.5, True, o, lse,
                    torch.bfloat16)
    o, lse = call(q, cache, table, (50, 60), cu, nqs, max_k=0)
    assert (o == 0).all() and (lse == -math.inf).all()
    o, lse = call(q, cache, table, (-5, 77), cu, nqs, max_k=200)
    check_attention(q, cache, table, (0, 77), nqs, 32, 128, 128 ** -0.5, True, o, lse,
                    torch.bfloat16)


def test_attention_wild_offsets_stay_inside():
    """Query offsets outside [0, total_q]: rows are cut, nothing else is written."""
    lens, nqs = (90, 33), (4, 4)
    q, cache, table, _ = small(14, lens, nqs)
    o = torch.full((12, 8, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((8 * 12,), 7.0, device=DEV)
    call(q, cache, table, lens, [-100, 4, 2 ** 31 - 1], nqs, out=o[:8], lse=lse[:64].view(8, 8))
    assert fa.fa_fwd_status(torch.cuda.current_stream().cuda_stream)[0] == fa.FA_OK
    assert (o[8:] == 7.0).all() and (lse[64:] == 7.0).all()
    check_attention(q, cache, table, lens, nqs, 16, 128, 128 ** -0.5, True, o[:8],
                    lse[:64].view(8, 8), torch.bfloat16)


NON_FINITE = [
    # key lengths, query lengths, Hq, Hk, d, width of the table in blocks (0: what they need)
    ((300, 33), (1, 1), 8, 2, 128, 0),           # clusters
    ((300, 33), (3, 1), 4, 1, 64, 65536),        # the line, joined or not
    ((20000, 90, 5000), (1, 2, 1), 8, 2, 128, 0),
    ((70, 40), (4, 2), 8, 1, 128, 0),            # the kernel for many queries at 32 rows
    ((513, 300), (64, 200), 6, 3, 64, 0),        # whole tiles
    ((9000, 3000), (70, 90), 4, 1, 128, 0),      # tiles that several CTAs share
]


@pytest.mark.parametrize("case", NON_FINITE, ids=[str(i) for i in range(len(NON_FINITE))])
@pytest.mark.parametrize("causal", [False, True])
def test_attention_shows_nan(case, causal):
    """A query row with a NaN gets NaN for O and LSE whichever path takes it; a NaN among
    a key's codes, the rows that see this key.  The other rows are as without it."""
    lens, nqs, Hq, Hk, d, width = case
    q, cache, table, cu = small(91, lens, nqs, Hq=Hq, Hk=Hk, d=d)
    wide = ints(table)
    if width:
        wide = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
        wide[:, :len(table[0])] = ints(table)
    bad = torch.zeros(q.shape[:2], dtype=torch.bool)
    spoiled = q.clone()
    for row, head in ((0, 0), (cu[1], Hq - 1), (cu[-1] - 1, 1)):
        spoiled[row, head, 5] = math.nan
        bad[row, head] = True
    # the last key of the last sequence: its last query alone sees it when causal
    keys = [c.clone() for c in cache]
    n = lens[-1]
    keys[0][table[-1][(n - 1) // 16], Hk - 1, (n - 1) % 16, 2] = 0x7F
    blind = torch.zeros_like(bad)
    blind[(-1 if causal else cu[-2]):, -(Hq // Hk):] = True
    for x, c, off in ((spoiled, cache, bad), (q, keys, blind)):
        o, lse = fa.attention_kv8(x.to(DEV), *k8.on(c, DEV), wide, ints(list(lens)),
                                  2 ** 31 - 1, cu_seqlens_q=ints(cu), max_seqlen_q=max(nqs),
                                  causal=causal)
        o, lse = o.cpu(), lse.cpu()
        assert torch.isnan(o[off]).all() and torch.isnan(lse.t()[off]).all()
        assert not torch.isnan(o[~off]).any() and not torch.isnan(lse.t()[~off]).any()
        # the rows without one against the reference, the others as if they were whole
        clean, cl = call(q, cache, table, lens, cu, nqs, causal=causal)
        o[off], lse.t()[off] = clean.cpu()[off], cl.cpu().t()[off]
        check_attention(q, cache, table, lens, nqs, 16, d, d ** -0.5, causal, o, lse, torch.bfloat16)


@pytest.mark.parametrize("nqs", [(4, 3), (70, 50)])
def test_attention_of_queries_ahead_of_a_token_of_nan(nqs):
    """A token whose key and value are NaN, hidden from all queries but the last,
    changes nothing for the others (it is stored as a large number)."""
    lens, Hq, Hk, d, bs = (90, 133), 4, 2, 64, 16
    g = gen(95)
    blocks = sum(-(-n // bs) for n in lens)
    table = paged(lens, bs, blocks, g)
    cache = fa.kv8_cache(blocks, Hk, bs, d, device=DEV)
    slots = sequence_slots(table, [(0, n) for n in lens], bs)
    rows = [torch.randn(sum(lens), Hk, d, generator=g).bfloat16() for _ in range(2)]
    for x in rows:
        x[lens[0] - 1] = x[-1] = math.nan
    fa.kv8_append(*(x.to(DEV) for x in rows), slots.to(DEV), *cache)
    q = torch.randn(sum(nqs), Hq, d, generator=g).bfloat16()
    cpu = raw(cache)
    o, lse = call(q, cpu, table, lens, [0, nqs[0], sum(nqs)], nqs)
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    check_attention(q, cpu, table, lens, nqs, bs, d, d ** -0.5, True, o, lse, torch.bfloat16)


def test_attention_long_context():
    """A long sequence (split over many CTAs) against the float64 sums."""
    n, Hq, Hk, d, bs = 70001, 4, 1, 128, 64
    g = gen(21)
    blocks = -(-n // bs) + 1
    cache = k8.random_store(blocks, Hk, bs, d, g) + k8.random_store(blocks, Hk, bs, d, g)
    table = paged([n], bs, blocks, g)
    poison(cache, table, [n], bs)
    q = torch.randn(1, Hq, d, generator=g).bfloat16()
    o, lse = call(q, cache, table, (n,), [0, 1], (1,))
    check_attention(q, cache, table, [n], [1], bs, d, d ** -0.5, True, o, lse, torch.bfloat16)


@pytest.mark.parametrize("nq", [1, 40])
def test_cache_beyond_32_bit_offsets(nq):
    """A cache of more than 2^32 bytes of codes: blocks at both ends of it, written,
    attended to and read."""
    Hk, d, bs = 8, 128, 128
    blocks = (1 << 32) // (Hk * bs * d) + 40
    kc = torch.empty(blocks, Hk, bs, d, dtype=F8, device=DEV)
    ks = torch.empty(blocks, Hk, device=DEV)
    vc, vs = torch.empty_like(kc), torch.empty_like(ks)
    g = gen(22)
    lens, ids = [300], [blocks - 1, 0, blocks - 17]
    part = k8.random_store(3, Hk, bs, d, g) + k8.random_store(3, Hk, bs, d, g)
    for i, b in enumerate(ids):
        for c, p in zip((kc, ks, vc, vs), part):
            c.view(torch.uint8)[b] = p[i].to(DEV).view(torch.uint8)
    x = torch.randn(44, Hk, d, generator=g)
    slots = torch.tensor([ids[2] * bs + t - 256 for t in range(256, 300)])
    fa.kv8_append(x.to(DEV), x.to(DEV), slots.to(DEV), kc, ks, vc, vs)
    part = k8.append(x, slots - ids[2] * bs + 2 * bs, *part[:2]) + \
        k8.append(x, slots - ids[2] * bs + 2 * bs, *part[2:])
    q = torch.randn(nq, 16, d, generator=g).bfloat16()
    o, lse = fa.attention_kv8(q.to(DEV), kc, ks, vc, vs, ints([ids]), ints(lens), 300,
                              cu_seqlens_q=ints([0, nq]), max_seqlen_q=nq)
    check_attention(q, part, [[0, 1, 2]], lens, [nq], bs, d, d ** -0.5, True, o, lse,
                    torch.bfloat16)
    slots = torch.tensor([b * bs + 5 for b in ids])
    k, _ = fa.kv8_gather(slots.to(DEV), kc, ks, vc, vs, dtype=torch.float32)
    assert torch.equal(k.double().cpu(), k8.values(*part[:2])[:, :, 5])


@pytest.mark.parametrize("nq", [1, 40])
def test_attention_of_a_sequence_as_long_as_its_type_allows(nq):
    """A length of 2^31 - 1 in a table of 2^31 - 16 tokens is cut to 2^31 - 4096."""
    bs, d, Hq = 16, 64, 2
    width = 2 ** 27 - 1
    end = 2 ** 31 - 4096
    g = gen(77)
    cache = k8.random_store(6, 1, bs, d, g) + k8.random_store(6, 1, bs, d, g)
    table = torch.full((1, width), -1, dtype=torch.int32, device=DEV)
    at = [0, 1, 2 ** 26 + 3, end // bs - 1, end // bs, width - 1]
    table[0, at] = torch.arange(6, dtype=torch.int32, device=DEV)
    q = torch.randn(nq, Hq, d, generator=g).bfloat16()
    o, lse = fa.attention_kv8(q.to(DEV), *k8.on(cache, DEV), table, ints([2 ** 31 - 1]),
                              2 ** 31 - 1, cu_seqlens_q=ints([0, nq]), max_seqlen_q=nq)
    assert fa.fa_fwd_status(torch.cuda.current_stream().cuda_stream) == (fa.FA_OK, 0)
    small_table, n = [[0, 1, 2] + [-1] * (nq // bs + 1) + [3]], (5 + nq // bs) * bs
    check_attention(q, cache, small_table, [n], [nq], bs, d, d ** -0.5, True, o, lse, torch.bfloat16)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq", [3, 8, 12, 16])  # rows a sequence: tiles of 8 and 16
@pytest.mark.parametrize("B", [1, 17, 40, 100, 200])
def test_attention_of_small_batches(B, Hq, d):
    """Up to one sequence a CTA, by a tight and by a loose bound on the keys: the
    bound decides how many CTAs a sequence gets and who joins their parts."""
    lens = [(137 * b + 1000) % 1025 if b % 7 != 3 else b % 2 for b in range(B)]
    nqs = [1] * B
    q, cache, table, _ = small(61 + B, lens, nqs, Hq=Hq, Hk=1, d=d)
    dev = k8.on(cache, DEV)
    for max_k in (1024, 1 << 20):
        o, lse = fa.attention_kv8(q.to(DEV), *dev, ints(table), ints(lens), max_k)
        check_attention(q, cache, table, lens, nqs, 16, d, d ** -0.5, True, o, lse, torch.bfloat16,
                        label=str(max_k))
        again = fa.attention_kv8(q.to(DEV), *dev, ints(table), ints(lens), max_k)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("nq", [1, 3, 61])
@pytest.mark.parametrize("Hq,d", [(1, 64), (5, 128), (7, 64), (11, 128), (13, 64)])
@pytest.mark.parametrize("B", [1, 70, 290])
def test_attention_of_odd_rows(B, Hq, d, nq):
    """Rows that end inside a warp at the joins of clusters and inside a warp's rows of
    a tile."""
    lens = [(91 * b + 300) % 350 for b in range(B if nq < 61 else 3)]
    nqs = [nq] * len(lens)
    q, cache, table, cu = small(101 + B, lens, nqs, Hq=Hq, Hk=1, d=d)
    o, lse = call(q, cache, table, lens, cu, nqs)
    assert fa.fa_fwd_status(torch.cuda.current_stream().cuda_stream) == (fa.FA_OK, 0)
    check_attention(q, cache, table, lens, nqs, 16, d, d ** -0.5, True, o, lse, torch.bfloat16)


@pytest.mark.parametrize("B,Hq,Hk,nq,d", [(1, 32, 8, 1, 128), (3, 8, 8, 3, 64), (40, 8, 8, 1, 64),
                                          (56, 8, 8, 1, 128), (64, 16, 8, 1, 64), (5, 32, 2, 2, 128),
                                          (9, 4, 2, 50, 64), (19, 16, 1, 2, 64)])
def test_attention_workspace_is_enough(B, Hq, Hk, nq, d):
    """Whatever the bound on the keys, nothing behind the workspace is written, and the
    workspace may hold anything."""
    lens = [(211 * b + 700) % 900 for b in range(B)]
    nqs = [nq] * B
    q, cache, table, cu = small(71 + B, lens, nqs, Hq=Hq, Hk=Hk, d=d)
    need = fa.fa_fwd_kv8_workspace(B, Hq, Hk, nq, d)
    got = []
    for max_k, fill in ((len(table[0]) * 16, 0x5A), (2 ** 31 - 128, 0xFF), (2 ** 31 - 1, 0)):
        ws = torch.full((need + 4096,), fill, dtype=torch.uint8, device=DEV)
        got.append(call(q, cache, table, lens, cu, nqs, max_k=max_k, workspace=ws[:need]))
        assert (ws[need:] == fill).all()
    assert fa.fa_fwd_status(torch.cuda.current_stream().cuda_stream) == (fa.FA_OK, 0)
    for o, lse in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(lse, got[0][1])
    check_attention(q, cache, table, lens, nqs, 16, d, d ** -0.5, True, *got[0], torch.bfloat16)


def test_attention_many_queries_report_a_wait_that_runs_out():
    """A kernel that gives up waiting records it in the status word, and the
    next call is right again.  The failure is made on the host: the test hook
    leaves out the first values, and the wait limit is 0.2 s."""
    lens, nqs = (500, 300), (60, 40)
    q, cache, table, cu = small(44, lens, nqs)
    want = call(q, cache, table, lens, cu, nqs)
    stream = torch.cuda.current_stream().cuda_stream
    assert fa.fa_fwd_status(stream) == (fa.FA_OK, 0)
    try:
        fa.fa_set_test_hooks(skip_v_load=1, wait_limit_ns=200_000_000)
        call(q, cache, table, lens, cu, nqs)
    finally:
        fa.fa_set_test_hooks(0, 0)
    st, word = fa.fa_fwd_status(stream)
    assert st == fa.FA_ERR_DEVICE_TIMEOUT
    assert word & 8, word   # the skipped load was recorded
    assert word & 2, word   # the issuer gave up waiting for the values
    got = call(q, cache, table, lens, cu, nqs)
    assert fa.fa_fwd_status(stream) == (fa.FA_OK, 0)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_repeated_and_captured_calls_are_the_same_bit_for_bit():
    """Parts are joined in a fixed order; two captured calls on two streams at once,
    whose workspaces the wrapper allocated in the captures, give what one alone gives."""
    cases = [((20000, 900), (1, 2)), ((5000, 300), (200, 130))]
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for n, (lens, nqs) in enumerate(cases):
        q, cache, table, cu = small(46 + n, lens, nqs, bs=64)
        args = (q.to(DEV), *k8.on(cache, DEV), ints(table), ints(list(lens)), max(lens))
        kw = dict(cu_seqlens_q=ints(cu), max_seqlen_q=max(nqs))
        want = fa.attention_kv8(*args, **kw)
        for _ in range(3):
            got = fa.attention_kv8(*args, **kw)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        torch.cuda.synchronize()
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg, stream=streams[n]):
            got = fa.attention_kv8(*args, **kw)
        graphs.append((cg, got, want, args, kw))
    for _ in range(10):
        for cg, got, *_ in graphs:
            got[0].fill_(9.0), got[1].fill_(9.0)
        torch.cuda.synchronize()
        for (cg, *_), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                cg.replay()
        torch.cuda.synchronize()
        for _, got, want, *_ in graphs:
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_stream_of_its_own():
    side = torch.cuda.Stream()
    q, cache, table, cu = small(43, (3000, 70), (5, 60))
    args = (q.to(DEV), *k8.on(cache, DEV), ints(table), ints([3000, 70]), 3000)
    kw = dict(cu_seqlens_q=ints(cu), max_seqlen_q=60)
    want = fa.attention_kv8(*args, **kw)
    slots = torch.arange(16, device=DEV)
    rows = fa.kv8_gather(slots, *args[1:5])
    torch.cuda.synchronize()
    for _ in range(20):
        o, lse = fa.attention_kv8(*args, **kw, stream=side.cuda_stream)
        k, v = fa.kv8_gather(slots, *args[1:5], stream=side.cuda_stream)
        torch.full((1 << 20,), 9.0, device=DEV)  # would take freed memory of the current stream
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        assert torch.equal(k, rows[0]) and torch.equal(v, rows[1])


def test_wrapper_refusals():
    q, cache, table, cu = small(51)
    dev = k8.on(cache, DEV)
    t, n = ints(table), ints([90, 33])
    good = [q.to(DEV), *dev, t, n, 90]
    fa.attention_kv8(*good)

    def refused(f, args, at, bad, **kw):
        for x in bad:
            a = list(args)
            a[at] = x
            with pytest.raises((ValueError, TypeError, fa.FaError)):
                f(*a, **kw)

    refused(fa.attention_kv8, good, 0, [good[0].float(), good[0][:, :7], q, good[0].transpose(0, 1), None])
    for i in (1, 3):
        refused(fa.attention_kv8, good, i, [dev[0].view(torch.uint8), dev[0][..., :64], dev[0][:-1], None])
    for i in (2, 4):
        refused(fa.attention_kv8, good, i, [dev[1].double(), dev[1][:-1], dev[1][:, :1], dev[1].flatten()])
    refused(fa.attention_kv8, good, 5, [t.long(), t[:1], t.t(), t.cpu()])
    refused(fa.attention_kv8, good, 6, [n.long(), n[:1], n.cpu()])
    refused(fa.attention_kv8, good, 7, [-1, 1 << 40, "x"])
    for kw in (dict(out=torch.empty(2, 8, 64, device=DEV)), dict(lse=torch.empty(2, 8, device=DEV)),
               dict(workspace=torch.empty(16, dtype=torch.uint8, device=DEV)), dict(scale="x"),
               dict(cu_seqlens_q=ints([0, 1])), dict(max_seqlen_q=2), dict(out=good[0])):
        with pytest.raises((ValueError, TypeError, fa.FaError)):
            fa.attention_kv8(*good, **kw)
    x = torch.zeros(3, 2, 128, device=DEV)
    s = ints([0, 1, 2], torch.int64)
    rows = [x, x.clone(), s, *dev]
    refused(fa.kv8_append, rows, 0, [x[:2], x.half(), x[:, :1], x.cpu(), x.transpose(0, 1)])
    refused(fa.kv8_append, rows, 2, [s.int(), s[:2], s.cpu()])
    refused(fa.kv8_append, rows, 3, [fa.kv4_cache(2, 2, 16, 128, device=DEV)[0]])
    got = [s, *dev]
    refused(fa.kv8_gather, got, 0, [s.int(), s.cpu()])
    for kw in (dict(dtype=torch.int32), dict(out=(x,)), dict(out=(x, x[:1])), dict(out=(x, x)),
               dict(out=(x, x.clone()), dtype=torch.float16)):
        with pytest.raises((ValueError, TypeError, fa.FaError)):
            fa.kv8_gather(*got, **kw)
    # rows of codes off 32 bytes
    odd = torch.zeros(2 * 2 * 16 * 128 + 16, dtype=torch.uint8, device=DEV)[16:].view(F8).view(2, 2, 16, 128)
    with pytest.raises(fa.FaError):
        fa.kv8_gather(s, odd, dev[1][:2], odd, dev[3][:2])


def test_wrappers_hand_back_what_they_are_given_and_keep_nothing():
    import sys
    q, cache, table, cu = small(59)
    dev, qd = k8.on(cache, DEV), q.to(DEV)
    t, n, s = ints(table), ints([90, 33]), ints([1, 2], torch.int64)
    o, lse = torch.empty_like(qd), torch.empty(8, 2, device=DEV)
    kv = (torch.empty(2, 2, 128, device=DEV), torch.empty(2, 2, 128, device=DEV))

    def calls(given):
        if given:
            a = fa.attention_kv8(qd, *dev, t, n, 90, out=o, lse=lse)
            assert a[0] is o and a[1] is lse
            assert fa.kv8_gather(s, *dev, out=kv) is kv
            assert fa.kv8_append(*kv, s, *dev) is None
        else:
            fa.attention_kv8(qd, *dev, t, n, 90), fa.kv8_gather(s, *dev)

    held = (o, lse, kv, qd, dev[0], dev[1], t, n, s)
    for given in (True, False):
        calls(given)
        before = [sys.getrefcount(x) for x in held], torch.cuda.memory_allocated()
        for _ in range(20):
            calls(given)
        assert ([sys.getrefcount(x) for x in held], torch.cuda.memory_allocated()) == before
