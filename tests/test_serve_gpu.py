"""The serving operators on the GPU against 64-bit references: block tables,
rotary positions, the 4-bit cache, attention over it, and a run of them
together (needs a GB300)."""
import math
import random

import pytest
import torch

import serve_util as ref
from exact_attention_57_gb300 import fa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device=DEV)


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------ plan
def run_plan(cached, new, free, table, bs, cap, head=0, **kw):
    t = ints(table)
    got = fa.kv_plan(ints(cached), ints(new), ints(free), t, bs, cap,
                     free_head=ints([head]) if head else None, **kw)
    return [t.tolist()] + [x.tolist() for x in got]


def check_plan(cached, new, free, table, bs, cap, head=0):
    got = run_plan(cached, new, free, table, bs, cap, head)
    want = ref.plan(cached, new, free, head, table, bs, cap)
    for name, a, b in zip(("table", "slots", "positions", "cu", "lens", "counts"), got, want):
        assert a == list(b), name


def plan_case(B, bs, top_cached, top_new, seed, spare=3, width_more=0):
    r = random.Random(seed)
    cached = [r.randrange(0, top_cached + 1) for _ in range(B)]
    new = [r.choice([0, 1, r.randrange(0, top_new + 1)]) for _ in range(B)]
    width = max(-(-(c + n) // bs) for c, n in zip(cached, new)) + width_more or 1
    need = sum(-(-(c + n) // bs) + -(-c // bs) for c, n in zip(cached, new)) + spare
    ids = list(range(need))
    r.shuffle(ids)
    table = []
    for c in cached:
        have = -(-c // bs)
        table.append(ids[:have] + [-7] * (width - have))
        ids = ids[have:]
    return cached, new, ids, table


@pytest.mark.parametrize("B,bs,top_cached,top_new,extra", [
    (1, 16, 0, 1, 0), (1, 16, 15, 40, 5), (3, 32, 100, 70, 1), (17, 64, 1000, 500, 0),
    (256, 16, 300, 2, 40), (257, 128, 700, 3, 0), (1000, 16, 60, 9, 2000), (5, 16, 10, 9000, 77),
    (2, 16, 0, 0, 3),
])
def test_plan_matches_reference(B, bs, top_cached, top_new, extra):
    cached, new, free, table = plan_case(B, bs, top_cached, top_new, seed=B + bs)
    cap = max(1, sum(new) + extra)
    check_plan(cached, new, free or [0], table, bs, cap)


def test_plan_many_requests():
    """More requests than one CTA takes at a time, each CTA's rounds apart."""
    B, bs = 20000, 16
    r = random.Random(1)
    cached = [r.randrange(0, 40) for _ in range(B)]
    new = [r.choice([0, 1, 1, 2, 30]) for _ in range(B)]
    width = 5
    table = [[b * 5 + j for j in range(width)] for b in range(B)]
    free = list(range(10 ** 6, 10 ** 6 + 60000))
    check_plan(cached, new, free, table, bs, sum(new) + 5000)


@pytest.mark.parametrize("bs", [16, 128])
def test_plan_capacity_ends_anywhere(bs):
    """Table entries of blocks whose tokens lie behind the capacity are written all
    the same, in whichever round of requests and inside whichever block it ends."""
    cached, new, free, table = plan_case(600, bs, 3 * bs, 2 * bs, seed=bs)
    total = sum(new)
    for cap in (1, 15, 17, 1023, 1024, 1025, sum(new[:256]), sum(new[:256]) + 1, total // 2,
                total - 1, total):
        check_plan(cached, new, free, table, bs, cap)


def test_plan_head_short_list_full_table_and_small_capacity():
    cached, new, free, table = plan_case(9, 16, 50, 60, seed=8)
    check_plan(cached, new, [5, 6, 7] + free, table, 16, sum(new), head=3)
    check_plan(cached, new, free[:4], table, 16, sum(new) + 1)          # blocks run out
    check_plan(cached, new, free[:4], table, 16, sum(new) + 1, head=2)
    check_plan(cached, new, free, table, 16, 7)                         # more tokens than capacity
    # a table too narrow: tokens past it get no slot and no block
    check_plan([30, 5, 40], [10, 60, 3], list(range(50, 70)),
               [[1, 2], [3, -1], [4, 5]], 16, 80)
    # negative lengths count as none
    check_plan([-5, 4, 20], [3, -2, 1], [9, 8, 7], [[-1, -1], [1, -1], [2, 3]], 16, 6)


def test_plan_without_free_blocks_and_twice():
    table = [[4, -1], [6, 7]]
    t = ints(table)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    for _ in range(2):  # the call keeps nothing: the same again
        got = fa.kv_plan(ints([3, 20]), ints([2, 20]), none, t, 16, 30)
        want = ref.plan([3, 20], [2, 20], [], 0, table, 16, 30)
        assert t.tolist() == want[0] and [x.tolist() for x in got] == [list(x) for x in want[1:]]


# ------------------------------------------------------------------ rotary
def ladder(rot, axes):
    half = rot // 2
    return ([10000.0 ** (-2.0 * i / rot) for i in range(half)],
            [min(axes - 1, i * axes // half) for i in range(half)])


ROPE_CASES = [
    # B, N, Hq, Hk, d, rot, axes, interleaved
    (1, 1, 1, 0, 64, 64, 1, False), (2, 37, 4, 2, 128, 128, 3, False), (1, 5, 3, 1, 72, 72, 2, False),
    (3, 11, 2, 2, 80, 64, 2, True), (2, 9, 5, 5, 256, 256, 4, False), (1, 300, 8, 1, 96, 48, 3, True),
    (2, 3, 1, 1, 2, 2, 1, False), (1, 7, 2, 1, 30, 14, 2, True), (1, 6, 17, 4, 33, 10, 1, False),
    (1, 1000, 40, 8, 128, 128, 1, True),
]


@pytest.mark.parametrize("case", ROPE_CASES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("inverse", [False, True])
def test_rotary_matches_reference(case, dtype, inverse):
    """Tolerance: the angle's fraction of a turn is exact to 2^-32 before it
    is rounded to fp32 (half a unit of an angle below pi: 2^-24 * pi), sine
    and cosine are within 2 units (2^-22), the products and their sum round
    three times: with s = |x1| + |x2|, off by (2^-24 pi + 2^-22 + 3 * 2^-24) s
    < 2^-21 s, and half a step of the output type."""
    B, N, Hq, Hk, d, rot, axes, inter = case
    g = gen(N + d)
    q, k = (torch.randn(B, h, N, d, generator=g).to(DT[dtype]) for h in (Hq, max(Hk, 1)))
    pos = torch.randint(-70, 200000, (axes, B, N), generator=g, dtype=torch.int32)
    pos[0, 0, 0] = 2 ** 31 - 1
    freq, axis = ladder(rot, axes)
    table = fa.rotary_table(freq, axis, device=DEV)
    fn = fa.rotary_backward if inverse else fa.rotary
    gq, gk = fn(q.to(DEV), k.to(DEV) if Hk else None, pos.to(DEV), table, interleaved=inter)
    for x, y in ((q, gq),) + (((k, gk),) if Hk else ()):
        want = ref.rotate(x, pos, torch.tensor(freq, dtype=torch.float64), torch.tensor(axis), rot,
                          inter, inverse)
        s = x.double().abs()
        if inter:
            pair = s[..., :rot].unflatten(-1, (-1, 2)).sum(-1).repeat_interleave(2, -1)
        else:
            pair = (s[..., :rot // 2] + s[..., rot // 2:rot]).repeat(1, 1, 1, 2)
        tol = HALF_STEP[DT[dtype]] * want.abs() + 2.0 ** -25
        tol[..., :rot] += 2.0 ** -21 * pair
        assert ((y.double().cpu() - want).abs() <= tol).all()
        assert torch.equal(y[..., rot:].cpu(), x[..., rot:])


def test_rotary_layouts_strides_and_in_place():
    """Token-major slices of a fused projection, at an odd offset too (the
    scalar path), in place and into another slice, against the contiguous
    call, bit for bit; everything around them stays as it was."""
    T, Hq, Hk, d = 13, 4, 2, 64
    g = gen(4)
    table = fa.rotary_table(*ladder(64, 2), device=DEV)
    pos = torch.randint(0, 5000, (2, T), generator=g, dtype=torch.int32).to(DEV)
    for shift in (0, 1, 4):
        flat = torch.randn(T * (Hq + 2 * Hk) * d + 8, generator=g).bfloat16().to(DEV)
        qkv = flat[shift:shift + T * (Hq + 2 * Hk) * d].view(T, Hq + 2 * Hk, d)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
        bh = [x.transpose(0, 1)[None].contiguous() for x in (q, k)]
        wq, wk = fa.rotary(*bh, pos.view(2, 1, T), table)
        oq, ok = fa.rotary(q, k, pos, table)
        assert torch.equal(oq, wq[0].transpose(0, 1)) and torch.equal(ok, wk[0].transpose(0, 1))
        v0, edge = v.clone(), flat[T * (Hq + 2 * Hk) * d + shift:].clone()
        a, b = fa.rotary(q, k, pos, table, q_out=q, k_out=k)
        assert a is q and torch.equal(q, oq) and torch.equal(k, ok) and torch.equal(v, v0)
        assert torch.equal(flat[T * (Hq + 2 * Hk) * d + shift:], edge)
        # there and back is the input, up to two roundings of the type
        r, _ = fa.rotary_backward(oq, None, pos, table)
        assert (r.double() - bh[0][0].transpose(0, 1).double()).abs().max() <= 4 * 2 * 2.0 ** -8 * 2


def test_rotary_from_one_slice_of_a_buffer_into_another():
    """Outputs in other columns of the rows that hold the inputs, and the halves of
    one row in place; an output on the other tensor is refused, nothing written."""
    T, H, d = 11, 3, 64
    g = gen(8)
    table = fa.rotary_table(*ladder(64, 1), device=DEV)
    pos = torch.randint(0, 5000, (1, T), generator=g, dtype=torch.int32).to(DEV)
    buf = torch.randn(T, 4 * H, d, generator=g).bfloat16().to(DEV)
    q, k, a, b = (buf[:, n * H:(n + 1) * H] for n in range(4))
    want = fa.rotary(q, k, pos, table)
    before = buf.clone()
    for bad in (dict(q_out=k), dict(q_out=q, k_out=q), dict(q_out=a, k_out=a), dict(k_out=q),
                dict(q_out=buf[:, 2 * H - 1:3 * H - 1])):
        with pytest.raises(fa.FaError):
            fa.rotary(q, k, pos, table, **bad)
    assert torch.equal(buf, before)
    fa.rotary(q, k, pos, table, q_out=a, k_out=b)
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    assert torch.equal(buf[:, :2 * H], before[:, :2 * H])
    both = torch.stack([q, k], 2)  # [T, H, 2, d]: a head's q beside its k
    fa.rotary(both[:, :, 0], both[:, :, 1], pos, table, q_out=both[:, :, 0], k_out=both[:, :, 1])
    assert torch.equal(both[:, :, 0], want[0]) and torch.equal(both[:, :, 1], want[1])


def test_rotary_gradient_is_the_transpose():
    """<rotary(x), y> = <x, rotary_backward(y)>, and differences: the rotation
    is linear, so rotary(x + h e) - rotary(x) over h is column e for any h."""
    B, H, N, d = 1, 2, 5, 32
    g = gen(6)
    x, y = (torch.randn(B, H, N, d, generator=g).to(DEV) for _ in range(2))
    pos = torch.randint(0, 900, (1, B, N), generator=g, dtype=torch.int32).to(DEV)
    table = fa.rotary_table(*ladder(d, 1), device=DEV)
    fx = fa.rotary(x, None, pos, table)[0]
    by = fa.rotary_backward(y, None, pos, table)[0]
    lhs, rhs = (fx.double() * y.double()).sum(), (x.double() * by.double()).sum()
    # every element within 2^-21 (|x1| + |x2|) (see above): 320 products of numbers below 6
    assert abs(lhs - rhs) <= 2 * 320 * 2.0 ** -21 * 12 * 6
    e = torch.zeros_like(x)
    e[0, 1, 3, 7] = 1.0
    col = (fa.rotary(x + e, None, pos, table)[0].double() - fx.double())
    lhs, rhs = (col * y.double()).sum(), by[0, 1, 3, 7].double()
    assert abs(lhs - rhs) <= 2 * 2 * 2.0 ** -21 * 12 * 6 + 2.0 ** -21 * 12


# ------------------------------------------------------------------ cache
def rows_of(cache, slots, bs):
    """(codes, scales) rows [R, Hk, ...] of K and V at slots, on the CPU."""
    s = slots.cpu()
    return [c.cpu()[s // bs, :, s % bs] for c in cache]


CACHE_CASES = [
    # T, Hk, d, bs, dtype, k_exp, v_exp
    (1, 1, 16, 16, "bf16", 0, 0), (37, 3, 64, 16, "fp16", 0, 0), (65, 8, 128, 64, "bf16", 0, 0),
    (100, 2, 48, 32, "fp32", 0, 0), (9, 1, 256, 128, "fp32", -4, 3), (33, 2, 80, 16, "bf16", 5, -6),
    (300, 4, 128, 32, "fp32", 0, 0),
]


@pytest.mark.parametrize("T,Hk,d,bs,dtype,ke,ve", CACHE_CASES)
def test_cache_write_and_read(T, Hk, d, bs, dtype, ke, ve):
    """Codes and scales are the nearest ones bit for bit (fp32 divisions and
    the rounded products decide no border differently from 64 bits: the proof
    is beside the kernel); reading back is exact."""
    g = gen(T + d)
    blocks = T // bs + 3
    x = torch.randn(T, 3 * Hk, d, generator=g) * torch.rand(T, 3 * Hk, 1, generator=g)
    x[:, :, ::16] *= 30
    x[T // 2, 0, :16] = 0.0                       # a group of zeros
    x[T // 3, Hk - 1, :16] = torch.tensor([6.0, 0.25, -0.75, 1.25, -1.75, 2.5, 3.5, -5.0] * 2)  # ties
    x[T // 4, 0, d - 16:] *= 1e-4                 # scales in the subnormal range
    x = x.to(DT[dtype])
    kv = x.to(DEV)
    k, v = kv[:, :Hk], kv[:, 2 * Hk:]
    cache = fa.kv4_cache(blocks, Hk, bs, d, device=DEV)
    for c in cache:
        c.fill_(0xAB)
    slots = torch.randperm(blocks * bs, generator=g)[:T]
    skip = torch.rand(T, generator=g) < 0.2
    sent = torch.where(skip, torch.tensor([-1, -9, blocks * bs])[torch.arange(T) % 3], slots)
    fa.kv4_append(k, v, sent.to(DEV), *cache, k_exp=ke, v_exp=ve)
    want = ref.quantise(x[:, :Hk], ke) + ref.quantise(x[:, 2 * Hk:], ve)
    got = rows_of(cache, slots, bs)
    for a, b in zip(got, want):
        # -0 and +0 are one value: compare codes where not both zero
        if a.shape[-1] == d // 2:
            for sh in (0, 4):
                p, q = (a >> sh) & 15, (b >> sh) & 15
                assert torch.equal(torch.where(p == 8, 0, p)[~skip], torch.where(q == 8, 0, q)[~skip])
        else:
            assert torch.equal(a[~skip], b[~skip])
        assert (a[skip] == 0xAB).all()
    # untouched rows
    mask = torch.ones(blocks * bs, dtype=torch.bool)
    mask[slots[~skip]] = False
    rest = mask.nonzero().flatten()
    for c in rows_of(cache, rest, bs):
        assert (c == 0xAB).all()
    # read back, with rows outside the cache
    back = torch.cat([torch.where(skip, -1, slots), torch.tensor([blocks * bs, -1])])
    for out in DT.values():
        gk, gv = fa.kv4_gather(back.to(DEV), *cache, dtype=out, k_exp=ke, v_exp=ve)
        for y, (c, s), e in ((gk, want[:2], ke), (gv, want[2:], ve)):
            val = ref.values(c, s, e)
            val[skip] = 0
            if out == torch.float16:
                # an exponent can move values below fp16's normal range
                assert ((y[:T].double().cpu() - val).abs() <= 2.0 ** -25).all()
            else:
                assert torch.equal(y[:T].double().cpu(), val)
            assert (y[T:] == 0).all()


def test_cache_borders_of_every_type():
    """x at s * border for every scale and border, and one step of its type to
    either side: the code is the nearest value's, ties the even one's."""
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        rows = []
        for s in ref.SCALES[8::3].tolist():
            if dtype == torch.float16 and 6 * s > 6e4:
                continue
            row = [6.0 * s]
            for b in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
                t = torch.tensor(b * s, dtype=dtype)
                row += [float(t), float(torch.nextafter(t, torch.tensor(9e9, dtype=dtype)))]
            row.append(-float(torch.nextafter(torch.tensor(2.5 * s, dtype=dtype),
                                              torch.tensor(0.0, dtype=dtype))))
            rows.append(row)
        x = torch.tensor(rows, dtype=torch.float64).to(dtype)[:, None]
        T = x.shape[0]
        cache = fa.kv4_cache(8, 1, 16, 16, device=DEV)
        slots = torch.arange(T)
        fa.kv4_append(x.to(DEV), (-x).contiguous().to(DEV), slots.to(DEV), *cache)
        got = rows_of(cache, slots, 16)
        for a, b in zip(got, ref.quantise(x) + ref.quantise(-x)):
            assert torch.equal(a, b)


def test_cache_non_finite_input_saturates():
    x = torch.ones(1, 1, 32)
    x[0, 0, 3], x[0, 0, 4], x[0, 0, 20] = math.inf, -math.inf, math.nan
    for dtype in DT.values():
        cache = fa.kv4_cache(1, 1, 16, 32, device=DEV)
        y = x.to(dtype).to(DEV)
        fa.kv4_append(y, y, ints([2], torch.int64), *cache)
        k, v = fa.kv4_gather(ints([2], torch.int64), *cache, dtype=torch.float32)
        assert torch.isfinite(k).all() and torch.equal(k, v)
        assert k[0, 0, 3] == 6 * 448 and k[0, 0, 4] == -6 * 448 and k[0, 0, 0] == 0
        # the second group's scale is e4m3(1 / 6) = 0.171875; the NaN is stored as +6
        assert k[0, 0, 20] == 6 * 0.171875 and k[0, 0, 21] == 6 * 0.171875


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_cache_groups_of_nothing_but_nan(dtype):
    """Stored as zeros in every type, with zeros or numbers that round to zero
    among them too; other groups of the row are as they were."""
    nan = math.nan
    x = torch.ones(3, 1, 64)
    x[0, 0, 16:32] = nan
    x[1, 0, :] = nan
    x[2, 0, 32:48] = torch.tensor([nan, 0.0, -nan, 1e-7] * 4)
    x[2, 0, 48:] = torch.tensor([nan] * 15 + [6.0])
    y = x.to(DT[dtype]).to(DEV)
    cache = fa.kv4_cache(1, 1, 16, 64, device=DEV)
    for c in cache:
        c.fill_(0xAB)
    slots = ints([3, 0, 15], torch.int64)
    fa.kv4_append(y, y, slots, *cache)
    k, v = fa.kv4_gather(slots, *cache, dtype=torch.float32)
    one = 6 * 0.171875  # e4m3(1 / 6) times e2m1(1 / that) = 6
    want = torch.full((3, 1, 64), one)
    want[0, 0, 16:32] = want[1] = 0.0
    want[2, 0, 32:48] = 0.0
    want[2, 0, 48:] = 6.0
    assert torch.equal(k.cpu(), want) and torch.equal(v.cpu(), want)
    for c in (cache[1], cache[3]):
        assert ((c[0, 0, [3, 0, 15]] & 0x7F) != 0x7F).all()


@pytest.mark.parametrize("nqs", [(4, 3), (70, 50)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_attention_of_queries_ahead_of_a_token_of_nan(nqs, dtype):
    """A token whose key and value are NaN, hidden from all queries but the last,
    changes nothing for the others."""
    lens, Hq, Hk, d, bs = (90, 133), 4, 2, 64, 16
    g = gen(95)
    blocks = sum(-(-n // bs) for n in lens)
    table = paged(lens, bs, blocks, g)
    cache = fa.kv4_cache(blocks, Hk, bs, d, device=DEV)
    slots = torch.tensor([t[j // bs] * bs + j % bs for t, n in zip(table, lens) for j in range(n)])
    rows = [torch.randn(sum(lens), Hk, d, generator=g).to(DT[dtype]) for _ in range(2)]
    for x in rows:
        x[lens[0] - 1] = x[-1] = math.nan
    fa.kv4_append(*(x.to(DEV) for x in rows), slots.to(DEV), *cache)
    q = torch.randn(sum(nqs), Hq, d, generator=g).bfloat16()
    cpu = [c.cpu() for c in cache]
    o, lse = call(q, cpu, table, lens, [0, nqs[0], sum(nqs)], nqs)
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    check_attention(q, cpu, table, lens, nqs, bs, d, d ** -0.5, True, o, lse, torch.bfloat16)


# ------------------------------------------------------------------ attention
def random_cache(blocks, Hk, bs, d, g):
    """Every code, scales 2^-2 .. 1: scores and values of the usual size."""
    def one():
        return (torch.randint(0, 256, (blocks, Hk, bs, d // 2), generator=g, dtype=torch.uint8),
                torch.randint(0x28, 0x39, (blocks, Hk, bs, d // 16), generator=g, dtype=torch.uint8))
    return one() + one()


def attention_tolerance(want, lse, a, big, scale, d, dtype):
    """|dO|, |dLSE| allowed.  Scores: products of at most 17 significant bits
    (fp16 or bf16 query, six-bit key), exact in fp32, d of them added: each
    addition is off by 2^-23 of the sum of magnitudes at most (the tensor
    cores truncate), so |ds| <= scale (d + 8) 2^-23 sum|q||k|; a weight is off
    by e^(2 ds) times 2^-21 (exponential, sum and quotient) and, rounded to
    fp16, by 2^-11 of itself.  O adds half a step of its type and 2^-24 for
    fp16's subnormals."""
    ds = abs(scale) * (d + 8) * 2.0 ** -23 * big + 2.0 ** -21
    w = (2 * ds.transpose(0, 1)[..., None] + 2.0 ** -11 + 2.0 ** -20) * a
    tol_o = HALF_STEP[dtype] * want.abs() + w * 1.01 + 2.0 ** -24 * (1 + a)
    tol_l = ds + 2.0 ** -20 + 2.0 ** -22 * torch.nan_to_num(lse, neginf=0.0).abs()
    return tol_o, tol_l


def check_attention(q, cache, table, lens, nqs, bs, d, scale, causal, o, lse, dtype, exps=(0, 0),
                    max_k=None, label=""):
    """Every row of every sequence against the reference."""
    K, V = ref.values(cache[0], cache[1], exps[0]), ref.values(cache[2], cache[3], exps[1])
    blocks = K.shape[0]
    row = 0
    o, lse = o.double().cpu(), lse.double().cpu()
    for b, (n, nq) in enumerate(zip(lens, nqs)):
        n = min(n, len(table[b]) * bs)
        if max_k is not None:
            n = min(n, max_k)
        ids = torch.tensor([table[b][j // bs] for j in range(n)], dtype=torch.long)
        ok = (ids >= 0) & (ids < blocks)
        at = ids.clamp(0, blocks - 1), torch.arange(n) % bs
        Kb, Vb = K[at[0], :, at[1]], V[at[0], :, at[1]]
        Vb = torch.where(ok[:, None, None], Vb, 0.0)
        Kb = torch.where(ok[:, None, None], Kb, 0.0)
        want, wl, a, big = ref.attend(q[row:row + nq].double(), Kb, Vb, scale, causal, ok)
        tol_o, tol_l = attention_tolerance(want, wl, a, big, scale, d, dtype)
        got, gl = o[row:row + nq], lse[:, row:row + nq]
        none = wl == -math.inf
        assert torch.equal(gl == -math.inf, none), f"{label} seq {b}: rows without keys"
        assert (got.transpose(0, 1)[none] == 0).all(), f"{label} seq {b}"
        off = (got - want).abs()
        assert (off <= tol_o).all(), f"{label} seq {b} n={n} nq={nq}: O off by {off.max():.3e}"
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


def poison_tails(cache, table, lens, bs):
    """NaN scales and full codes in every row no sequence holds."""
    blocks, Hk = cache[0].shape[:2]
    used = torch.zeros(blocks, bs, dtype=torch.bool)
    for row, n in zip(table, lens):
        for j in range(min(n, len(row) * bs)):
            if 0 <= row[j // bs] < blocks:
                used[row[j // bs], j % bs] = True
    for c in cache:
        c.transpose(1, 2)[~used] = 0xFF


ATTN_CASES = [
    # key lengths, query lengths (None: one each, no offsets), Hq, Hk, d, bs, dtype
    ([1], None, 1, 1, 64, 16, "bf16"),
    ([5, 0, 16, 17, 300], None, 8, 2, 128, 16, "bf16"),
    ([1023], None, 32, 8, 128, 16, "bf16"),
    ([1000, 31, 64, 2, 0, 777, 129], None, 5, 1, 64, 32, "fp16"),
    ([4097, 130], None, 16, 1, 128, 64, "fp16"),
    ([200, 513], None, 40, 2, 64, 128, "bf16"),
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
    ([3 * (i % 50) for i in range(600)], [i % 4 for i in range(600)], 8, 1, 64, 16, "bf16"),
    ([5 + i % 40 for i in range(530)], [33 + (i == 7) for i in range(530)], 2, 2, 64, 16, "bf16"),
    ([2500, 2049], [700, 2049], 8, 2, 64, 16, "fp16"),
    # tiles of one and two steps: every ring of the pipeline runs far ahead
    ([5 + i % 140 for i in range(700)], [34] * 700, 2, 2, 128, 16, "bf16"),
    ([250, 3, 130, 0] * 20, [300, 260, 129, 131] * 20, 3, 3, 128, 32, "fp16"),
    ([1537], [1537], 4, 4, 128, 64, "bf16"),
]


@pytest.mark.parametrize("case", ATTN_CASES, ids=[str(i) for i in range(len(ATTN_CASES))])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_matches_reference(case, causal):
    lens, nqs, Hq, Hk, d, bs, dt = case
    g = gen(len(lens) + Hq + d)
    blocks = sum(-(-n // bs) for n in lens) + 2
    cache = random_cache(blocks, Hk, bs, d, g)
    table = paged(lens, bs, blocks, g)
    poison_tails(cache, table, lens, bs)
    total = len(lens) if nqs is None else sum(nqs) + 3  # rows behind the last sequence
    q = torch.randn(total, Hq, d, generator=g).to(DT[dt])
    scale = 1.0 / math.sqrt(d)
    o = torch.full((total, Hq, d), 7.0, dtype=DT[dt], device=DEV)
    lse = torch.full((Hq, total), 7.0, device=DEV)
    cu = None
    if nqs is not None:
        cu = ints([sum(nqs[:i]) for i in range(len(nqs) + 1)])
    fa.attention_kv4(q.to(DEV), *(c.to(DEV) for c in cache), ints(table), ints(lens),
                     max(max(lens), 1), cu_seqlens_q=cu, max_seqlen_q=1 if nqs is None else max(nqs),
                     scale=scale, causal=causal, out=o, lse=lse)
    st, word = fa.fa_fwd_status(torch.cuda.current_stream().cuda_stream)
    assert st == fa.FA_OK, word
    nq = [1] * len(lens) if nqs is None else nqs
    check_attention(q, cache, table, lens, nq, bs, d, scale, causal, o, lse, DT[dt])
    assert (o[sum(nq):] == 7.0).all() and (lse[:, sum(nq):] == 7.0).all()


def small(seed, lens=(90, 33), nqs=(1, 1), Hq=8, Hk=2, d=128, bs=16, dt="bf16"):
    g = gen(seed)
    blocks = sum(-(-n // bs) for n in lens) + 2
    cache = random_cache(blocks, Hk, bs, d, g)
    table = paged(lens, bs, blocks, g)
    q = torch.randn(sum(nqs), Hq, d, generator=g).to(DT[dt])
    cu = [sum(nqs[:i]) for i in range(len(nqs) + 1)]
    return q, cache, table, cu


def call(q, cache, table, lens, cu, nqs, max_k=None, **kw):
    return fa.attention_kv4(q.to(DEV), *(c.to(DEV) for c in cache), ints(table), ints(list(lens)),
                            max(lens) if max_k is None else max_k, cu_seqlens_q=ints(cu),
                            max_seqlen_q=max(nqs), **kw)


@pytest.mark.parametrize("nqs", [(1, 1), (5, 40)])
@pytest.mark.parametrize("scale", [0.0, -0.2, 0.6])
def test_attention_scales_and_exponents(nqs, scale):
    lens, exps = (90, 133), (3, -5)
    q, cache, table, cu = small(11, lens, nqs)
    s = scale / 8
    o, lse = call(q, cache, table, lens, cu, nqs, scale=s, k_exp=exps[0], v_exp=exps[1])
    check_attention(q, cache, table, lens, nqs, 16, 128, s, True, o, lse, torch.bfloat16, exps)


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


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_attention_queries_of_extreme_size(dt):
    """Rows whose elements spread over the type's whole range, and a row of
    zeros: the query is rescaled by a power of two on its way to fp16, which
    costs an element below 2^-14 of its row's largest an absolute 2^-25 of
    that largest; the tolerance gets d * 2^-25 * max|q| * max|k| * scale."""
    lens, nqs = (70, 50, 20), (1, 1, 1)
    q, cache, table, cu = small(15, lens, nqs, dt=dt)
    q = q.double()
    big = 2.0 ** 100 if dt == "bf16" else 2.0 ** 12
    q[0] *= big
    q[1] *= 2.0 ** -12
    q[1, :, ::3] *= 2.0 ** -12
    q[2] = 0
    q = q.to(DT[dt])
    scale = 0.05 / big
    for b, s in ((0, scale), (1, 0.05), (2, 0.05)):
        o, lse = call(q[b:b + 1], cache, [table[b]], (lens[b],), [0, 1], (1,), scale=s)
        K, V = ref.values(*cache[:2]), ref.values(*cache[2:])
        ids = torch.tensor([table[b][j // 16] for j in range(lens[b])])
        at = ids, torch.arange(lens[b]) % 16
        want, wl, a, size = ref.attend(q[b:b + 1].double(), K[at[0], :, at[1]], V[at[0], :, at[1]], s,
                                       True)
        extra = 128 * 2.0 ** -25 * float(q[b].double().abs().max()) * 6 * s
        tol_o, tol_l = attention_tolerance(want, wl, a, size, s, 128, DT[dt])
        assert ((o.double().cpu() - want).abs() <= tol_o + 2 * extra * a).all()
        assert ((lse.double().cpu() - wl).abs() <= tol_l + extra).all()


NON_FINITE = [
    # key lengths, query lengths, Hq, Hk, d, width of the table in blocks (0: what they need)
    ((300, 33), (1, 1), 8, 2, 128, 0),           # clusters
    ((300, 33), (3, 1), 4, 1, 64, 65536),        # the line, joined or not
    ((20000, 90, 5000), (1, 2, 1), 8, 2, 128, 0),
    ((70, 40), (4, 2), 8, 1, 128, 65536),        # the kernel for many queries at 32 rows
    ((513, 300), (64, 200), 6, 3, 64, 0),        # whole tiles
    ((9000, 3000), (70, 90), 4, 1, 128, 0),      # tiles that several CTAs share
]


@pytest.mark.parametrize("case", NON_FINITE, ids=[str(i) for i in range(len(NON_FINITE))])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_shows_nan_and_infinity(case, causal):
    """A query row with a NaN, or with an infinity that some key meets, gets NaN
    for O and LSE whichever path takes it; a NaN in a key's scale, the rows that
    see this key.  The other rows are as without it."""
    lens, nqs, Hq, Hk, d, width = case
    q, cache, table, cu = small(91, lens, nqs, Hq=Hq, Hk=Hk, d=d)
    wide = ints(table)
    if width:
        wide = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
        wide[:, :len(table[0])] = ints(table)
    bad = torch.zeros(q.shape[:2], dtype=torch.bool)
    spoiled = q.clone()
    for row, head, value in ((0, 0, math.nan), (cu[1], Hq - 1, math.inf), (cu[-1] - 1, 1, -math.inf)):
        spoiled[row, head, 5] = value
        bad[row, head] = True
    # the last key of the last sequence: its last query alone sees it when causal
    keys = [c.clone() for c in cache]
    n = lens[-1]
    keys[1][table[-1][(n - 1) // 16], Hk - 1, (n - 1) % 16, 2] = 0x7F
    blind = torch.zeros_like(bad)
    blind[(-1 if causal else cu[-2]):, -(Hq // Hk):] = True
    for x, c, off in ((spoiled, cache, bad), (q, keys, blind)):
        o, lse = fa.attention_kv4(x.to(DEV), *(t.to(DEV) for t in c), wide, ints(list(lens)),
                                  2 ** 31 - 1, cu_seqlens_q=ints(cu), max_seqlen_q=max(nqs),
                                  causal=causal)
        o, lse = o.cpu(), lse.cpu()
        assert torch.isnan(o[off]).all() and torch.isnan(lse.t()[off]).all()
        assert not torch.isnan(o[~off]).any() and not torch.isnan(lse.t()[~off]).any()
        # the rows without one against the reference, the others as if they were whole
        clean, cl = call(q, cache, table, lens, cu, nqs, causal=causal)
        o[off], lse.t()[off] = clean.cpu()[off], cl.cpu().t()[off]
        check_attention(q, cache, table, lens, nqs, 16, d, d ** -0.5, causal, o, lse, torch.bfloat16)


@pytest.mark.parametrize("nqs", [(1, 2), (40, 60)])
def test_attention_of_infinities_that_take_keys_away(nqs):
    """Scores of -inf have no weight: keys whose element meets the query's infinity
    with the other sign are as if masked, and where that is all of them the row is
    one without keys."""
    lens = (200, 90)
    q, cache, table, cu = small(93, lens, nqs, Hq=4, Hk=2, d=64)
    kc = cache[0]
    kc[..., 0] = (kc[..., 0] & 0xF0) | 0xA       # element 0 of every key is -1 times its scale
    q[0, 1, 0] = math.inf
    q[-1, 2, 0] = math.inf
    kc[table[1][2], :, 7, 0] = 0x0              # an infinity times zero: NaN (token 39)
    o, lse = call(q, cache, table, lens, cu, nqs)
    assert (o[0, 1] == 0).all() and lse[1, 0] == -math.inf
    assert torch.isnan(o[-1, 2]).all() and torch.isnan(lse[2, -1])
    q[0, 1, 0] = q[-1, 2, 0] = 0.0
    other = call(q, cache, table, lens, cu, nqs)
    o[0, 1], lse[1, 0] = other[0][0, 1], other[1][1, 0]
    o[-1, 2], lse[2, -1] = other[0][-1, 2], other[1][2, -1]
    check_attention(q, cache, table, lens, nqs, 16, 64, 64 ** -0.5, True, o, lse, torch.bfloat16)


def test_attention_long_context():
    """A long sequence (split over many CTAs) against the float64 sums."""
    n, Hq, Hk, d, bs = 70001, 4, 1, 128, 64
    g = gen(21)
    blocks = -(-n // bs) + 1
    cache = random_cache(blocks, Hk, bs, d, g)
    table = paged([n], bs, blocks, g)
    poison_tails(cache, table, [n], bs)
    q = torch.randn(1, Hq, d, generator=g).bfloat16()
    o, lse = call(q, cache, table, (n,), [0, 1], (1,))
    check_attention(q, cache, table, [n], [1], bs, d, d ** -0.5, True, o, lse, torch.bfloat16)


def test_attention_cache_beyond_32_bit_offsets():
    """A cache of more than 2^32 bytes of codes: blocks at both ends of it."""
    Hk, d, bs = 8, 128, 128
    blocks = (1 << 32) // (Hk * bs * d // 2) + 40  # codes alone pass 4 GB
    kc = torch.empty(blocks, Hk, bs, d // 2, dtype=torch.uint8, device=DEV)
    ks = torch.empty(blocks, Hk, bs, d // 16, dtype=torch.uint8, device=DEV)
    g = gen(22)
    lens, ids = [300], [blocks - 1, 0, blocks - 17]
    part = random_cache(3, Hk, bs, d, g)
    for i, b in enumerate(ids):
        kc[b], ks[b] = part[0][i].to(DEV), part[1][i].to(DEV)
    q = torch.randn(1, 16, d, generator=g).bfloat16()
    o, lse = fa.attention_kv4(q.to(DEV), kc, ks, kc, ks, ints([ids]), ints(lens), 300)
    check_attention(q, (part[0], part[1]) * 2, [[0, 1, 2]], lens, [1], bs, d, d ** -0.5, True, o, lse,
                    torch.bfloat16)
    slots = torch.tensor([b * bs + 5 for b in ids])
    k, _ = fa.kv4_gather(slots.to(DEV), kc, ks, kc, ks)
    want = torch.stack([ref.values(part[0][i, :, 5], part[1][i, :, 5]) for i in range(3)])
    assert torch.equal(k.double().cpu(), want)


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("graph", [False, True])
def test_a_served_batch_step_by_step(graph):
    """A prompt step and decode steps of a ragged batch: tables from lengths,
    rotary positions, the new rows into the cache, attention over it; against
    the same in 64 bits from the stored cache.  With `graph` the decode step
    is captured once and replayed with the lengths fed back on the GPU."""
    B, Hq, Hk, d, bs, width, steps = 3, 8, 2, 64, 16, 12, 5
    g = gen(31)
    blocks = B * width + 1
    cache = fa.kv4_cache(blocks, Hk, bs, d, device=DEV)
    for c in cache:
        c.fill_(0xFF)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    free = torch.randperm(blocks, generator=g).int().to(DEV)
    freq, axis = ladder(d, 1)
    rt = fa.rotary_table(freq, axis, device=DEV)
    lens, head = torch.zeros(B, dtype=torch.int32, device=DEV), ints([0])
    history = [[] for _ in range(B)]

    def step(new, qkv, cap, max_q):
        slots, pos, cu, seq, counts = fa.kv_plan(lens, new, free, table, bs, cap, free_head=head)
        q, k = fa.rotary(qkv[:, :Hq], qkv[:, Hq:Hq + Hk], pos.view(1, cap), rt)
        fa.kv4_append(k, qkv[:, Hq + Hk:], slots, *cache)
        o, lse = fa.attention_kv4(q, *cache, table, seq, width * bs, cu_seqlens_q=cu,
                                  max_seqlen_q=max_q)
        lens.copy_(seq)
        head.add_(counts[:1])
        return q, k, o, lse, cu

    def check(new, qkv, q, k, o, lse):
        row = 0
        x = qkv.cpu()
        for b, n in enumerate(new):
            for t in range(row, row + n):
                history[b].append((k[t].cpu(), x[t, Hq + Hk:]))
            K = ref.values(*ref.quantise(torch.stack([h[0] for h in history[b]])))
            V = ref.values(*ref.quantise(torch.stack([h[1] for h in history[b]])))
            qb = q[row:row + n].double().cpu()
            p = torch.arange(len(history[b]) - n, len(history[b])).view(1, 1, n)
            turned = ref.rotate(x[row:row + n, :Hq].double().transpose(0, 1)[None], p,
                                torch.tensor(freq, dtype=torch.float64), torch.tensor(axis), d)
            assert (turned[0].transpose(0, 1) - qb).abs().max() <= 2.0 ** -8 * 6 + 2.0 ** -20
            want, wl, a, big = ref.attend(qb, K, V, d ** -0.5, True)
            tol_o, tol_l = attention_tolerance(want, wl, a, big, d ** -0.5, d, torch.bfloat16)
            assert ((o[row:row + n].double().cpu() - want).abs() <= tol_o).all()
            assert ((lse[:, row:row + n].double().cpu() - wl).abs() <= tol_l).all()
            row += n

    new = [37, 5, 64]
    qkv = torch.randn(sum(new) + 4, Hq + 2 * Hk, d, generator=g).bfloat16().to(DEV)
    q, k, o, lse, _ = step(ints(new), qkv, sum(new) + 4, max(new))
    check(new, qkv, q, k, o, lse)
    ones = ints([1] * B)
    qkv = torch.randn(B, Hq + 2 * Hk, d, generator=g).bfloat16().to(DEV)
    if graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        keep = [t.clone() for t in (lens, head, table) + cache]
        with torch.cuda.stream(side):
            step(ones, qkv, B, 1)  # warm-up
            for t, x in zip((lens, head, table) + cache, keep):
                t.copy_(x)
            side.synchronize()
            cg = torch.cuda.CUDAGraph()
            with torch.cuda.graph(cg, stream=side):
                q, k, o, lse, _ = step(ones, qkv, B, 1)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(steps):
        qkv.copy_(torch.randn(qkv.shape, generator=g).bfloat16())
        if graph:
            cg.replay()
        else:
            q, k, o, lse, _ = step(ones, qkv, B, 1)
        check([1] * B, qkv, q, k, o, lse)
    assert lens.tolist() == [n + steps for n in new]
    assert head.item() == sum(-(-(n + steps) // bs) for n in new)


def test_two_streams_at_once():
    """Two calls on two streams, a workspace each: the results of one alone."""
    lens, nqs = (5000, 3000), (1, 1)
    a, b = small(41, lens, nqs), small(42, lens, nqs)
    args = []
    for q, cache, table, cu in (a, b):
        args.append((q.to(DEV), *(c.to(DEV) for c in cache), ints(table), ints(list(lens)), 5000))
    alone = [fa.attention_kv4(*x) for x in args]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for x, st in zip(args, s):
            with torch.cuda.stream(st):
                got.append(fa.attention_kv4(*x))
        torch.cuda.synchronize()
        for (o, l), (wo, wl) in zip(got, alone):
            assert torch.equal(o, wo) and torch.equal(l, wl)


def test_two_graphs_at_once():
    """Two captured calls, whose workspaces the wrapper allocated in the captures,
    replayed on two streams: the results of one alone.  One joins the shares of a
    line of units, the other the tiles of many queries."""
    cases = [((20000, 900), (1, 2)), ((5000, 300), (200, 130))]
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for n, (lens, nqs) in enumerate(cases):
        q, cache, table, cu = small(46 + n, lens, nqs, bs=64)
        args = (q.to(DEV), *(c.to(DEV) for c in cache), ints(table), ints(list(lens)), max(lens))
        kw = dict(cu_seqlens_q=ints(cu), max_seqlen_q=max(nqs))
        want = fa.attention_kv4(*args, **kw)
        torch.cuda.synchronize()
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg, stream=streams[n]):
            got = fa.attention_kv4(*args, **kw)
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


def test_calls_from_several_threads():
    """The wrappers let go of the interpreter's lock: threads with a stream each get
    what one thread gets."""
    import threading
    work = []
    for n, (lens, nqs) in enumerate((((3000, 70), (1, 1)), ((900, 5), (60, 4)), ((64, 64), (1, 1)))):
        q, cache, table, cu = small(48 + n, lens, nqs)
        args = (q.to(DEV), *(c.to(DEV) for c in cache), ints(table), ints(list(lens)), max(lens))
        kw = dict(cu_seqlens_q=ints(cu), max_seqlen_q=max(nqs))
        work.append((args, kw, fa.attention_kv4(*args, **kw)))
    torch.cuda.synchronize()
    wrong = []

    def run(args, kw, want):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(50):
                got = fa.attention_kv4(*args, **kw)
                st.synchronize()
                if not (torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])):
                    wrong.append(args)

    threads = [threading.Thread(target=run, args=w) for w in work * 2]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    assert fa.fa_fwd_status(torch.cuda.current_stream().cuda_stream) == (fa.FA_OK, 0)


def test_a_stream_of_its_own():
    """Calls on a stream that is not the current one: what the wrappers
    allocate belongs to that stream."""
    side = torch.cuda.Stream()
    q, cache, table, cu = small(43, (3000, 70), (5, 60))
    args = (q.to(DEV), *(c.to(DEV) for c in cache), ints(table), ints([3000, 70]), 3000)
    kw = dict(cu_seqlens_q=ints(cu), max_seqlen_q=60)
    want = fa.attention_kv4(*args, **kw)
    pos, rt = ints([list(range(65))]), fa.rotary_table([1.0 / 2 ** i for i in range(64)], device=DEV)
    turned = fa.rotary(args[0], None, pos, rt)[0]
    slots = torch.arange(16, device=DEV)
    rows = fa.kv4_gather(slots, *args[1:5])
    torch.cuda.synchronize()
    for _ in range(20):
        o, lse = fa.attention_kv4(*args, **kw, stream=side.cuda_stream)
        x = fa.rotary(args[0], None, pos, rt, stream=side.cuda_stream)[0]
        k, v = fa.kv4_gather(slots, *args[1:5], stream=side.cuda_stream)
        torch.full((1 << 20,), 9.0, device=DEV)  # would take freed memory of the current stream
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1]) and torch.equal(x, turned)
        assert torch.equal(k, rows[0]) and torch.equal(v, rows[1])


def test_many_queries_report_a_wait_that_runs_out():
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


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq", [3, 8, 12, 16])  # rows a sequence: tiles of 8 and 16
@pytest.mark.parametrize("B", [1, 17, 40, 100, 200])
def test_attention_of_small_batches(B, Hq, d):
    """Up to one sequence a CTA, by a tight and by a loose bound on the keys: the
    bound decides how many CTAs a sequence gets and who joins their parts."""
    lens = [(137 * b + 1000) % 1025 if b % 7 != 3 else b % 2 for b in range(B)]
    nqs = [1] * B
    q, cache, table, _ = small(61 + B, lens, nqs, Hq=Hq, Hk=1, d=d)
    for max_k in (1024, 1 << 20):
        o, lse = fa.attention_kv4(q.to(DEV), *(c.to(DEV) for c in cache), ints(table), ints(lens),
                                  max_k)
        check_attention(q, cache, table, lens, nqs, 16, d, d ** -0.5, True, o, lse, torch.bfloat16,
                        label=str(max_k))
        again = fa.attention_kv4(q.to(DEV), *(c.to(DEV) for c in cache), ints(table), ints(lens),
                                 max_k)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("nq", [1, 3, 61])
@pytest.mark.parametrize("Hq", [1, 3, 5, 7, 11, 13])
@pytest.mark.parametrize("B", [1, 70, 140, 290])
def test_attention_of_odd_rows(B, Hq, nq):
    """Rows that end inside a warp at the joins of clusters (64 elements: 16 threads
    a row) and inside a warp's rows of a tile."""
    lens = [(91 * b + 300) % 350 for b in range(B if nq < 61 else 3)]
    nqs = [nq] * len(lens)
    q, cache, table, cu = small(101 + B, lens, nqs, Hq=Hq, Hk=1, d=64)
    o, lse = call(q, cache, table, lens, cu, nqs)
    assert fa.fa_fwd_status(torch.cuda.current_stream().cuda_stream) == (fa.FA_OK, 0)
    check_attention(q, cache, table, lens, nqs, 16, 64, 0.125, True, o, lse, torch.bfloat16)


@pytest.mark.parametrize("lens,max_k", [((8192, 5000), 8192), ((2000,) * 3, 2048),
                                        ((4096, 0, 1, 4000) * 2, 4096), ((127, 129, 128), 130)])
def test_attention_of_few_long_sequences(lens, max_k):
    """The longest caches that a cluster takes, drafted tokens among their queries,
    and one sequence of the batch with more queries than a tile holds."""
    nqs = [1 + b % 2 for b in range(len(lens))]
    for extra in (0, 9):
        nqs[-1] += extra
        q, cache, table, cu = small(67, lens, nqs, Hq=8, Hk=2, bs=64)
        o, lse = call(q, cache, table, lens, cu, nqs, max_k=max_k)
        check_attention(q, cache, table, lens, nqs, 64, 128, 128 ** -0.5, True, o, lse,
                        torch.bfloat16, max_k=max_k, label=str(extra))


@pytest.mark.parametrize("nqs", [(4, 2), (1, 3), (40, 4)])
def test_attention_of_32_rows_and_a_bound_of_many_keys(nqs):
    """Rows that fill a tile go to the kernel for many queries when max_seqlen_k
    leaves room for a million keys, whatever the lengths are; the workspace is
    the same."""
    lens = (700, 33)
    q, cache, table, cu = small(57, lens, nqs, Hq=16, Hk=2)
    need = fa.fa_fwd_kv4_workspace(2, 16, 2, max(nqs), 128)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    for max_k in (700, 1 << 20):
        o, lse = call(q, cache, table, lens, cu, nqs, max_k=max_k, workspace=ws)
        check_attention(q, cache, table, lens, nqs, 16, 128, 128 ** -0.5, True, o, lse,
                        torch.bfloat16, label=str(max_k))


@pytest.mark.parametrize("B,Hq,Hk,nq,d", [(1, 32, 8, 1, 128), (3, 8, 8, 3, 64), (40, 8, 8, 1, 64),
                                          (56, 8, 8, 1, 128), (64, 16, 8, 1, 64), (5, 32, 2, 2, 128),
                                          (9, 4, 2, 50, 64), (19, 16, 1, 2, 64)])
def test_attention_without_a_bound_on_the_keys(B, Hq, Hk, nq, d):
    """max_seqlen_k of 2^31 - 1 is the table's width: the same launches, the same
    results bit for bit, nothing behind the workspace is written."""
    lens = [(211 * b + 700) % 900 for b in range(B)]
    nqs = [nq] * B
    q, cache, table, cu = small(71 + B, lens, nqs, Hq=Hq, Hk=Hk, d=d)
    need = fa.fa_fwd_kv4_workspace(B, Hq, Hk, nq, d)
    got = []
    for max_k in (len(table[0]) * 16, 2 ** 31 - 128, 2 ** 31 - 1):
        ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
        got.append(call(q, cache, table, lens, cu, nqs, max_k=max_k, workspace=ws[:need]))
        assert (ws[need:] == 0x5A).all()
    assert fa.fa_fwd_status(torch.cuda.current_stream().cuda_stream) == (fa.FA_OK, 0)
    for o, lse in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(lse, got[0][1])
    check_attention(q, cache, table, lens, nqs, 16, d, d ** -0.5, True, *got[0], torch.bfloat16)


@pytest.mark.parametrize("B,Hq,Hk,nqs,d", [(1, 3, 1, 1, 64), (1, 16, 1, 1, 128), (17, 8, 1, 1, 128),
                                           (40, 12, 1, 1, 64), (100, 16, 1, 1, 128), (2, 16, 2, 4, 128),
                                           (2, 8, 2, 2, 64), (5, 64, 2, 1, 128), (3, 16, 2, 40, 128)])
def test_attention_of_short_sequences_in_a_wide_table(B, Hq, Hk, nqs, d):
    """Where table and bound leave room for a million keys the line of units is
    dealt out and joined, and 32 rows of 128 elements go to the kernel for many
    queries, however short the sequences are."""
    lens = [(137 * b + 1000) % 1025 if b % 7 != 3 else b % 2 for b in range(B)]
    nqs = [nqs] * B
    q, cache, table, cu = small(81 + B, lens, nqs, Hq=Hq, Hk=Hk, d=d)
    wide = torch.full((B, 65536), 2 ** 31 - 1, dtype=torch.int32, device=DEV)
    wide[:, :len(table[0])] = ints(table)
    rows, cl = fa.fa_fwd_kv4_schedule(B, Hq, Hk, nqs[0], 2 ** 31 - 1, 65536, 16, d, 152)[2:4]
    assert cl == 0 and rows == (0 if d == 128 and nqs[0] * Hq // Hk == 32 else rows)
    o, lse = fa.attention_kv4(q.to(DEV), *(c.to(DEV) for c in cache), wide, ints(lens), 2 ** 31 - 1,
                              cu_seqlens_q=ints(cu), max_seqlen_q=nqs[0])
    assert fa.fa_fwd_status(torch.cuda.current_stream().cuda_stream) == (fa.FA_OK, 0)
    check_attention(q, cache, table, lens, nqs, 16, d, d ** -0.5, True, o, lse, torch.bfloat16)


@pytest.mark.parametrize("nq", [1, 40])
def test_attention_of_a_sequence_as_long_as_its_type_allows(nq):
    """A length of 2^31 - 1 in a table of 2^31 - 16 tokens is cut to 2^31 - 4096:
    of the few blocks that are there, those at the start, in the middle and at
    that end count, the ones behind it do not."""
    bs, d, Hq = 16, 64, 2
    width = 2 ** 27 - 1
    end = 2 ** 31 - 4096
    g = gen(77)
    cache = random_cache(6, 1, bs, d, g)
    table = torch.full((1, width), -1, dtype=torch.int32, device=DEV)
    at = [0, 1, 2 ** 26 + 3, end // bs - 1, end // bs, width - 1]
    table[0, at] = torch.arange(6, dtype=torch.int32, device=DEV)
    q = torch.randn(nq, Hq, d, generator=g).bfloat16()
    o, lse = fa.attention_kv4(q.to(DEV), *(c.to(DEV) for c in cache), table, ints([2 ** 31 - 1]),
                              2 ** 31 - 1, cu_seqlens_q=ints([0, nq]), max_seqlen_q=nq)
    assert fa.fa_fwd_status(torch.cuda.current_stream().cuda_stream) == (fa.FA_OK, 0)
    # the last block's keys are the last 16 of the sequence; the rest everyone sees
    small_table, n = [[0, 1, 2] + [-1] * (nq // bs + 1) + [3]], (5 + nq // bs) * bs
    check_attention(q, cache, small_table, [n], [nq], bs, d, d ** -0.5, True, o, lse, torch.bfloat16)


def test_repeated_calls_are_the_same_bit_for_bit():
    """Parts are joined in a fixed order: no result depends on which CTA was
    first, at one query a sequence and at many."""
    for nqs in ((1, 1, 1), (3, 200, 1)):
        lens = (20000, 900, 5000)
        q, cache, table, cu = small(45, lens, nqs, bs=64)
        args = (q.to(DEV), *(c.to(DEV) for c in cache), ints(table), ints(list(lens)), max(lens))
        first = fa.attention_kv4(*args, cu_seqlens_q=ints(cu), max_seqlen_q=max(nqs))
        for _ in range(5):
            o, lse = fa.attention_kv4(*args, cu_seqlens_q=ints(cu), max_seqlen_q=max(nqs))
            assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


def test_wrapper_refusals_on_the_gpu():
    q, cache, table, cu = small(51)
    dev = [c.to(DEV) for c in cache]
    with pytest.raises(ValueError):
        fa.attention_kv4(q.to(DEV), *dev, ints(table).long(), ints([90, 33]), 90)
    with pytest.raises(ValueError):
        fa.attention_kv4(q.to(DEV)[..., :64], *dev, ints(table), ints([90, 33]), 90)
    with pytest.raises(ValueError):
        fa.attention_kv4(q, *dev, ints(table), ints([90, 33]), 90)
    with pytest.raises(ValueError):
        fa.kv4_append(q.to(DEV), q.to(DEV), ints([1, 2], torch.int64), *dev)
    with pytest.raises(ValueError):
        fa.kv4_gather(ints([1, 2]), *dev)
    with pytest.raises(ValueError):
        fa.rotary(q.to(DEV), None, torch.zeros(1, 3, dtype=torch.int32, device=DEV),
                  fa.rotary_table([1.0], device=DEV))
    with pytest.raises(fa.FaError):
        fa.attention_kv4(q.float().to(DEV), *dev, ints(table), ints([90, 33]), 90)


def test_wrapper_arguments_one_by_one():
    """Every tensor of every wrapper in a wrong type, shape, layout or place is
    refused, and the same call with the right one works before and after."""
    q, cache, table, cu = small(53)
    dev = [c.to(DEV) for c in cache]
    qd = q.to(DEV)
    k = torch.randn(2, 2, 128, device=DEV).bfloat16()

    def refused(fn, args, at, bad, **kw):
        fn(*args, **kw)
        for b in bad:
            with pytest.raises((ValueError, fa.FaError)):
                fn(*args[:at], b, *args[at + 1:], **kw)
        fn(*args, **kw)

    def spoiled(t):
        wide = torch.stack([t, t], -1)[..., 0]  # strided
        return [t.cpu(), t.double(), wide if t.numel() > 1 else t.cpu(), t[:-1], 7, None]

    attn = (qd, *dev, ints(table), ints([90, 33]), 90)
    for at in (*range(1, 5), 5, 6):
        refused(fa.attention_kv4, attn, at, spoiled(attn[at]))
    for bad in (q, qd.transpose(0, 1), qd[..., ::2], 3):
        refused(fa.attention_kv4, attn, 0, [bad])
    lse = torch.empty(8, 2, device=DEV)
    for kw in (dict(out=q), dict(out=qd.float()), dict(out=qd[:1]), dict(lse=lse.half()),
               dict(lse=lse[:7]), dict(lse=lse.t()), dict(cu_seqlens_q=ints([0, 1])),
               dict(cu_seqlens_q=ints([0, 1, 2]).long()), dict(workspace=lse.t()),
               dict(workspace=lse.cpu())):
        with pytest.raises(ValueError):
            fa.attention_kv4(*attn, **kw)
    with pytest.raises(fa.FaError):
        fa.attention_kv4(*attn, workspace=lse)  # too small
    with pytest.raises(TypeError):
        fa.attention_kv4(*attn[:-1], 90.5)

    put = (k, k.clone(), ints([1, 2], torch.int64), *dev)
    for at in range(1, 7):
        refused(fa.kv4_append, put, at, spoiled(put[at]))
    get = (ints([1, 2], torch.int64), *dev)
    for at in range(5):
        bad = spoiled(get[at])
        refused(fa.kv4_gather, get, at, [b for b in bad if at or b is not bad[3]])
    for out in ((k,), (k, k.float()), (k, k[:1]), (k, k.cpu()), (k, k.transpose(0, 1))):
        with pytest.raises(ValueError):
            fa.kv4_gather(*get, out=out)
    with pytest.raises(ValueError):
        fa.kv4_gather(*get, dtype="bf16")
    with pytest.raises(ValueError):
        fa.kv4_gather(*get, dtype=torch.float64)

    turn = (qd, qd[:, :2], ints([[3, 4]]), fa.rotary_table([1.0, 0.1], device=DEV))
    for at in (2, 3):
        bad = spoiled(turn[at])
        refused(fa.rotary, turn, at, [b for b in bad if at == 2 or b is not bad[3]])
    for bad in (q, qd.float(), qd[..., :64], qd[:1], 3):
        refused(fa.rotary, turn, 1, [bad])
    for kw in (dict(q_out=q), dict(q_out=qd[:, :4]), dict(k_out=qd), dict(k_out=qd[:, :2].half())):
        with pytest.raises(ValueError):
            fa.rotary(*turn, **kw)

    plan = (ints([0, 5]), ints([3, 1]), ints([1, 2, 3]), torch.full((2, 4), -1, device=DEV).int(),
            16, 8)
    for at in (0, 1, 3):
        refused(fa.kv_plan, plan, at, spoiled(plan[at]))
    refused(fa.kv_plan, plan, 2, [plan[2].cpu(), plan[2].long(), 7, None])
    outs = fa.kv_plan(*plan)
    for i in range(5):
        bad = [*outs]
        bad[i] = bad[i][:-1]
        with pytest.raises(ValueError):
            fa.kv_plan(*plan, out=bad)
    with pytest.raises(ValueError):
        fa.kv_plan(*plan, out=outs[:4])


def test_wrappers_hand_back_what_they_are_given_and_keep_nothing():
    import sys
    q, cache, table, cu = small(59)
    dev, qd = [c.to(DEV) for c in cache], q.to(DEV)
    t, n, s = ints(table), ints([90, 33]), ints([1, 2], torch.int64)
    pos, rot = ints([[3, 4]]), fa.rotary_table([1.0, 0.1], device=DEV)
    plan = (ints([0, 5]), ints([3, 1]), ints([1, 2, 3]), torch.full((2, 4), -1, device=DEV).int(),
            16, 8)
    o, lse = torch.empty_like(qd), torch.empty(8, 2, device=DEV)
    kv = (torch.empty(2, 2, 128, device=DEV), torch.empty(2, 2, 128, device=DEV))
    outs = fa.kv_plan(*plan)
    fused = torch.randn(2, 12, 128, device=DEV).bfloat16()  # rows of q, k, v side by side

    def calls(given):
        if given:
            a = fa.attention_kv4(qd, *dev, t, n, 90, out=o, lse=lse)
            assert a[0] is o and a[1] is lse
            assert fa.kv4_gather(s, *dev, out=kv) is kv
            assert fa.kv_plan(*plan, out=outs) is outs
            r = fa.rotary(qd, None, pos, rot, q_out=o)
            assert r[0] is o and r[1] is None
            return fa.kv_plan(*plan, out=list(outs)), fa.kv4_gather(s, *dev, out=list(kv))
        r = fa.rotary(fused[:, :8], fused[:, 8:10], pos, rot)
        assert r[0].is_contiguous() and r[1].is_contiguous()
        swapped = fused.view(2, 12, 1, 128).transpose(0, 1).transpose(1, 2)  # [12, 1, 2, d]
        turned = fa.rotary(swapped, None, ints([[[3, 4]] * 12]), rot)[0]
        assert turned.shape == swapped.shape and turned.stride() == torch.empty_like(swapped).stride()
        return fa.attention_kv4(qd, *dev, t, n, 90), fa.kv4_gather(s, *dev), fa.kv_plan(*plan)

    held = (o, lse, outs, kv, qd, dev[0], t, pos, rot, plan)
    for given in (True, False):
        calls(given)
        before = [sys.getrefcount(x) for x in held], torch.cuda.memory_allocated()
        for _ in range(20):
            calls(given)
        assert ([sys.getrefcount(x) for x in held], torch.cuda.memory_allocated()) == before
