"""Host-side checks of the serving operators (no GPU work: every call here is
refused, or is host-only) and the reference helpers of their GPU tests."""
import ctypes
import math
import os
from fractions import Fraction

import pytest
import torch

import serve_util as ref
from exact_attention_57_gb300 import fa

# 1 / (2 pi) to 75 digits
INV_2PI = Fraction("0.15915494309189533576888376337251436203445964574045644874766734405889679763")


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(fa.LIB_PATH):
        from exact_attention_57_gb300 import build
        build.build_library()
    return fa.load()


def A(i):
    """Fake device addresses, 16 TB apart; never dereferenced."""
    return (i + 1) << 44


# ------------------------------------------------------------------ plan
PLAN = dict(cached=A(0), new=A(1), free=A(2), head=None, table=A(3), slots=A(4), pos=A(5),
            cu=A(6), lens=A(7), counts=A(8), B=3, width=4, bs=16, num_free=9, cap=20)


def plan(**kw):
    a = dict(PLAN, **kw)
    return fa.fa_kv_plan(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(cached=None), dict(new=None), dict(free=None), dict(table=None), dict(slots=None),
    dict(pos=None), dict(cu=None), dict(lens=None), dict(counts=None),
    dict(B=0), dict(B=65536), dict(width=0), dict(bs=8), dict(bs=48), dict(bs=256),
    dict(num_free=-1), dict(cap=0), dict(width=1 << 28),
    dict(slots=A(4) + 4), dict(table=A(3) + 2), dict(head=A(9) + 1),
    dict(slots=A(0)), dict(lens=A(1) + 4), dict(pos=A(4) + 8), dict(counts=A(2) + 32),
    dict(head=A(3) + 8),
], ids=str)
def test_plan_refusals(kw):
    assert plan(**kw) == fa.FA_ERR_INVALID_ARG


# ------------------------------------------------------------------ rope
def L6(*v):
    return (ctypes.c_longlong * 6)(*v)


ROPE = dict(q=A(0), qo=A(1), qs=None, Hq=4, k=A(2), ko=A(3), ks=None, Hk=2, pos=A(4), axes=2,
            table=A(5), B=2, N=7, d=64, rot=64, inter=0, inv=0, dtype=fa.FA_DTYPE_BF16)


def rope(**kw):
    return fa.fa_rope(*dict(ROPE, **kw).values(), None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(qo=None), dict(k=None), dict(ko=None), dict(pos=None), dict(table=None),
    dict(Hq=0), dict(Hk=-1), dict(B=0), dict(N=0), dict(d=0), dict(axes=0), dict(axes=5),
    dict(rot=0), dict(rot=63), dict(rot=66), dict(inter=2), dict(inv=-1), dict(dtype=4),
    dict(q=A(0) + 1), dict(pos=A(4) + 2), dict(table=A(5) + 4),
    dict(qo=A(0) + 64),                                     # shifted onto its own input
    dict(qo=A(0), qs=L6(1792, 448, 64, 1792, 64, 256)),     # in place at other strides
    dict(qs=L6(1792, 448, 64, 1792, 448, 63)),              # rows of the output meet
    dict(qs=L6(1792, 448, 64, 0, 448, 64)),
    dict(qs=L6(1792, 448, 64, 1792, 64, 64)),
    dict(qs=L6(1792, -448, 64, 1792, 448, 64)),
    dict(ko=A(4)), dict(ko=A(5)),
], ids=str)
def test_rope_refusals(kw):
    assert rope(**kw) == fa.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(qo=A(2)), dict(ko=A(0)), dict(qo=A(3)), dict(ko=A(1) + 4096), dict(qo=A(2), ko=A(0)),
    dict(q=A(2), qo=A(2)), dict(k=A(0), ko=A(0), qo=A(0), Hk=4),          # one tensor twice, in place
    dict(k=A(0) + 128, ko=A(0) + 128, qo=A(0)),                           # in place, shifted
    dict(qo=A(2) + 512, ks=L6(896, 448, 64, 896, 448, 64)),
    # slices of one projection's rows of 512 elements: columns that meet by one element
    dict(q=A(0), qo=A(0), qs=L6(3584, 64, 512, 3584, 64, 512),
         k=A(0) + 510, ko=A(0) + 510, ks=L6(3584, 64, 512, 3584, 64, 512)),
    dict(qs=L6(1 << 62, 448, 64, 1792, 448, 64)), dict(ks=L6(896, 448, 64, 1 << 62, 448, 64)),
], ids=str)
def test_rope_refuses_outputs_on_the_other_tensor(kw):
    assert rope(**kw) == fa.FA_ERR_INVALID_ARG


host_only = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only: fake device addresses")


@host_only
@pytest.mark.parametrize("kw", [
    dict(qo=A(0)), dict(qo=A(0), ko=A(2)), dict(),
    # rows of 512 elements: q's four heads, then k's two, in place, or moved behind them
    dict(qo=A(0), qs=L6(3584, 64, 512, 3584, 64, 512), k=A(0) + 512, ko=A(0) + 512,
         ks=L6(3584, 64, 512, 3584, 64, 512)),
    dict(q=A(0), qo=A(0), qs=L6(3584, 64, 512, 3584, 64, 512), k=A(0) + 512, ko=A(0) + 768,
         ks=L6(3584, 64, 512, 3584, 64, 512)),
    # heads in one buffer, [B, 6, N, d]
    dict(qo=A(0), qs=L6(2688, 448, 64, 2688, 448, 64), k=A(0) + 3584, ko=A(0) + 3584,
         ks=L6(2688, 448, 64, 2688, 448, 64)),
    # the halves of rows of 128 elements
    dict(qo=A(0), Hk=4, qs=L6(3584, 896, 128, 3584, 896, 128), k=A(0) + 128, ko=A(0) + 128,
         ks=L6(3584, 896, 128, 3584, 896, 128)),
    dict(B=1, N=1, qs=L6(1 << 62, 64, 1 << 62, 1 << 62, 64, 1 << 62)),
], ids=str)
def test_rope_takes_rows_that_lie_apart(kw):
    """These pass all checks and end at the device's, as there is none."""
    assert rope(**kw) in (fa.FA_ERR_CUDA, fa.FA_ERR_UNSUPPORTED)


@host_only
def test_rope_overlap_check_against_the_elements_themselves():
    """Random layouts in one small arena: a call whose outputs share an element
    with the other tensor, with each other or, unless in place, with their own
    input is refused; one at a common pitch that shares none is not."""
    import itertools
    import random
    r = random.Random(7)
    taken = refused = 0
    for _ in range(4000):
        B, N, H, d = r.choice([1, 2]), r.choice([1, 2, 3]), r.choice([1, 2, 3]), r.choice([2, 4])
        pitch = d * r.choice([2 * H, 2 * H + 1, 3 * H])
        fused = (N * pitch, d, pitch)

        def layout():
            kind = r.choice(["fused", "fused", "fused", "rows", "heads", "any"])
            if kind == "any":
                return tuple(r.randrange(0, 40) for _ in range(3))
            return {"fused": fused, "rows": (H * N * d, N * d, d), "heads": (N * H * d, d, H * d)}[kind]

        def where():
            return r.randrange(0, 3 * pitch) if r.random() < 0.5 else r.choice([0, d, H * d, 2 * H * d])

        def elements(at, st):
            return [at + b * st[0] + h * st[1] + n * st[2] + x for b, h, n, x in
                    itertools.product(range(B), range(H), range(N), range(d))]

        t = {}
        for name in ("q", "k"):
            t[name] = (where(), layout())
            t[name + "o"] = t[name] if r.random() < 0.4 else (where(), layout())
        e = {n: elements(*v) for n, v in t.items()}
        bad = any(len(set(e[n])) < len(e[n]) for n in ("qo", "ko"))
        clash = [("qo", "ko"), ("qo", "k"), ("ko", "q")]
        for n in ("q", "k"):
            if t[n][0] == t[n + "o"][0]:  # in place: the strides that count are the same
                bad |= any(c > 1 and a != b for c, a, b in zip((B, H, N), t[n][1], t[n + "o"][1]))
            else:
                clash.append((n, n + "o"))
        bad |= any(set(e[a]) & set(e[b]) for a, b in clash)
        st = rope(q=A(0) + 2 * t["q"][0], qo=A(0) + 2 * t["qo"][0], qs=L6(*t["q"][1], *t["qo"][1]),
                  Hq=H, k=A(0) + 2 * t["k"][0], ko=A(0) + 2 * t["ko"][0],
                  ks=L6(*t["k"][1], *t["ko"][1]), Hk=H, B=B, N=N, d=d, rot=d)
        if bad:
            assert st == fa.FA_ERR_INVALID_ARG, (t, B, N, H, d)
            refused += 1
        elif all(v[1] == fused for v in t.values()):
            assert st != fa.FA_ERR_INVALID_ARG or any(
                (v[0] % pitch) + H * d > pitch for v in t.values()), (t, B, N, H, d)
            taken += st != fa.FA_ERR_INVALID_ARG
    assert taken > 20 and refused > 500


def test_rope_head_dim_above_256_is_unsupported():
    assert rope(d=264) == fa.FA_ERR_UNSUPPORTED


@pytest.mark.parametrize("f", [1.0, 0.31, 1e-4, 2 * math.pi, 7.25, 12345.678, 1e6, -0.5, -1e-9,
                               0.0, 5e-324])
@pytest.mark.parametrize("axis", [0, 3])
def test_rope_table_is_the_turn_fraction(f, axis):
    """table = f / (2 pi) mod 1, scaled by 2^64, axis in the low bits.  The
    two doubles that stand for 1 / (2 pi) are off by 2^-108 of it (f <= 1e6 <
    2^20: 2^-27 of a unit at 2^64), the two truncations and the rounding by
    less than 2.5 units, the cleared bits by 3; fma's own rounding of the
    remainder is below 2^-53 * 2^-53 * 2^18."""
    t = (ctypes.c_ulonglong * 1)()
    assert fa.fa_rope_table((ctypes.c_double * 1)(f), (ctypes.c_int * 1)(axis), 1, t) == fa.FA_OK
    assert t[0] & 3 == axis
    want = Fraction(f) * INV_2PI * 2 ** 64
    off = (Fraction(t[0] & ~3) - want) % 2 ** 64
    assert min(off, 2 ** 64 - off) < 6


@pytest.mark.parametrize("f,axis", [(float("nan"), 0), (float("inf"), 0), (1.1e6, 0), (1.0, 4),
                                    (1.0, -1)])
def test_rope_table_refusals(f, axis):
    t = (ctypes.c_ulonglong * 1)(7)
    r = fa.fa_rope_table((ctypes.c_double * 1)(f), (ctypes.c_int * 1)(axis), 1, t)
    assert r == fa.FA_ERR_INVALID_ARG and t[0] == 7
    assert fa.fa_rope_table(None, None, 1, t) == fa.FA_ERR_INVALID_ARG
    assert fa.fa_rope_table((ctypes.c_double * 1)(1.0), None, 0, t) == fa.FA_ERR_INVALID_ARG


# ------------------------------------------------------------------ cache
STORE = dict(kc=A(10), ks=A(11), vc=A(12), vs=A(13))
TAIL = dict(blocks=5, Hk=2, bs=16, d=64, ke=0, ve=0)


def append(**kw):
    a = dict(dict(k=A(0), v=A(1), kst=128, vst=128, slots=A(2), T=3), **STORE, **TAIL,
             dtype=fa.FA_DTYPE_BF16)
    a.update(kw)
    return fa.fa_kv4_append(*a.values(), None)


def gather(**kw):
    a = dict(dict(slots=A(2), R=3), **STORE, ko=A(3), vo=A(4), **TAIL, dtype=fa.FA_DTYPE_BF16)
    a.update(kw)
    return fa.fa_kv4_gather(*a.values(), None)


BAD_STORE = [dict(kc=None), dict(ks=None), dict(vc=None), dict(vs=None), dict(kc=A(10) + 8),
             dict(vs=A(13) + 1), dict(blocks=0), dict(Hk=0), dict(bs=24), dict(bs=0), dict(ke=65),
             dict(ve=-65), dict(dtype=9), dict(d=0)]


@pytest.mark.parametrize("kw", BAD_STORE + [
    dict(k=None), dict(v=None), dict(slots=None), dict(T=0), dict(kst=127), dict(kst=132),
    dict(vst=120), dict(k=A(0) + 8), dict(slots=A(2) + 4), dict(vc=A(10) + 1024),
    dict(kc=A(0)), dict(vs=A(2) + 16),
], ids=str)
def test_append_refusals(kw):
    assert append(**kw) == fa.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", BAD_STORE + [
    dict(slots=None), dict(ko=None), dict(vo=None), dict(R=0), dict(ko=A(3) + 8), dict(vo=A(3)),
    dict(ko=A(10)), dict(vo=A(2) + 16),
], ids=str)
def test_gather_refusals(kw):
    assert gather(**kw) == fa.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("d", [8, 72, 272])
def test_cache_head_dims_outside_the_set_are_unsupported(d):
    assert append(d=d, kst=2 * d, vst=2 * d) == fa.FA_ERR_UNSUPPORTED
    assert gather(d=d) == fa.FA_ERR_UNSUPPORTED


# ------------------------------------------------------------------ attention
ATTN = dict(q=A(0), o=A(1), lse=A(2), **STORE, table=A(5), lens=A(6), cu=A(7), B=3, Hq=4, Hk=2,
            total=9, max_q=5, max_k=64, blocks=5, bs=16, width=4, d=64, scale=0.125, causal=1,
            ke=0, ve=0, dtype=fa.FA_DTYPE_BF16, ws=A(14), wsb=1 << 40)


def attn(**kw):
    return fa.fa_fwd_kv4(*dict(ATTN, **kw).values(), None)


@pytest.mark.parametrize("kw", BAD_STORE + [
    dict(q=None), dict(o=None), dict(lse=None), dict(table=None), dict(lens=None),
    dict(cu=None), dict(cu=None, max_q=1), dict(B=0), dict(B=65536), dict(Hq=0), dict(Hq=3),
    dict(total=0), dict(max_q=0), dict(max_q=10), dict(max_k=-1), dict(width=0),
    dict(width=1 << 28), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(scale=3e38, ke=64), dict(causal=2), dict(q=A(0) + 8), dict(o=A(1) + 2),
    dict(lse=A(2) + 2), dict(table=A(5) + 1), dict(cu=A(7) + 2), dict(o=A(0)), dict(lse=A(1) + 16),
    dict(o=A(10) + 16), dict(lse=A(6) + 4),
], ids=str)
def test_attention_refusals(kw):
    assert attn(**kw) == fa.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(d=32), dict(d=256), dict(d=80), dict(Hq=258, Hk=2), dict(dtype=fa.FA_DTYPE_F32),
                                dict(dtype=fa.FA_DTYPE_F32_SIMT)], ids=str)
def test_attention_outside_the_set_is_unsupported(kw):
    assert attn(**kw) == fa.FA_ERR_UNSUPPORTED


@pytest.mark.parametrize("Hq,Hk,max_q", [(4, 2, 1), (32, 1, 1), (33, 1, 1), (8, 1, 4), (8, 8, 300),
                                         (128, 1, 9)])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_workspace(Hq, Hk, max_q, d):
    """It does not depend on the lengths; a missing, short or misaligned one is
    refused."""
    need = fa.fa_fwd_kv4_workspace(3, Hq, Hk, max_q, d)
    assert 0 < need < 64 << 20
    assert need == fa.fa_fwd_kv4_workspace(60000, Hq, Hk, max_q, d)
    kw = dict(Hq=Hq, Hk=Hk, total=3 * max_q, max_q=max_q, d=d)
    for bad in (dict(ws=None), dict(wsb=need - 1), dict(ws=A(14) + 128), dict(ws=A(0)), dict(ws=A(11))):
        assert attn(**kw, **bad) == fa.FA_ERR_INVALID_ARG
    for args in ((0, Hq, Hk, max_q, d), (3, 0, Hk, max_q, d), (3, 7, 2, max_q, d), (3, Hq, Hk, 0, d),
                 (3, 129, 1, 1, d), (3, Hq, Hk, max_q, 0)):
        assert fa.fa_fwd_kv4_workspace(*args) == 0


@pytest.mark.parametrize("d", [-128, 1, 16, 32, 63, 80, 96, 192, 256])
def test_attention_needs_no_workspace_where_it_is_unsupported(d):
    for Hq, max_q in ((2, 1), (32, 9), (256, 1)):
        assert fa.fa_fwd_kv4_workspace(3, Hq, 2, max_q, d) == 0
        if d > 0 and d % 16 == 0:
            assert attn(Hq=Hq, total=max_q * 3, max_q=max_q, d=d) == fa.FA_ERR_UNSUPPORTED


SM = 152
MAX_KEYS = 2 ** 31 - 4096


@pytest.mark.parametrize("bound", [0, 1, 127, 128, 129, 8191, 8192, 131072, 2 ** 20, 2 ** 30,
                                   2 ** 31 - 4097, 2 ** 31 - 4096, 2 ** 31 - 129, 2 ** 31 - 127,
                                   2 ** 31 - 64, 2 ** 31 - 2, 2 ** 31 - 1])
@pytest.mark.parametrize("Hq,Hk,max_q", [(8, 8, 1), (32, 8, 1), (64, 8, 1), (8, 8, 9), (32, 1, 1),
                                         (32, 8, 64), (128, 1, 3), (1, 1, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_grid_for_any_bound(bound, Hq, Hk, max_q, d):
    """The grids for every bound on the keys up to the type's end and 1 to 65535
    sequences: at least one CTA, none whose parts the workspace does not hold,
    clusters only where one wave holds them and a CTA gets few units; and the
    table's width bounds the keys like the argument."""
    need = fa.fa_fwd_kv4_workspace(1, Hq, Hk, max_q, d)
    for B in (1, 2, 5, 19, 38, 39, 40, 56, 64, 152, 153, 304, 305, 448, 65535):
        for bs, width in ((16, 2 ** 27 - 1), (128, 2 ** 24 - 1), (16, 64), (128, 1)):
            st, keys, rows, cl, ctas, many = fa.fa_fwd_kv4_schedule(B, Hq, Hk, max_q, bound, width,
                                                                    bs, d, SM)
            assert st == fa.FA_OK
            assert keys == min(bound, width * bs, MAX_KEYS)
            assert rows in (0, 8, 16, 32) and cl in (0, 1, 2, 4, 8)
            heads, group = B * Hk, Hq // Hk
            assert rows == 0 or rows >= group
            assert (many > 0) == (max_q * group > rows) and 0 <= many <= SM
            if rows == 0:
                assert ctas == cl == 0 and many > 0
                continue
            unit = 64 if rows == 32 and d == 64 else 128
            units = max(1, -(-keys // unit))
            if cl:
                assert ctas == cl * heads <= 2 * SM and units <= 8 * cl
            else:
                assert 1 <= ctas <= min(2 * SM, heads * units)
                part = rows * (d + 2) * 4  # a CTA's record and its two parts
                assert need >= 304 * 16 + 2 * ctas * part
                if rows < 32 and heads <= SM:  # even one CTA a cluster would get too many
                    assert units > 8
            again = fa.fa_fwd_kv4_schedule(B, Hq, Hk, max_q, keys, width, bs, d, SM)
            assert again == (st, keys, rows, cl, ctas, many)


@pytest.mark.parametrize("kw,want", [
    (dict(), fa.FA_OK), (dict(B=0), 1), (dict(B=65536), 1), (dict(Hq=0), 1), (dict(Hq=9), 1),
    (dict(Hk=0), 1), (dict(max_q=0), 1), (dict(max_k=-1), 1), (dict(width=0), 1),
    (dict(width=2 ** 27), 1), (dict(bs=8), 1), (dict(sms=0), 1), (dict(sms=65536), 1),
    (dict(sms=2 ** 31 - 1), 1), (dict(d=0), 1),
    (dict(d=32), fa.FA_ERR_UNSUPPORTED), (dict(Hq=516), fa.FA_ERR_UNSUPPORTED)], ids=str)
def test_attention_schedule_refusals(kw, want):
    a = dict(dict(B=3, Hq=8, Hk=4, max_q=2, max_k=500, width=40, bs=16, d=128, sms=SM), **kw)
    assert fa.fa_fwd_kv4_schedule(*a.values())[0] == want


def test_wrappers_refuse_cpu_tensors_and_wrong_shapes():
    i32 = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.kv_plan(i32, i32, i32, torch.zeros(3, 2, dtype=torch.int32), 16, 4)
    cache = fa.kv4_cache(2, 1, 16, 64, device="cpu")
    assert [tuple(t.shape) for t in cache] == [(2, 1, 16, 32), (2, 1, 16, 4)] * 2
    x = torch.zeros(3, 1, 64)
    with pytest.raises(ValueError):
        fa.kv4_append(x, x, torch.zeros(3, dtype=torch.int64), *cache)
    with pytest.raises(ValueError):
        fa.rotary(x, None, torch.zeros(1, 3, dtype=torch.int32), torch.zeros(32, dtype=torch.int64))


# ------------------------------------------------------------------ the references
def test_reference_quantiser_picks_the_nearest_value():
    """Brute force over all codes, and the borders' ties."""
    x = torch.randn(50, 32, dtype=torch.float64, generator=torch.Generator().manual_seed(3))
    codes, scales = ref.quantise(x)
    got = ref.values(codes, scales)
    grid = torch.cat([ref.CODES, -ref.CODES])
    for r in range(50):
        for g in range(2):
            s = ref.SCALES[int(scales[r, g])]
            for e in range(16):
                v = x[r, 16 * g + e]
                assert abs(got[r, 16 * g + e] - v) == (grid * s - v).abs().min()
    tie = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0] * 2, dtype=torch.float64)
    codes, scales = ref.quantise(tie[None])
    assert ref.values(codes, scales)[0, :8].tolist() == [6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0]


@pytest.mark.parametrize("causal", [False, True])
def test_reference_attention_matches_a_loop(causal):
    g = torch.Generator().manual_seed(5)
    q, K, V = (torch.randn(s, dtype=torch.float64, generator=g) for s in
               ((3, 4, 16), (5, 2, 16), (5, 2, 16)))
    o, lse, _, _ = ref.attend(q, K, V, 0.3, causal)
    for i in range(3):
        for h in range(4):
            js = [j for j in range(5) if not causal or j <= 2 + i]
            w = [math.exp(0.3 * float(q[i, h] @ K[j, h // 2])) for j in js]
            assert abs(lse[h, i] - math.log(sum(w))) < 1e-12
            want = sum(x * V[j, h // 2] for x, j in zip(w, js)) / sum(w)
            assert (o[i, h] - want).abs().max() < 1e-12
