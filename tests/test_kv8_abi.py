"""Host-side checks of the 8-bit cache's operators and of the pages' (no GPU work:
every call here is refused, or is host-only) and the references of their GPU tests."""
import ctypes
import math
import os

import pytest
import torch

import kv8_util as k8
from exact_attention_57_gb300 import fa


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(fa.LIB_PATH):
        from exact_attention_57_gb300 import build
        build.build_library()
    return fa.load()


def A(i):
    """Fake device addresses, 16 TB apart; never dereferenced."""
    return (i + 1) << 44


host_only = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only: fake device addresses")
STORE = dict(kc=A(10), ks=A(11), vc=A(12), vs=A(13))
TAIL = dict(blocks=5, Hk=2, bs=16, d=64)
BAD_STORE = [dict(kc=None), dict(ks=None), dict(vc=None), dict(vs=None), dict(kc=A(10) + 16),
             dict(vc=A(12) + 8), dict(vs=A(13) + 2), dict(blocks=0), dict(Hk=0), dict(Hk=65536),
             dict(bs=24), dict(bs=0), dict(dtype=9), dict(d=0)]


def append(**kw):
    a = dict(dict(k=A(0), v=A(1), kst=128, vst=128, slots=A(2), T=3), **STORE, **TAIL,
             dtype=fa.FA_DTYPE_BF16)
    a.update(kw)
    return fa.fa_kv8_append(*a.values(), None)


def gather(**kw):
    a = dict(dict(slots=A(2), R=3), **STORE, ko=A(3), vo=A(4), **TAIL, dtype=fa.FA_DTYPE_BF16)
    a.update(kw)
    return fa.fa_kv8_gather(*a.values(), None)


@pytest.mark.parametrize("kw", BAD_STORE + [
    dict(k=None), dict(v=None), dict(slots=None), dict(T=0), dict(kst=127), dict(kst=132),
    dict(vst=120), dict(k=A(0) + 8), dict(slots=A(2) + 4), dict(vc=A(10) + 1024),
    dict(kc=A(0)), dict(vs=A(2) + 16), dict(ks=A(12) + 64), dict(vs=A(11) + 36),
], ids=str)
def test_append_refusals(kw):
    assert append(**kw) == fa.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", BAD_STORE + [
    dict(slots=None), dict(ko=None), dict(vo=None), dict(R=0), dict(ko=A(3) + 8), dict(vo=A(3)),
    dict(ko=A(10)), dict(vo=A(2) + 16), dict(vo=A(11)),
], ids=str)
def test_gather_refusals(kw):
    assert gather(**kw) == fa.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("d", [8, 72, 272])
def test_cache_head_dims_outside_the_set_are_unsupported(d):
    assert append(d=d, kst=2 * d, vst=2 * d) == fa.FA_ERR_UNSUPPORTED
    assert gather(d=d) == fa.FA_ERR_UNSUPPORTED


ATTN = dict(q=A(0), o=A(1), lse=A(2), **STORE, table=A(5), lens=A(6), cu=A(7), B=3, Hq=4, Hk=2,
            total=9, max_q=5, max_k=64, blocks=5, bs=16, width=4, d=64, scale=0.125, causal=1,
            dtype=fa.FA_DTYPE_BF16, ws=A(14), wsb=1 << 40)


def attn(**kw):
    return fa.fa_fwd_kv8(*dict(ATTN, **kw).values(), None)


@pytest.mark.parametrize("kw", BAD_STORE + [
    dict(q=None), dict(o=None), dict(lse=None), dict(table=None), dict(lens=None),
    dict(cu=None), dict(cu=None, max_q=1), dict(B=0), dict(B=65536), dict(Hq=0), dict(Hq=3),
    dict(total=0), dict(max_q=0), dict(max_q=10), dict(max_k=-1), dict(width=0),
    dict(width=1 << 28), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(scale=3e38), dict(causal=2), dict(q=A(0) + 8), dict(o=A(1) + 2),
    dict(lse=A(2) + 2), dict(table=A(5) + 1), dict(cu=A(7) + 2), dict(o=A(0)), dict(lse=A(1) + 16),
    dict(o=A(10) + 16), dict(lse=A(6) + 4), dict(lse=A(13) + 8),
], ids=str)
def test_attention_refusals(kw):
    assert attn(**kw) == fa.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(d=32), dict(d=256), dict(d=80), dict(Hq=258, Hk=2),
                                dict(dtype=fa.FA_DTYPE_F32), dict(dtype=fa.FA_DTYPE_F32_SIMT)],
                         ids=str)
def test_attention_outside_the_set_is_unsupported(kw):
    assert attn(**kw) == fa.FA_ERR_UNSUPPORTED


@pytest.mark.parametrize("Hq,Hk,max_q", [(4, 2, 1), (32, 1, 1), (33, 1, 1), (8, 1, 4), (8, 8, 300),
                                         (128, 1, 9)])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_workspace(Hq, Hk, max_q, d):
    need = fa.fa_fwd_kv8_workspace(3, Hq, Hk, max_q, d)
    assert 0 < need < 64 << 20
    assert need == fa.fa_fwd_kv8_workspace(60000, Hq, Hk, max_q, d)
    kw = dict(Hq=Hq, Hk=Hk, total=3 * max_q, max_q=max_q, d=d)
    for bad in (dict(ws=None), dict(wsb=need - 1), dict(ws=A(14) + 128), dict(ws=A(0)), dict(ws=A(11))):
        assert attn(**kw, **bad) == fa.FA_ERR_INVALID_ARG
    for args in ((0, Hq, Hk, max_q, d), (3, 0, Hk, max_q, d), (3, 7, 2, max_q, d), (3, Hq, Hk, 0, d),
                 (3, 129, 1, 1, d), (3, Hq, Hk, max_q, 0), (3, Hq, Hk, max_q, 96)):
        assert fa.fa_fwd_kv8_workspace(*args) == 0


SM = 152
MAX_KEYS = 2 ** 31 - 4096


@pytest.mark.parametrize("bound", [0, 1, 95, 96, 127, 128, 129, 160, 8191, 8192, 131072, 2 ** 20,
                                   2 ** 30, 2 ** 31 - 4097, 2 ** 31 - 4096, 2 ** 31 - 129,
                                   2 ** 31 - 1])
@pytest.mark.parametrize("Hq,Hk,max_q", [(8, 8, 1), (32, 8, 1), (64, 8, 1), (8, 8, 9), (32, 1, 1),
                                         (32, 8, 64), (128, 1, 3), (1, 1, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_grid_for_any_bound(bound, Hq, Hk, max_q, d):
    """The grids for every bound on the keys up to the type's end and 1 to 65535
    sequences: at least one CTA, none whose parts the workspace does not hold,
    clusters only where one wave holds them; and the table's width bounds the keys like
    the argument."""
    need = fa.fa_fwd_kv8_workspace(1, Hq, Hk, max_q, d)
    for B in (1, 2, 5, 19, 38, 39, 40, 56, 64, 152, 153, 304, 305, 448, 65535):
        for bs, width in ((16, 2 ** 27 - 1), (128, 2 ** 24 - 1), (16, 64), (128, 1)):
            st, keys, rows, cl, ctas, many = fa.fa_fwd_kv8_schedule(B, Hq, Hk, max_q, bound, width,
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
            if cl:
                assert ctas == cl * heads <= 2 * SM and keys <= 8 * 160 * cl
            else:
                assert 1 <= ctas <= 2 * SM
                part = rows * (d + 2) * 4  # a CTA's record and its two parts
                assert need >= 304 * 16 + 2 * ctas * part
            again = fa.fa_fwd_kv8_schedule(B, Hq, Hk, max_q, keys, width, bs, d, SM)
            assert again == (st, keys, rows, cl, ctas, many)


@pytest.mark.parametrize("kw,want", [
    (dict(), fa.FA_OK), (dict(B=0), 1), (dict(Hq=9), 1), (dict(Hk=0), 1), (dict(max_q=0), 1),
    (dict(max_k=-1), 1), (dict(width=2 ** 27), 1), (dict(bs=8), 1), (dict(sms=0), 1), (dict(d=0), 1),
    (dict(d=32), fa.FA_ERR_UNSUPPORTED), (dict(Hq=516), fa.FA_ERR_UNSUPPORTED)], ids=str)
def test_attention_schedule_refusals(kw, want):
    a = dict(dict(B=3, Hq=8, Hk=4, max_q=2, max_k=500, width=40, bs=16, d=128, sms=SM), **kw)
    assert fa.fa_fwd_kv8_schedule(*a.values())[0] == want


# ------------------------------------------------------------------ pages
def copy(**kw):
    a = dict(src=A(0), dst=A(1), n=3, frm=[A(10), A(11)], to=[A(10), A(11)], sizes=[64, 4], fb=9, tb=9)
    a.update(kw)
    return fa.fa_kv_copy(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(src=None), dict(dst=None), dict(src=A(0) + 2), dict(dst=A(1) + 1), dict(n=0), dict(fb=0),
    dict(tb=0), dict(frm=[], to=[], sizes=[]), dict(frm=[A(10), None]), dict(to=[None, A(11)]),
    dict(sizes=[64, 0]), dict(sizes=[1 << 31, 4]), dict(to=[A(10) + 64, A(11)]),
    dict(to=[A(11), A(10)], sizes=[64, 64]), dict(to=[A(12), A(12) + 64]),
    dict(frm=[A(10), A(10)], to=[A(10), A(11)]), dict(src=A(10) + 8), dict(dst=A(11)),
    dict(tb=8, frm=[A(10), A(11)], to=[A(10), A(10) + 8 * 64]),  # read behind what is written
], ids=str)
def test_copy_refusals(kw):
    assert copy(**kw) == fa.FA_ERR_INVALID_ARG


def test_copy_of_too_many_arrays_is_unsupported():
    many = [A(10) + 4096 * i for i in range(257)]
    assert copy(frm=many, to=many, sizes=[64] * 257) == fa.FA_ERR_UNSUPPORTED


@host_only
@pytest.mark.parametrize("kw", [
    dict(), dict(to=[A(12), A(13)], tb=3), dict(frm=[A(10), A(10) + 9 * 64], to=[A(10), A(10) + 9 * 64]),
    dict(frm=[A(10), A(10)], to=[A(12), A(13)], sizes=[64, 64]),  # one array read twice
    dict(frm=[A(10) + 4096 * i for i in range(256)], to=[A(10) + 4096 * i for i in range(256)],
         sizes=[64] * 256),
], ids=["one cache", "two caches", "side by side", "read twice", "256 arrays"])
def test_copy_takes_arrays_that_lie_apart(kw):
    """These pass all checks and end at the device's, as there is none."""
    assert copy(**kw) in (fa.FA_ERR_CUDA, fa.FA_ERR_UNSUPPORTED)


@host_only
def test_overlap_check_against_the_bytes_themselves():
    import random
    r = random.Random(3)
    taken = refused = 0
    for _ in range(3000):
        n = r.choice([1, 2, 3, 5])
        fb, tb = r.choice([1, 2, 3]), r.choice([1, 2, 3])
        sizes = [r.choice([1, 4, 7]) for _ in range(n)]
        frm = [r.randrange(0, 120) for _ in range(n)]
        to = [f if r.random() < 0.5 else r.randrange(0, 120) for f in frm]
        rd = [set(range(f, f + s * fb)) for f, s in zip(frm, sizes)]
        wr = [set(range(t, t + s * tb)) for t, s in zip(to, sizes)]
        bad = any(wr[i] & wr[j] for i in range(n) for j in range(i))
        bad |= any(wr[i] & rd[j] for i in range(n) for j in range(n) if i != j or frm[i] != to[i])
        st = copy(frm=[A(10) + x for x in frm], to=[A(10) + x for x in to], sizes=sizes, fb=fb, tb=tb)
        assert (st == fa.FA_ERR_INVALID_ARG) == bad, (frm, to, sizes, fb, tb)
        refused += bad
        taken += not bad
    assert taken > 100 and refused > 500


FORK = dict(table=A(0), lens=A(1), parents=A(2), free=A(3), head=None, table_out=A(4), lens_out=A(5),
            counts=A(6), B=3, n=4, width=5, bs=16, num_free=9, blocks=20, end=0, arrays=[A(10)],
            sizes=[64])


def fork(**kw):
    return fa.fa_kv_fork(*dict(FORK, **kw).values(), None)


@pytest.mark.parametrize("kw", [
    dict(table=None), dict(lens=None), dict(parents=None), dict(free=None), dict(table_out=None),
    dict(lens_out=None), dict(counts=None), dict(B=0), dict(B=65536), dict(n=0), dict(n=65536),
    dict(width=0), dict(width=1 << 28), dict(bs=48), dict(num_free=-1), dict(blocks=0), dict(end=2),
    dict(table=A(0) + 2), dict(counts=A(6) + 1), dict(head=A(7) + 2), dict(table_out=A(0) + 16),
    dict(lens_out=A(1)), dict(counts=A(3) + 32), dict(head=A(4) + 8), dict(table_out=A(10) + 32),
    dict(parents=A(10)), dict(arrays=[None]), dict(sizes=[0]), dict(arrays=[A(10), A(10)], sizes=[8, 8]),
], ids=str)
def test_fork_refusals(kw):
    assert fork(**kw) == fa.FA_ERR_INVALID_ARG


@host_only
@pytest.mark.parametrize("kw", [dict(), dict(arrays=[], sizes=[]), dict(free=None, num_free=0),
                                dict(head=A(7)), dict(end=1)], ids=str)
def test_fork_takes(kw):
    assert fork(**kw) in (fa.FA_ERR_CUDA, fa.FA_ERR_UNSUPPORTED)


FREE = dict(table=A(0), lens=A(1), ended=None, free=A(2), head=A(3), B=3, width=5, bs=16, blocks=20)


def free(**kw):
    return fa.fa_kv_free(*dict(FREE, **kw).values(), None)


@pytest.mark.parametrize("kw", [
    dict(table=None), dict(lens=None), dict(free=None), dict(head=None), dict(B=0), dict(B=65536),
    dict(width=0), dict(width=1 << 28), dict(bs=8), dict(blocks=0), dict(table=A(0) + 1),
    dict(head=A(3) + 2), dict(free=A(0)), dict(lens=A(0) + 20), dict(head=A(2) + 40),
    dict(ended=A(1) + 3), dict(ended=A(2)),
], ids=str)
def test_free_refusals(kw):
    assert free(**kw) == fa.FA_ERR_INVALID_ARG


COMPACT = dict(table=A(0), lens=A(1), table_out=A(2), new_ids=A(3), counts=A(4), B=3, width=5, bs=16,
               blocks=20, arrays=[A(10)], sizes=[64], ws=A(5), wsb=1 << 30)


def compact(**kw):
    return fa.fa_kv_compact(*dict(COMPACT, **kw).values(), None)


@pytest.mark.parametrize("kw", [
    dict(table=None), dict(lens=None), dict(table_out=None), dict(new_ids=None), dict(counts=None),
    dict(B=0), dict(B=65536), dict(width=0), dict(width=1 << 28), dict(bs=8), dict(blocks=0),
    dict(ws=None), dict(wsb=8 * 10 + 7), dict(ws=A(5) + 2), dict(table_out=A(0) + 4),
    dict(new_ids=A(0)), dict(counts=A(1) + 8), dict(ws=A(3) + 16), dict(new_ids=A(10)),
    dict(lens=A(10) + 64), dict(ws=A(10)), dict(arrays=[None]), dict(sizes=[0]), dict(table=A(0) + 1),
], ids=str)
def test_compact_refusals(kw):
    assert compact(**kw) == fa.FA_ERR_INVALID_ARG


def test_more_blocks_than_a_sweep_takes_are_unsupported():
    assert free(blocks=(1 << 23) + 1) == fa.FA_ERR_UNSUPPORTED
    assert compact(blocks=(1 << 23) + 1) == fa.FA_ERR_UNSUPPORTED
    assert fa.fa_kv_compact_workspace((1 << 23) + 1) == fa.fa_kv_compact_workspace(0) == 0
    assert 0 < fa.fa_kv_compact_workspace(1) <= fa.fa_kv_compact_workspace(1 << 23) < 64 << 20


@host_only
def test_compact_takes_its_own_table():
    assert compact(table_out=A(0)) in (fa.FA_ERR_CUDA, fa.FA_ERR_UNSUPPORTED)
    assert free() in (fa.FA_ERR_CUDA, fa.FA_ERR_UNSUPPORTED)
    assert free(blocks=1 << 23) in (fa.FA_ERR_CUDA, fa.FA_ERR_UNSUPPORTED)


def test_wrappers_refuse_cpu_tensors():
    i32 = torch.zeros(3, dtype=torch.int32)
    cache = fa.kv8_cache(2, 1, 16, 64, device="cpu")
    assert [tuple(t.shape) for t in cache] == [(2, 1, 16, 64), (2, 1)] * 2
    assert [t.dtype for t in cache] == [torch.float8_e4m3fn, torch.float32] * 2
    x, t = torch.zeros(3, 1, 64), torch.zeros(3, 2, dtype=torch.int32)
    for call in (lambda: fa.kv8_append(x, x, torch.zeros(3, dtype=torch.int64), *cache),
                 lambda: fa.kv8_gather(torch.zeros(3, dtype=torch.int64), *cache),
                 lambda: fa.attention_kv8(x.half(), *cache, t, i32, 9),
                 lambda: fa.kv_copy(i32, i32, cache), lambda: fa.kv_fork(t, i32, i32, i32, 16, cache),
                 lambda: fa.kv_free(t, i32, 9, 16), lambda: fa.kv_compact(t, i32, cache, 16)):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------------ the references
def test_reference_codes_are_the_nearest():
    """Brute force over all codes, and the ties."""
    x = torch.randn(4000, dtype=torch.float64, generator=torch.Generator().manual_seed(3)) * 3
    got = k8.numbers(k8.codes_of(x))
    every = torch.cat([k8.GRID, -k8.GRID])
    assert torch.equal((got - x).abs(), (every[None] - x[:, None]).abs().amin(1))
    mid = (k8.GRID[1:] + k8.GRID[:-1]) / 2
    assert (k8.codes_of(mid) % 2 == 0).all() and (k8.codes_of(-mid) % 2 == 0).all()
    # as torch rounds them
    f = (torch.randn(4000, generator=torch.Generator().manual_seed(4)) * 30).clamp(-448, 448)
    assert torch.equal(k8.codes_of(f.double()), f.to(torch.float8_e4m3fn).view(torch.uint8))
    assert k8.codes_of(torch.tensor([math.inf, -math.inf, math.nan])).tolist() == [126, 254, 126]


def test_reference_exponent():
    for e in range(-40, 41):
        a = 448 * 2.0 ** e
        assert k8.exponent(a) == e
        assert k8.exponent(math.nextafter(a, math.inf)) == min(e + 1, 40)
    assert k8.exponent(0.0) == -40 and k8.exponent(1e300) == 40


def test_reference_pages_against_sets():
    """The free list and the compacted tables against what they have to be."""
    import random
    r = random.Random(1)
    for _ in range(200):
        B, width, bs, blocks = r.randrange(1, 5), r.randrange(1, 5), 16, r.randrange(1, 30)
        table = [[r.randrange(-2, blocks + 2) for _ in range(width)] for _ in range(B)]
        lens = [r.randrange(-5, width * bs + 20) for _ in range(B)]
        free, L = k8.free_list(table, lens, bs, blocks)
        have = k8.held(table, lens, bs, blocks)
        assert sorted(have | set(free[L:])) == list(range(blocks)) and len(have) == L
        out, new, (held, moved), moves = k8.compact(table, lens, bs, blocks)
        assert held == L and moved == len(moves)
        assert {new[i] for i in have} == set(range(L))
        for row, o, n in zip(table, out, lens):
            for j, (a, b) in enumerate(zip(row, o)):
                inside = j < -(-max(n, 0) // bs) and 0 <= a < blocks
                assert b == (new[a] if inside else -1)
