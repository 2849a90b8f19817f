"""Plain 64-bit references of the 8-bit cache and of the pages' operators (CPU,
torch and Python integers only; nothing of the library is used)."""
import math

import torch

import serve_util as ref

GRID = ref.SCALES  # e4m3, 0 .. 448: index and code are the same


def codes_of(y):
    """uint8 codes of the nearest e4m3 numbers; NaN as 448."""
    y = torch.nan_to_num(y.double(), nan=448.0, posinf=448.0, neginf=-448.0)
    return (ref.nearest(y.abs(), GRID) + 128 * (y < 0)).to(torch.uint8)


def numbers(codes):
    """float64 numbers of uint8 codes; 0x7F and 0xFF are NaN."""
    every = torch.cat([GRID, torch.tensor([math.nan], dtype=torch.float64)])
    v = every[(codes & 127).long()]
    return torch.where(codes >= 128, -v, v)


def values(codes, scales):
    """float64 values of codes [blocks, Hk, bs, d] and scales [blocks, Hk]."""
    return numbers(codes) * scales.double()[:, :, None, None]


def exponent(a):
    """The least e in -40 .. 40 with a <= 448 * 2^e."""
    e = -40
    while e < 40 and a > 448 * 2.0 ** e:
        e += 1
    return e


def append(x, slots, codes, scales):
    """Rows x [T, Hk, d] written into copies of codes (uint8) and scales.  Quotients
    are fp32's, correctly rounded: exact for scales that are powers of two."""
    codes, scales = codes.clone(), scales.clone()
    blocks, Hk, bs, d = codes.shape
    runs = {}
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < blocks * bs:
            runs.setdefault(s // bs, []).append((t, s % bs))
    for b, rows in runs.items():
        t, off = (torch.tensor(v) for v in zip(*rows))
        first = int(off.min())
        for h in range(Hk):
            y = x[t, h].double()
            fin = y[torch.isfinite(y)].abs()
            fit = 2.0 ** exponent(float(fin.max()) if fin.numel() else 0.0)
            old = float(scales[b, h])
            old = old if 0 < old < math.inf else 0.0
            new = fit if first == 0 else max(old, fit)
            if first > 0 and new != old:
                by = torch.tensor(old) / torch.tensor(new)  # in fp32, as the format says
                codes[b, h, :first] = codes_of(numbers(codes[b, h, :first]).float() * by)
            codes[b, h, off] = codes_of(y.float() / torch.tensor(new))
            scales[b, h] = new
    return codes, scales


def random_store(blocks, Hk, bs, d, g, spread=3, odd=False):
    """(codes uint8, scales float32) of normal numbers, blocks of different size;
    odd: scales that are no powers of two."""
    x = torch.randn(blocks, Hk, bs, d, generator=g)
    scales = 2.0 ** torch.randint(-8 - spread, -6 + spread, (blocks, Hk), generator=g).float()
    size = scales * (64 + 300 * torch.rand(blocks, Hk, generator=g)) / 4
    if odd:
        scales = scales * (1 + torch.rand(blocks, Hk, generator=g))
    x = x * size[:, :, None, None]
    return codes_of(x.double() / scales.double()[:, :, None, None]), scales


def on(cache, device):
    """Arrays (codes uint8, scales, ...) as the library takes them."""
    return [c.to(device).view(torch.float8_e4m3fn) if c.dtype == torch.uint8 else c.to(device)
            for c in cache]


# ------------------------------------------------------------------ pages
def blocks_of(n, width, bs):
    return min(width, -(-max(0, n) // bs))


def fork(table, lens, parents, free, head, bs, blocks, end):
    """(table_out, lens_out, counts, copies [(src, dst)])."""
    width = len(table[0])
    out, new, copies, used, seen = [], [], [], 0, set()
    for p in parents:
        ok = 0 <= p < len(table)
        n = min(max(0, lens[p]), width * bs) if ok else 0
        full = n // bs
        row = (list(table[p][:full]) if ok else []) + [-1] * (width - full)
        if n % bs:
            src = table[p][full]
            if end and p not in seen:
                row[full] = src
            elif 0 <= src < blocks:
                at = head + used
                used += 1
                f = free[at] if at < len(free) else -1
                row[full] = f if 0 <= f < blocks else -1
                if row[full] >= 0:
                    copies.append((src, f))
        seen.add(p)
        out.append(row)
        new.append(n)
    return out, new, [used, min(head + used, len(free))], copies


def held(table, lens, bs, blocks, ended=None):
    got = set()
    for b, row in enumerate(table):
        if ended is None or not ended[b]:
            got |= {i for i in row[:blocks_of(lens[b], len(row), bs)] if 0 <= i < blocks}
    return got


def free_list(table, lens, bs, blocks, ended=None):
    have = held(table, lens, bs, blocks, ended)
    return [-1] * len(have) + [i for i in range(blocks) if i not in have], len(have)


def compact(table, lens, bs, blocks):
    """(table_out, new_ids, counts, moves [(src, dst)])."""
    have = held(table, lens, bs, blocks)
    L = len(have)
    moves = list(zip(sorted(i for i in have if i >= L), [i for i in range(L) if i not in have]))
    new = [i if i in have and i < L else -1 for i in range(blocks)]
    for s, d in moves:
        new[s] = d
    out = []
    for b, row in enumerate(table):
        need = blocks_of(lens[b], len(row), bs)
        out.append([new[i] if j < need and 0 <= i < blocks else -1 for j, i in enumerate(row)])
    return out, new, [L, len(moves)], moves
