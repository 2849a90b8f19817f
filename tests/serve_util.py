"""Plain 64-bit references of the serving operators (CPU, torch and Python
integers only; nothing of the library is used)."""
import math

import torch

CODES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
SCALES = torch.tensor([math.ldexp(n % 8, -9) if n < 8 else math.ldexp(8 + n % 8, n // 8 - 10)
                       for n in range(127)], dtype=torch.float64)  # e4m3, 0 .. 448
BS_LOG2 = {16: 4, 32: 5, 64: 6, 128: 7}


def nearest(y, grid):
    """Index of the nearest of ascending `grid` to y >= 0, the even one of two
    as near; past the end, the last."""
    y = y.clamp(max=float(grid[-1]))
    hi = torch.searchsorted(grid, y.contiguous()).clamp(1, grid.numel() - 1)
    lo = hi - 1
    dl, dh = y - grid[lo], grid[hi] - y
    return torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def quantise(x, exp=0):
    """(codes [..., d/2], scales [..., d/16]) uint8 of x [..., d]."""
    g = x.double().unflatten(-1, (-1, 16)) * 2.0 ** -exp
    s = nearest(g.abs().amax(-1) / 6, SCALES)
    f = SCALES[s].unsqueeze(-1)
    y = torch.where(f > 0, g / f, 0.0)
    c = nearest(y.abs(), CODES) + 8 * (y < 0)
    c = c.flatten(-2).unflatten(-1, (-1, 2))
    return (c[..., 0] + 16 * c[..., 1]).to(torch.uint8), s.to(torch.uint8)


def values(codes, scales, exp=0):
    """float64 values of packed rows."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    v = torch.where(c >= 8, -CODES[c % 8], CODES[c % 8])
    every = torch.cat([SCALES, torch.full((129,), math.nan, dtype=torch.float64)])
    return v * every[scales.long()].repeat_interleave(16, -1) * 2.0 ** exp


def plan(cached, new, free, head, table, bs, cap):
    """Block tables and slot maps, request by request, on lists of ints."""
    table = [list(r) for r in table]
    width = len(table[0])
    reach = width * bs
    slots, pos, cu, lens, used = [], [], [0], [], 0
    for b, (c, n) in enumerate(zip(cached, new)):
        c, n = max(0, c), max(0, n)
        have, tot = -(-min(c, reach) // bs), -(-min(c + n, reach) // bs)
        for j in range(have, tot):
            at = head + used
            table[b][j] = free[at] if at < len(free) else -1
            used += 1
        for p in range(c, c + n):
            blk = table[b][p // bs] if p < reach else -1
            slots.append(blk * bs + p % bs if blk >= 0 else -1)
            pos.append(p)
        cu.append(min(cap, cu[-1] + n))
        lens.append(min(c + n, reach))
    total = len(slots)
    slots, pos = slots[:cap], pos[:cap]
    pad = cap - len(slots)
    return (table, slots + [-1] * pad, pos + [0] * pad, cu, lens, [used, total])


def rotate(x, pos, freq, axis, rot, interleaved=False, inverse=False):
    """x [B, H, N, d] turned by pos [axes, B, N]; float64."""
    t = pos.double()[axis].permute(1, 2, 0) * freq  # [B, N, rot/2]
    z = torch.polar(torch.ones_like(t), -t if inverse else t).unsqueeze(1)
    y = x.double().clone()
    if interleaved:
        w = torch.view_as_complex(y[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * z
        y[..., :rot] = torch.view_as_real(w).flatten(-2)
    else:
        w = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * z
        y[..., :rot // 2], y[..., rot // 2:rot] = w.real, w.imag
    return y


def attend(q, K, V, scale, causal, allowed=None):
    """O [nq, Hq, d], LSE [Hq, nq], A (the softmax average of |v|, [nq, Hq, d])
    and S (largest sum |q||k| over a row's keys, [Hq, nq]) of one sequence: q
    [nq, Hq, d], K and V [nk, Hk, d], float64; allowed: bool [nk]."""
    nq, Hq, d = q.shape
    nk, Hk, _ = K.shape
    g = Hq // Hk
    K, V = (x.repeat_interleave(g, 1) for x in (K, V))
    s = torch.einsum("ihd,jhd->hij", q, K) * scale
    size = torch.einsum("ihd,jhd->hij", q.abs(), K.abs())
    ok = torch.ones(nq, nk, dtype=torch.bool)
    if causal:
        i, j = torch.arange(nq)[:, None], torch.arange(nk)[None]
        ok &= j <= nk - nq + i
    if allowed is not None:
        ok &= allowed[None]
    s = s.masked_fill(~ok, -math.inf)
    lse = torch.logsumexp(s, -1) if nk else torch.full((Hq, nq), -math.inf, dtype=torch.float64)
    p = torch.where(lse[..., None] > -math.inf, (s - lse[..., None]).exp(), 0.0)
    p = torch.nan_to_num(p, nan=0.0)
    o, a = (torch.einsum("hij,jhd->ihd", p, v) for v in (V, V.abs()))
    big = size.masked_fill(~ok, 0.0).amax(-1) if nk else torch.zeros(Hq, nq, dtype=torch.float64)
    return o, lse, a, big
