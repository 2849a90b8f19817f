"""Measured cases of the serving operators around the attention kernels.

Four operators, in the order in which a server's step uses them:

  plan    block tables and slot maps of a paged cache, from request lengths
  rotary  rotary positions with several axes on queries and keys (and the
          inverse rotation, their gradient)
  cache   new keys and values written into a paged cache held in 4 bits, and
          rows of that cache read back
  attn    attention of the new queries over that cache

`own` selects what `run` executes: False, the plain form in elementary torch
operations; True, the calls of exact_attention_57_gb300.fa.

Cache format: a block holds `bs` tokens; codes [blocks, Hk, bs, d/2] uint8
(two e2m1 numbers a byte, the even element in the low half), scales
[blocks, Hk, bs, d/16] uint8 (one e4m3 number for 16 elements); an element is
code * scale * 2^exp.
"""
import math
from fractions import Fraction

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
INV_2PI = Fraction("0.15915494309189533576888376337251436203445964574045644874766734405889679763")


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token more for each of 256 running requests: a server's decode step
        dict(name="plan decode b256", op="plan", B=256, bs=16, cached=8192, new=1, cap=256),
        # 37 prompts admitted together, ragged, some with a cached prefix
        dict(name="plan prefill b37", op="plan", B=37, bs=64, cached=1024, new=8192, cap=160000),
        # queries and keys of a decode step, slices of a fused projection's output
        dict(name="rotary decode t64", op="rotary", layout="thd", B=1, N=64, Hq=32, Hk=8, d=128,
             rot=128, axes=1, interleaved=False, inverse=False, dtype="bf16"),
        # a video of 18 frames of 32 x 32 patches (time, height, width)
        dict(name="rotary video n18432", op="rotary", layout="bhnd", B=1, N=18432, Hq=16, Hk=16,
             d=128, rot=128, axes=3, interleaved=False, inverse=False, dtype="bf16"),
        # gradients of a partial rotation in a training step, odd length
        dict(name="rotary backward n3001", op="rotary", layout="bhnd", B=2, N=3001, Hq=8, Hk=8,
             d=80, rot=64, axes=2, interleaved=True, inverse=True, dtype="fp32"),
        # a decode step's 64 new tokens written, their rows read back
        dict(name="cache decode t64", op="cache", T=64, R=64, Hk=8, d=128, bs=16, blocks=4096,
             dtype="bf16"),
        # a prompt written behind a cached prefix, and the whole context read back
        dict(name="cache prefill t16383", op="cache", T=16383, R=24575, Hk=8, d=128, bs=64,
             blocks=1024, dtype="fp16"),
        # one user, a short context: latency
        dict(name="attn decode b1 k1023", op="attn", B=1, nq=1, k_max=1023, Hq=32, Hk=8, d=128,
             bs=16, dtype="bf16"),
        # a batch of users with ragged contexts: a server's usual step
        dict(name="attn decode b64 k8192", op="attn", B=64, nq=1, k_max=8192, Hq=32, Hk=8, d=128,
             bs=16, dtype="bf16"),
        # one long document
        dict(name="attn decode b1 k131071", op="attn", B=1, nq=1, k_max=131071, Hq=32, Hk=8, d=128,
             bs=64, dtype="bf16"),
        # a few drafted tokens checked at once, one key head a query head
        dict(name="attn draft b16 k3001", op="attn", B=16, nq=4, k_max=3001, Hq=16, Hk=16, d=64,
             bs=32, dtype="fp16"),
        # a chunk of a prompt against what is cached
        dict(name="attn chunk b2 q2048", op="attn", B=2, nq=2048, k_max=8192, Hq=32, Hk=8, d=128,
             bs=64, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["plan", "rotary", "rotary", "cache", "attn", "attn", "attn"])
    if op == "plan":
        B = _log(rng, 1, 512)
        new = rng.choice([1, 1, _log(rng, 2, 8192)])
        cap = sum(_lens(B, new, 1 if new == 1 else 0)) + rng.randrange(0, 99)
        while cap > 160000:
            B = max(1, B // 2)
            cap = sum(_lens(B, new, 0)) + rng.randrange(0, 99)
        return dict(op="plan", B=B, bs=rng.choice([16, 32, 64, 128]), cached=_log(rng, 16, 8192),
                    new=new, cap=cap)
    if op == "rotary":
        axes = rng.choice([1, 2, 3])
        d = rng.choice([32, 64, 72, 80, 96, 128, 256])
        rot = rng.choice([d, d, d // 2])
        Hk = rng.choice([1, 2, 4, 8])
        Hq = Hk * rng.choice([1, 2, 4])
        layout = rng.choice(["thd", "bhnd"])
        B = 1 if layout == "thd" else rng.choice([1, 2, 3])
        top = 18432 * 32 * 128 // ((Hq + Hk) * d * B)
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        N = _log(rng, 1, min(18432, top // (2 if dtype == "fp32" else 1)))
        return dict(op="rotary", layout=layout, B=B, N=N, Hq=Hq, Hk=Hk, d=d, rot=rot, axes=axes,
                    interleaved=rng.random() < 0.4, inverse=rng.random() < 0.4, dtype=dtype)
    if op == "cache":
        d, Hk = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
        bs = rng.choice([16, 32, 64, 128])
        T = _log(rng, 1, 16383)
        R = T + rng.randrange(0, 8192)
        return dict(op="cache", T=T, R=R, Hk=Hk, d=d, bs=bs, blocks=-(-R // bs) + rng.randrange(1, 512),
                    dtype=rng.choice(["bf16", "fp16", "fp32"]))
    d, Hk, g = rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 4, 5, 8, 16])
    bs, dtype = rng.choice([16, 32, 64, 128]), rng.choice(["bf16", "fp16"])
    kind = rng.choice(["decode", "decode", "draft", "chunk"])
    if kind == "decode":
        nq, B = 1, _log(rng, 1, 128)
        k_max = _log(rng, 1, 65536)
    elif kind == "draft":
        nq, B = rng.randrange(2, 9), _log(rng, 1, 64)
        k_max = _log(rng, 16, 16384)
    else:
        nq, B = _log(rng, 9, 2048), rng.choice([1, 2, 3])
        k_max = max(nq, _log(rng, 64, 8192))
    # no larger than the listed ones: tokens * heads of the cache, and scores
    while B * k_max * Hk * d > 64 * 8192 * 8 * 128 or B * nq * Hk * g * k_max > 2 ** 30:
        B, k_max = (B // 2, k_max) if B > 1 else (1, k_max // 2)
        nq = min(nq, k_max)
    return dict(op="attn", B=B, nq=nq, k_max=k_max, Hq=Hk * g, Hk=Hk, d=d, bs=bs, dtype=dtype)


# ------------------------------------------------------------------ inputs
def _lens(n, top, low=0):
    """n ragged lengths in low .. top, the longest first: the same for every
    seed, so that a case's work is known; prepare() puts them in an order."""
    return [top] + [low + (top - low) * ((i * 7919 + 13) % 997) // 996 for i in range(1, n)]


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _shuffled(values, g):
    t = torch.tensor(values, dtype=torch.int64, device="cuda")
    return t[torch.randperm(len(values), device="cuda", generator=g)]


def _k_lens(case):
    return [max(0, x) for x in _lens(case["B"], case["k_max"], case["nq"])] if case["B"] > 1 \
        else [case["k_max"]]


def _prepare_plan(case, g):
    B, bs = case["B"], case["bs"]
    cached = _shuffled(_lens(B, case["cached"], 0 if case["new"] > 1 else 1), g)
    new = _shuffled(_lens(B, case["new"], 1 if case["new"] == 1 else 0), g)
    have, tot = (cached + bs - 1) // bs, (cached + new + bs - 1) // bs
    need, n_have = int((tot - have).sum()), int(have.sum())
    blocks = torch.randperm(need + n_have + 64, device="cuda", generator=g).int()
    width = -(-(case["cached"] + case["new"]) // bs)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    held = torch.arange(width, device="cuda")[None] < have[:, None]
    table[held] = blocks[:n_have]
    cap = case["cap"]
    out = tuple(torch.empty(n, dtype=t, device="cuda") for n, t in
                ((cap, torch.int64), (cap, torch.int32), (B + 1, torch.int32), (B, torch.int32),
                 (2, torch.int32)))
    return dict(cached=cached.int(), new=new.int(), free=blocks[n_have:].contiguous(), table=table,
                out=out)


def _prepare_rotary(case, g):
    B, N, Hq, Hk, d, rot, A = (case[k] for k in ("B", "N", "Hq", "Hk", "d", "rot", "axes"))
    dt = DT[case["dtype"]]
    if case["layout"] == "thd":  # slices of one projection's output
        qkv = torch.randn(N, Hq + 2 * Hk, d, device="cuda", generator=g).to(dt)
        q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    else:
        q, k = (torch.randn(B, h, N, d, device="cuda", generator=g).to(dt) for h in (Hq, Hk))
    # positions: a grid of the axes behind an offset that differs by row, far in for text
    n = torch.arange(N, device="cuda")
    first = torch.randint(0, 100000 if A == 1 else 3000, (B, 1), device="cuda", generator=g)
    if A == 1:
        pos = (first + n)[None]
    elif A == 2:
        pos = torch.stack([first + n // 57, first + n % 57])
    else:
        pos = torch.stack([first + n // 1024, first + n // 32 % 32, first + n % 32])
    pos = pos.int().reshape(A, N if case["layout"] == "thd" else B * N).reshape(
        (A, N) if case["layout"] == "thd" else (A, B, N)).contiguous()
    # one ladder of frequencies over the pairs, dealt to the axes in sections
    half = rot // 2
    freq = [10000.0 ** (-2.0 * i / rot) for i in range(half)]
    axis = [min(A - 1, i * A // half) for i in range(half)]
    words = [((int(Fraction(f) * INV_2PI * 2 ** 64) % 2 ** 64) & ~3) | a for f, a in zip(freq, axis)]
    table = torch.tensor([w - 2 ** 64 if w >= 2 ** 63 else w for w in words], dtype=torch.int64,
                         device="cuda")
    return dict(q=q, k=k, pos=pos, table=table,
                freq=torch.tensor(freq, dtype=torch.float64, device="cuda"),
                axis=torch.tensor(axis, dtype=torch.int64, device="cuda"))


def _random_cache(blocks, Hk, bs, d, g):
    """Cache buffers of quantised normal numbers, made block row by block row."""
    codes = torch.empty(blocks, Hk, bs, d // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(blocks, Hk, bs, d // 16, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (Hk * bs * d))
    for b in range(0, blocks, step):
        n = min(step, blocks - b)
        x = torch.randn(n, Hk, bs, d, device="cuda", generator=g)
        codes[b:b + n], scales[b:b + n] = _quantise(x)
    return codes, scales


def _prepare_cache(case, g):
    T, R, Hk, d, bs, blocks = (case[k] for k in ("T", "R", "Hk", "d", "bs", "blocks"))
    dt = DT[case["dtype"]]
    qkv = torch.randn(T, 4 * Hk, d, device="cuda", generator=g).to(dt)
    qkv[:, :, ::16] *= 4.0  # a few large channels, as keys have them
    need = -(-R // bs)
    ids = torch.randperm(blocks, device="cuda", generator=g)[:need]
    rows = torch.arange(R, device="cuda")
    slots = ids[rows // bs] * bs + rows % bs
    cache = _random_cache(blocks, Hk, bs, d, g) + _random_cache(blocks, Hk, bs, d, g)
    out = tuple(torch.empty(R, Hk, d, dtype=dt, device="cuda") for _ in range(2))
    return dict(k=qkv[:, 2 * Hk:3 * Hk], v=qkv[:, 3 * Hk:], write=slots[R - T:].contiguous(),
                read=slots, cache=cache, out=out)


def _prepare_attn(case, g):
    B, nq, Hq, Hk, d, bs = (case[k] for k in ("B", "nq", "Hq", "Hk", "d", "bs"))
    lens = _shuffled(_k_lens(case), g)
    need = (lens + bs - 1) // bs
    total = int(need.sum())
    blocks = total + 8
    cache = _random_cache(blocks, Hk, bs, d, g) + _random_cache(blocks, Hk, bs, d, g)
    width = -(-case["k_max"] // bs)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(width, device="cuda")[None] < need[:, None]] = \
        torch.randperm(blocks, device="cuda", generator=g)[:total].int()
    dt = DT[case["dtype"]]
    q = torch.randn(B * nq, Hq, d, device="cuda", generator=g).to(dt)
    cu = torch.arange(0, (B + 1) * nq, nq, dtype=torch.int32, device="cuda")
    return dict(q=q, cu=cu, lens=lens.int(), table=table, cache=cache, out=torch.empty_like(q),
                lse=torch.empty(Hq, B * nq, device="cuda"))


def prepare(case, seed):
    g = _gen(seed)
    state = {"plan": _prepare_plan, "rotary": _prepare_rotary, "cache": _prepare_cache,
             "attn": _prepare_attn}[case["op"]](case, g)
    return dict(case, **state)


# ------------------------------------------------------------- plain forms
def _quantise(x):
    """(codes, scales) of x [..., d], d a multiple of 16: one e4m3 scale for
    16 elements, amax / 6 rounded to nearest; e2m1 codes of x / scale, rounded
    to nearest, ties to the even code.  In 64 bits: borders decide codes."""
    g = x.double().unflatten(-1, (-1, 16))
    scale = (g.abs().amax(-1) / 6).float().clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.double().unsqueeze(-1)
    y = torch.where(s > 0, g / s, 0.0)
    a = y.abs()
    code = torch.zeros_like(a, dtype=torch.uint8)
    # a border between codes i and i + 1 belongs to the even one
    code += a > 0.25
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    code |= torch.where(y < 0, 8, 0).to(torch.uint8)
    code = code.flatten(-2).unflatten(-1, (-1, 2))
    return code[..., 0] | (code[..., 1] << 4), scale.view(torch.uint8)


def _values(codes, scales):
    """float32 values of packed rows [..., d/2] and their scales [..., d/16]."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    grid = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device)
    s = scales.view(torch.float8_e4m3fn).float()
    return (grid[c.int()].unflatten(-1, (-1, 16)) * s.unsqueeze(-1)).flatten(-2)


def _plain_plan(s):
    bs, cap, B = s["bs"], s["cap"], s["B"]
    cached, new, table, free = s["cached"].long(), s["new"].long(), s["table"], s["free"]
    have = (cached + bs - 1) // bs
    need = (cached + new + bs - 1) // bs - have
    off = need.cumsum(0) - need
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    j = torch.arange(table.shape[1], device=table.device)[None] - have[:, None]
    fresh = (j >= 0) & (j < need[:, None])
    at = (off[:, None] + j).clamp(0, free.numel() - 1)
    table.copy_(torch.where(fresh, free[at], table))
    t = torch.arange(cap, device=table.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    inside = b < B
    b = b.clamp(max=B - 1)
    pos = cached[b] + t - cu[b]
    page = (pos // bs).clamp(max=table.shape[1] - 1)
    slots = torch.where(inside, table[b, page].long() * bs + pos % bs, -1)
    counts = torch.stack([need.sum(), cu[-1]]).int()
    return dict(table=table, slots=slots, positions=torch.where(inside, pos, 0).int(), cu=cu.int(),
                lens=(cached + new).int(), counts=counts)


def _plain_rotary(s):
    pos, rot = s["pos"].double(), s["rot"]
    angle = pos[s["axis"]].movedim(0, -1) * s["freq"]  # [(B,) N, rot/2], far positions: 64 bits
    c, sn = angle.cos(), angle.sin()
    c, sn = c.float(), (-sn if s["inverse"] else sn).float()
    where = 1  # heads: [N, H, d] or [B, H, N, d]
    c, sn = c.unsqueeze(where), sn.unsqueeze(where)

    def turn(x):
        y = x.float()
        if s["interleaved"]:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            z = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
        else:
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            z = torch.cat([a * c - b * sn, b * c + a * sn], -1)
        return torch.cat([z, y[..., rot:]], -1).to(x.dtype)

    return dict(q=turn(s["q"]), k=turn(s["k"]))


def _plain_cache(s):
    bs, Hk = s["bs"], s["Hk"]
    w, r = s["write"], s["read"]
    h = torch.arange(Hk, device=w.device)[None]
    got = {}
    for name, x, codes, scales in (("k", s["k"], s["cache"][0], s["cache"][1]),
                                   ("v", s["v"], s["cache"][2], s["cache"][3])):
        c, f = _quantise(x)
        at = (w // bs)[:, None], h, (w % bs)[:, None]
        codes[at], scales[at] = c, f
        at = (r // bs)[:, None], h, (r % bs)[:, None]
        got[name] = _values(codes[at], scales[at]).to(x.dtype)
    return got


def _plain_attn(s):
    B, nq, Hq, Hk, d, bs = (s[k] for k in ("B", "nq", "Hq", "Hk", "d", "bs"))
    kc, ks, vc, vs = s["cache"]
    page = s["table"].clamp(min=0).long()

    def rows(codes, scales):  # [B, Hk, tokens, d]
        x = _values(codes[page], scales[page])  # [B, pages, Hk, bs, d]
        return x.transpose(1, 2).flatten(2, 3)[:, :, :s["k_max"]]

    K, V = rows(kc, ks), rows(vc, vs)
    q = s["q"].float().view(B, nq, Hk, Hq // Hk, d).permute(0, 2, 3, 1, 4).flatten(2, 3)
    S = (q @ K.transpose(-1, -2)) * d ** -0.5  # [B, Hk, g * nq, tokens]
    S = S.unflatten(2, (Hq // Hk, nq))
    lens = s["lens"].long()
    last = lens[:, None] - nq + torch.arange(nq, device=q.device)  # a query sees keys <= last
    j = torch.arange(S.shape[-1], device=q.device)
    seen = (j <= last[..., None]) & (j < lens[:, None, None])
    S = S.masked_fill(~seen[:, None, None], -math.inf)
    m = S.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    P = (S - m).exp()
    l = P.sum(-1, keepdim=True)
    O = (P.flatten(2, 3) @ V).unflatten(2, (Hq // Hk, nq))
    O = torch.where(l > 0, O / l, 0.0)
    lse = (l.log() + m).squeeze(-1)
    return dict(o=O.permute(0, 3, 1, 2, 4).reshape(B * nq, Hq, d).to(s["q"].dtype),
                lse=lse.permute(1, 2, 0, 3).reshape(Hq, B * nq))


# ------------------------------------------------------- the library's calls
def _own(s):
    from exact_attention_57_gb300 import fa
    if s["op"] == "plan":
        slots, positions, cu, lens, counts = fa.kv_plan(
            s["cached"], s["new"], s["free"], s["table"], s["bs"], s["cap"], out=s["out"])
        return dict(table=s["table"], slots=slots, positions=positions, cu=cu, lens=lens,
                    counts=counts)
    if s["op"] == "rotary":
        turn = fa.rotary_backward if s["inverse"] else fa.rotary
        q, k = turn(s["q"], s["k"], s["pos"], s["table"], interleaved=s["interleaved"])
        return dict(q=q, k=k)
    if s["op"] == "cache":
        fa.kv4_append(s["k"], s["v"], s["write"], *s["cache"])
        k, v = fa.kv4_gather(s["read"], *s["cache"], dtype=s["k"].dtype, out=s["out"])
        return dict(k=k, v=v)
    o, lse = fa.attention_kv4(s["q"], *s["cache"], s["table"], s["lens"], s["k_max"],
                              cu_seqlens_q=s["cu"], max_seqlen_q=s["nq"], causal=True,
                              out=s["out"], lse=s["lse"])
    return dict(o=o, lse=lse)


def run(state):
    if own:
        return _own(state)
    return {"plan": _plain_plan, "rotary": _plain_rotary, "cache": _plain_cache,
            "attn": _plain_attn}[state["op"]](state)


# ------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op == "plan":
        B, bs = case["B"], case["bs"]
        new = sum(_lens(B, case["new"], 1 if case["new"] == 1 else 0))
        # lengths in, offsets and lengths out, a slot and a position a token,
        # a block of the list read and an entry of the table written for each new block
        return {"bytes": 16 * B + 12 * case["cap"] + 8 * (new // bs), "flops": 0}
    es = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
    if op == "rotary":
        rows = case["B"] * case["N"]
        n = rows * (case["Hq"] + case["Hk"])
        return {"bytes": 2 * n * case["d"] * es + 4 * case["axes"] * rows + 4 * case["rot"],
                "flops": 3 * n * case["rot"]}
    if op == "cache":
        row = case["Hk"] * case["d"]
        return {"bytes": 2 * row * (case["T"] * (es + 0.5625) + case["R"] * (es + 0.5625))
                + 8 * (case["T"] + case["R"]), "flops": 2 * row * (3 * case["T"] + case["R"])}
    nq, Hq, Hk, d = case["nq"], case["Hq"], case["Hk"], case["d"]
    lens = _k_lens(case)
    pairs = sum(nq * (n - nq) + nq * (nq + 1) // 2 for n in lens)
    kv = sum(lens) * Hk * d * 2 * 0.5625
    return {"bytes": kv + case["B"] * nq * Hq * (2 * d * es + 4)
            + 4 * sum(-(-n // case["bs"]) for n in lens), "flops": 4 * pairs * Hq * d}


# ------------------------------------------------------------------ exact
def _exact_tables():
    """float64 values of the 16 e2m1 codes and the 256 e4m3 ones, from their
    bits (made on the host, where a power of two is exact)."""
    code = [(0.5 * (n % 2) if n // 2 % 4 == 0 else math.ldexp(1 + 0.5 * (n % 2), n // 2 % 4 - 1))
            * (-1 if n >= 8 else 1) for n in range(16)]
    scale = [(math.ldexp(n % 8, -9) if n // 8 % 16 == 0 else math.ldexp(8 + n % 8, n // 8 % 16 - 10))
             * (-1 if n >= 128 else 1) for n in range(256)]
    return tuple(torch.tensor(t, dtype=torch.float64, device="cuda") for t in (code, scale))


def _exact_values(codes, scales):
    code, scale = _exact_tables()
    n = torch.empty(codes.shape[:-1] + (codes.shape[-1] * 2,), dtype=torch.int64, device=codes.device)
    n[..., 0::2] = codes.long() % 16
    n[..., 1::2] = codes.long() // 16
    return code[n] * scale[scales.long()].repeat_interleave(16, -1)


def _exact_attn(s):
    B, nq, Hq, Hk, d, bs = (s[k] for k in ("B", "nq", "Hq", "Hk", "d", "bs"))
    G = Hq // Hk
    O = torch.zeros(B * nq, Hq, d, dtype=torch.float64, device="cuda")
    L = torch.full((Hq, B * nq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        ids = s["table"][b, :-(-n // bs)].long()
        for h in range(Hk):
            K, V = (_exact_values(c[ids, h].flatten(0, 1)[:n], f[ids, h].flatten(0, 1)[:n])
                    for c, f in (s["cache"][:2], s["cache"][2:]))
            for x in range(h * G, h * G + G):
                S = s["q"][b * nq:b * nq + nq, x].double() @ K.T / math.sqrt(d)
                if nq > 1:
                    hide = torch.ones(nq, n, dtype=torch.bool, device="cuda").triu(n - nq + 1)
                    S[hide] = -math.inf
                lse = S.logsumexp(-1)
                w = (S - lse[:, None]).exp()
                O[b * nq:b * nq + nq, x] = torch.where(lse[:, None] > -math.inf, w @ V, 0.0)
                L[x, b * nq:b * nq + nq] = lse
    return dict(o=O, lse=L)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None  # whole numbers
    if case["op"] == "attn":
        return _exact_attn(s)
    if case["op"] == "rotary":
        rot = s["rot"]
        turn = s["pos"].double()[s["axis"]].movedim(0, -1) * s["freq"]
        z = torch.polar(torch.ones_like(turn), -turn if s["inverse"] else turn).unsqueeze(1)
        got = {}
        for name in ("q", "k"):
            x = s[name].double().clone()
            if s["interleaved"]:
                y = torch.view_as_complex(x[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * z
                x[..., :rot] = torch.view_as_real(y).flatten(-2)
            else:
                y = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * z
                x[..., :rot // 2], x[..., rot // 2:rot] = y.real, y.imag
            got[name] = x
        return got
    # cache: the nearest of the code's values, found by distance
    grid, f8 = _exact_tables()
    grid, f8 = grid[:8], f8[:127]

    def nearest(y, values):  # the even index where two are as near
        hi = torch.searchsorted(values, y.contiguous()).clamp(1, values.numel() - 1)
        lo = hi - 1
        dl, dh = y - values[lo], values[hi] - y
        return values[torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)]

    got = {}
    for name, x, (codes, scales) in (("k", s["k"], s["cache"][:2]), ("v", s["v"], s["cache"][2:])):
        y = x.double().unflatten(-1, (-1, 16))
        f = nearest((y.abs().amax(-1) / 6).clamp(max=448.0), f8).unsqueeze(-1)
        unit = torch.where(f > 0, y.abs() / f, 0.0)
        new = (nearest(unit.clamp(max=6.0), grid) * f * y.sign()).flatten(-2)
        r = s["read"]
        at = (r // s["bs"])[:, None], torch.arange(s["Hk"], device="cuda")[None], (r % s["bs"])[:, None]
        rows = _exact_values(codes[at], scales[at])
        rows[s["R"] - s["T"]:] = new
        got[name] = rows
    return got
