"""Measured cases of the operators over a key/value cache held in 4 bits.

Three operators of serving: ``write`` quantises keys and values into the pages of a cache and reads the written tokens
back, ``read`` reads a stretch of the cache back to bf16, ``attend`` is attention of new query rows over the cache.

The cache is uint8 [num_pages, Hkv, page_size * 9d/8].  Tokens are stored in blocks of 16 (18 d bytes each), channels
in groups of 32 with one bf16 scale: s = bf16(max|x| / 6), zero if that is below 2^-126; a value is a 4-bit e2m1 code
(0, .5, 1, 1.5, 2, 3, 4, 6 and a sign bit) times s.  Within a block, with NG = d / 32 and p the token's place in it:

* keys, bytes [0, 8d): row p of d/2 bytes; the 4-byte word at (grp // 4) * 16 + t * min(NG, 4) + grp % 4 holds channels
  32 grp + 8 t + (0..7), lowest nibble first; at d = 256 the two 64-byte halves of odd rows are exchanged;
* values, bytes [8d, 16d): row 4 * ((p & 1) + 2 * (p >> 3)) + ((p >> 1) & 3) =: r of d/2 bytes; the 2-byte unit at
  g * NG + grp holds channels 32 grp + 4 g + (0..3); the byte's place is exchanged (xor) with 32 * ((r >> 1) & 1) at
  d = 128 and with 32 * (r & 3) at d = 256;
* scales, bytes [16d, 18d): for each p, NG bf16 of the keys, then NG of the values.
"""

import math
import random

import torch

own = False

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
SMALLEST = 2.0 ** -126


# ------------------------------------------------------------------- cases

def _attend(name, B, H, Hkv, Nq, L, d, page, ragged, causal):
    return {"name": name, "op": "attend", "B": B, "H": H, "Hkv": Hkv, "Nq": Nq, "L": L, "d": d, "page": page,
            "ragged": ragged, "causal": causal}


def _move(name, op, B, Hkv, N, start, d, page, ragged):
    return {"name": name, "op": op, "B": B, "Hkv": Hkv, "N": N, "start": start, "d": d, "page": page,
            "ragged": ragged}


def listed():
    return [
        # The first steps of one conversation: nothing but latency.
        _attend("attend_first_steps", 1, 32, 8, 1, 40, 128, 16, False, "none"),
        # The decoding step of the benchmark: 8 sequences of 8192 tokens, four query heads to a key/value head.
        _attend("attend_decode", 8, 32, 8, 1, 8192, 128, 64, False, "bottom_right"),
        # A busy server's batch: 64 sequences of all lengths up to 16384, one slot idle.
        _attend("attend_server", 64, 32, 8, 1, 16384, 128, 64, True, "bottom_right"),
        # A small model without shared heads, pages of 16 tokens.
        _attend("attend_mha_d64", 16, 16, 16, 1, 4096, 64, 16, True, "none"),
        # One long document, an odd number of tokens.
        _attend("attend_long", 1, 32, 8, 1, 131071, 128, 256, False, "bottom_right"),
        # Checking five drafted tokens at once; three query heads to a key/value head.
        _attend("attend_drafts_d96", 9, 12, 4, 5, 6001, 96, 32, True, "bottom_right"),
        # Wide heads.
        _attend("attend_d256", 16, 16, 4, 1, 8192, 256, 64, True, "bottom_right"),
        # Each decoding step's append: one token of each of 64 sequences.
        _move("write_step", "write", 64, 8, 1, 4097, 128, 64, False),
        # Prompts that arrive together.
        _move("write_prompts", "write", 4, 8, 8192, 0, 128, 64, False),
        # Ragged pieces of prompts behind what is cached already, small heads, small pages.
        _move("write_pieces_d64", "write", 24, 16, 1000, 37, 64, 16, True),
        # Reading long histories back, for the prefill of a further chunk by the bf16 kernels.
        _move("read_histories", "read", 2, 8, 32768, 0, 128, 64, False),
        # Reading a few recent tokens back, across page borders.
        _move("read_recent_d96", "read", 3, 4, 100, 1001, 96, 32, True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "write", "read"])
    d = rng.choice([64, 96, 128, 256])
    page = rng.choice([16, 32, 64, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    B = _log(rng, 1, 64)
    ragged = rng.random() < 0.6
    if op == "attend":
        G = rng.randint(1, 8)
        Nq = rng.choice([1, 1, 1, 2, 3, 5, 8])
        while G * Nq > 32:
            Nq = max(1, Nq - 1)
        most = 64 * 8 * 8192 * 128 // (B * Hkv * d)
        L = _log(rng, 1, max(1, min(131072, most)))
        c = _attend("", B, G * Hkv, Hkv, Nq, L, d, page, ragged, rng.choice(["none", "bottom_right", "bottom_right"]))
    else:
        most = 4 * 8 * 8192 * 128 // (B * Hkv * d)
        N = _log(rng, 1, max(1, min(32768, most)))
        c = _move("", op, B, Hkv, N, rng.choice([0, 0, rng.randint(1, 2000)]), d, page, ragged)
    del c["name"]
    return c


def _lengths(case):
    """Lengths of the sequences (attend) or counts of the tokens moved: part of the case, not of the seed."""
    B, most = case["B"], case["L"] if case["op"] == "attend" else case["N"]
    if not case["ragged"]:
        return [most] * B
    r = random.Random(B * 1000003 + most)
    n = [r.randint(1, most) for _ in range(B)]
    n[r.randrange(B)] = most
    if B > 4:
        n[n.index(min(n))] = 0
    return n


def _visible(case):
    """Visible (query row, key) pairs of one head, summed over the batch."""
    Nq = case["Nq"]
    if case["causal"] == "none":
        return sum(Nq * n for n in _lengths(case))
    return sum(max(0, n - Nq + 1 + i) for n in _lengths(case) for i in range(Nq))


def work(case):
    d, Hkv, T = case["d"], case["Hkv"], sum(_lengths(case))
    held = T * Hkv * (9 * d // 8)
    if case["op"] == "attend":
        rows = case["B"] * case["H"] * case["Nq"]
        return {"bytes": held + rows * (4 * d + 4), "flops": 4 * d * case["H"] * _visible(case)}
    # A value costs about eight operations each way; a write is read back, so the held bytes move twice.
    ways = 2 if case["op"] == "write" else 1
    return {"bytes": ways * (held + 4 * d * T * Hkv), "flops": ways * 16 * d * T * Hkv}


# ------------------------------------------------- the format, in plain form

def _layout(d, device):
    """Byte offsets within a 16-token block: of the pair of channels (2c, 2c+1) of the keys and of the values of
    token p, both [16, d/2], and of the scales [16, NG] (keys, values)."""
    ng = d // 32
    p = torch.arange(16, device=device)[:, None]
    c = torch.arange(0, d, 2, device=device)[None, :]
    grp, in_grp = c // 32, c % 32
    k = ((grp // 4) * 16 + (in_grp // 8) * min(ng, 4) + grp % 4) * 4 + (in_grp % 8) // 2
    if d == 256:
        k = k ^ (64 * (p & 1))
    r = 4 * ((p & 1) + 2 * (p >> 3)) + ((p >> 1) & 3)
    v = ((in_grp // 4) * ng + grp) * 2 + (in_grp % 4) // 2
    if d == 128:
        v = v ^ (32 * ((r >> 1) & 1))
    if d == 256:
        v = v ^ (32 * (r & 3))
    s = torch.arange(ng, device=device)[None, :]
    return {"k": p * (d // 2) + k, "v": 8 * d + r * (d // 2) + v, "ks": 8 * d + p * 2 * ng + s,
            "vs": 8 * d + p * 2 * ng + ng + s}  # scales in 2-byte units


def _codes(x, d):
    """4-bit codes [..., d] and bf16 scales [..., NG] of x."""
    g = x.float().reshape(*x.shape[:-1], d // 32, 32)
    top = g.abs().amax(-1)
    s = (top / 6).to(torch.bfloat16).float()
    s = torch.where(s < SMALLEST, torch.zeros_like(s), s)
    q = torch.where(s[..., None] > 0, g.abs() / s[..., None], torch.zeros_like(g))
    # Round to the nearest level, ties to the even code.
    n = ((q > 0.25).to(torch.uint8) + (q >= 0.75) + (q > 1.25) + (q >= 1.75) + (q > 2.5) + (q >= 3.5) + (q > 5.0))
    n = n.to(torch.uint8) | ((g < 0).to(torch.uint8) << 3)
    finite = torch.isfinite(top)
    n = torch.where(finite[..., None], n, torch.zeros_like(n))
    s = torch.where(finite, s, torch.full_like(s, math.nan))
    return n.reshape(x.shape), s.to(torch.bfloat16)


def _place(table, page, pos, b):
    """Page and block within the page of the positions pos of the sequences b, and the place in the block."""
    return table[b, pos // page].long(), (pos % page) // 16, pos % 16


def _store(cache, lay, table, d, page, b, pos, k, v):
    """Writes tokens k, v [R, Hkv, d] to the positions pos [R] of the sequences b [R]."""
    Hkv = k.shape[1]
    at, blk, p = _place(table, page, pos, b)
    base = ((at * Hkv)[:, None] + torch.arange(Hkv, device=k.device)) * (page // 16) + blk[:, None]
    flat, halves = cache.view(-1), cache.view(torch.bfloat16).view(-1)
    for x, codes_at, scales_at in ((k, lay["k"], lay["ks"]), (v, lay["v"], lay["vs"])):
        n, s = _codes(x, d)
        flat[base[..., None] * (18 * d) + codes_at[p][:, None, :]] = n[..., 0::2] | (n[..., 1::2] << 4)
        halves[base[..., None] * (9 * d) + scales_at[p][:, None, :]] = s


def _fetch(blocks, lay, d):
    """fp32 keys and values [..., 16, d] of blocks [..., 18 d]."""
    sign = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device=blocks.device)
    halves = blocks.view(torch.bfloat16)
    out = []
    for codes_at, scales_at in ((lay["k"], lay["ks"]), (lay["v"], lay["vs"])):
        pair = blocks[..., codes_at]
        x = torch.stack([sign[(pair & 15).int()], sign[(pair >> 4).int()]], -1).flatten(-2)
        s = halves[..., scales_at].float()
        out.append((x.view(*x.shape[:-1], d // 32, 32) * s[..., None]).view(x.shape))
    return out


def _gathered(st, positions):
    """fp32 keys and values [B, Hkv, positions, d] of the first positions of every sequence."""
    case, cache = st["case"], st["cache"]
    d, page = case["d"], case["page"]
    pages = -(-positions // page)
    blocks = cache[st["table"][:, :pages].long()].view(case["B"], pages, case["Hkv"], page // 16, 18 * d)
    k, v = _fetch(blocks, st["layout"], d)
    flat = (case["B"], case["Hkv"], pages * page, d)
    return k.transpose(1, 2).reshape(flat), v.transpose(1, 2).reshape(flat)


# ------------------------------------------------------------------ inputs

def _pages(case, tokens, g, device):
    """A block table [B, pages] with every sequence's pages scattered over the cache, and the number of pages."""
    each = -(-max(1, tokens) // case["page"])
    n = case["B"] * each
    order = torch.randperm(n, generator=g, device=device).to(torch.int32)
    return order.view(case["B"], each).contiguous(), n


def _tokens(g, shape, device, keys):
    """Keys with a few strong channels, as rotary keys have; values near normal."""
    x = torch.randn(shape, generator=g, device=device)
    if keys:
        x = x * (1.0 + 3.0 * (torch.rand(shape[-1], generator=g, device=device) < 0.05))
    return x.to(torch.bfloat16)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    d, page, B, Hkv, op = case["d"], case["page"], case["B"], case["Hkv"], case["op"]
    lens = _lengths(case)
    first = 0 if op == "attend" else case["start"]
    table, n = _pages(case, first + max(lens), g, dev)
    cache = torch.zeros((n, Hkv, page * 9 * d // 8), dtype=torch.uint8, device=dev)
    lay = _layout(d, dev)
    st = {"case": case, "cache": cache, "table": table, "layout": lay}
    number = torch.tensor(lens, dtype=torch.int32, device=dev)
    if op != "write":
        # What the cache holds: written in stretches, as prompts and steps filled it.
        for b in range(B):
            for at in range(0, lens[b], 16384):
                m = min(16384, lens[b] - at)
                pos = first + torch.arange(at, at + m, device=dev)
                k, v = (_tokens(g, (m, Hkv, d), dev, keys) for keys in (True, False))
                _store(cache, lay, table, d, page, torch.full_like(pos, b), pos, k, v)
    if op == "attend":
        shape = (B, case["H"], case["Nq"], d)
        st["q"] = torch.randn(shape, generator=g, device=dev).to(torch.bfloat16)
        st["lens"] = number
        st["o"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty(shape[:3], dtype=torch.float32, device=dev)
        return st
    N = case["N"]
    st["start"] = torch.full((B,), first, dtype=torch.int32, device=dev)
    st["count"] = number
    st["k_out"], st["v_out"] = (torch.zeros((B, Hkv, N, d), dtype=torch.bfloat16, device=dev) for _ in range(2))
    if op == "write":
        st["k"], st["v"] = (_tokens(g, (B, Hkv, N, d), dev, keys) for keys in (True, False))
    # The rows that take part, for the plain form: (sequence, row) pairs.
    row = torch.arange(N, device=dev)
    st["rows"] = tuple(t.contiguous() for t in torch.nonzero(row[None, :] < number[:, None], as_tuple=True))
    return st


# ------------------------------------------------------------- the operators

def run(st):
    op = st["case"]["op"]
    if own:
        import exact_attention_92_gb300 as fa

        if op == "attend":
            fa.fa_kv4_fwd(st["q"], st["cache"], st["table"], st["lens"], st["o"], st["lse"],
                          causal=st["case"]["causal"])
            return {"o": st["o"], "lse": st["lse"]}
        if op == "write":
            fa.fa_kv4_write(st["k"], st["v"], st["cache"], st["table"], st["start"], count=st["count"])
        fa.fa_kv4_read(st["cache"], st["table"], st["start"], st["k_out"], st["v_out"], count=st["count"])
        return {"k": st["k_out"], "v": st["v_out"]}
    if op == "attend":
        return _plain_attend(st)
    return _plain_move(st)


def _plain_move(st):
    case, table = st["case"], st["table"]
    d, page, Hkv = case["d"], case["page"], case["Hkv"]
    b, i = st["rows"]
    pos = st["start"][b].long() + i
    if case["op"] == "write":
        k, v = st["k"][b, :, i], st["v"][b, :, i]
        _store(st["cache"], st["layout"], table, d, page, b, pos, k, v)
    at, blk, p = _place(table, page, pos, b)
    base = ((at * Hkv)[:, None] + torch.arange(Hkv, device=at.device)) * (page // 16) + blk[:, None]
    sign = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device=at.device)
    flat, halves = st["cache"].view(-1), st["cache"].view(torch.bfloat16).view(-1)
    lay = st["layout"]
    for out, codes_at, scales_at in ((st["k_out"], lay["k"], lay["ks"]), (st["v_out"], lay["v"], lay["vs"])):
        pair = flat[base[..., None] * (18 * d) + codes_at[p][:, None, :]]
        x = torch.stack([sign[(pair & 15).int()], sign[(pair >> 4).int()]], -1).flatten(-2)
        s = halves[base[..., None] * (9 * d) + scales_at[p][:, None, :]].float()
        out[b, :, i] = (x.view(*x.shape[:-1], d // 32, 32) * s[..., None]).view(x.shape).to(torch.bfloat16)
    return {"k": st["k_out"], "v": st["v_out"]}


def _plain_attend(st):
    case, q, lens = st["case"], st["q"], st["lens"].long()
    B, H, Hkv, Nq, L, d = (case[n] for n in ("B", "H", "Hkv", "Nq", "L", "d"))
    k, v = _gathered(st, L)
    G = H // Hkv
    rows = q.float().view(B, Hkv, G * Nq, d) / math.sqrt(d)
    s = rows @ k.transpose(-1, -2)
    j = torch.arange(k.shape[2], device=q.device)
    i = torch.arange(G * Nq, device=q.device) % Nq
    last = lens[:, None] - 1
    if case["causal"] == "bottom_right":
        last = lens[:, None] - Nq + i[None, :]
    seen = (j[None, None, :] < lens[:, None, None]) & (j[None, None, :] <= last[:, :, None])
    s = s.masked_fill(~seen[:, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    # A block behind the last token may hold anything: it takes no part.
    v = torch.where((j[None, :] < lens[:, None])[:, None, :, None], v, torch.zeros_like(v))
    o = (p @ v) / torch.where(l > 0, l, torch.ones_like(l))
    lse = torch.where(l > 0, m + torch.log(l), torch.full_like(l, -math.inf))
    return {"o": o.to(torch.bfloat16).view(B, H, Nq, d), "lse": lse.view(B, H, Nq)}


# ----------------------------------------------- the definition, in 64 bits

def _exact_values(raw, heads, d):
    """Values in 64 bits of one sequence's pages: raw uint8 [pages, heads, bytes] -> keys, values [heads, tokens, d].
    The block is taken apart by its axes."""
    ng = d // 32
    blocks = raw.transpose(0, 1).reshape(heads, -1, 18 * d)
    halves = blocks[..., 16 * d:].contiguous().view(torch.bfloat16).double().view(heads, -1, 16, 2, ng)
    mag = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device=raw.device) / 2

    def values(pairs, scale):  # pairs [..., 16, ng, 16] bytes in channel order
        n = torch.stack([pairs % 16, pairs // 16], -1).long().flatten(-2)
        x = mag[n % 8] * (1 - 2 * (n // 8)).double()
        return (x * scale[..., None]).reshape(heads, -1, d)

    kb = blocks[..., :8 * d].reshape(heads, -1, 16, d // 2)
    if d == 256:
        kb = kb.view(heads, -1, 8, 2, 2, 64)
        kb = torch.stack([kb[:, :, :, 0], kb[:, :, :, 1].flip(3)], 3).reshape(heads, -1, 16, 128)
    few = min(ng, 4)
    kb = kb.view(heads, -1, 16, ng // few, 4, few, 4).permute(0, 1, 2, 3, 5, 4, 6).reshape(heads, -1, 16, ng, 16)
    # Rows of the values are ordered by (p >> 3, p & 1, (p >> 1) & 3).
    vb = blocks[..., 8 * d:16 * d].reshape(heads, -1, 2, 2, 4, d // 2)
    quarters = []
    for mid in range(4):
        row = vb[:, :, :, :, mid]
        if d >= 128:
            row = row.reshape(*row.shape[:-1], d // 64, 32)
            turn = mid >> 1 if d == 128 else mid
            row = torch.stack([row[..., i ^ turn, :] for i in range(d // 64)], -2).flatten(-2)
        quarters.append(row)
    vb = torch.stack(quarters, 3).reshape(heads, -1, 16, d // 2)  # (p >> 3, (p >> 1) & 3, p & 1) = p
    vb = vb.view(heads, -1, 16, 8, ng, 2).transpose(3, 4).reshape(heads, -1, 16, ng, 16)
    return values(kb, halves[:, :, :, 0]), values(vb, halves[:, :, :, 1])


def _exact_quantised(x):
    """The value in 64 bits that the format holds for x (bf16)."""
    y = x.double().reshape(*x.shape[:-1], -1, 32)
    scale = (y.abs().amax(-1, keepdim=True) / 6).to(torch.bfloat16).double()
    scale = scale * (scale >= SMALLEST)
    level = torch.tensor(LEVELS, dtype=torch.float64, device=x.device)
    ratio = y.abs() / torch.where(scale > 0, scale, torch.ones_like(scale))
    down = (torch.searchsorted(level, ratio.contiguous(), right=True) - 1).clamp(0, 7)
    up = (down + 1).clamp(max=7)
    lo, hi = ratio - level[down], level[up] - ratio
    pick = torch.where((hi < lo) | ((hi == lo) & (down % 2 == 1)), up, down)
    out = torch.where(scale > 0, level[pick] * scale, torch.zeros_like(y)) * torch.where(y < 0, -1.0, 1.0)
    return torch.where(torch.isfinite(y).all(-1, keepdim=True), out, torch.full_like(y, math.nan)).reshape(x.shape)


def exact(case, seed):
    st = prepare(case, seed)
    B, Hkv, d, page, lens = case["B"], case["Hkv"], case["d"], case["page"], _lengths(case)
    if case["op"] == "attend":
        H, Nq = case["H"], case["Nq"]
        o = torch.zeros((B, H, Nq, d), dtype=torch.float64, device="cuda")
        lse = torch.full((B, H, Nq), -math.inf, dtype=torch.float64, device="cuda")
        for b in range(B):
            n = lens[b]
            if n == 0:
                continue
            k, v = _exact_values(st["cache"][st["table"][b, :-(-n // page)].long()], Hkv, d)
            for h in range(H):
                logits = st["q"][b, h].double() @ k[h // (H // Hkv), :n].T * d ** -0.5
                if case["causal"] == "bottom_right":
                    ahead = torch.arange(n, device="cuda")[None] > torch.arange(Nq, device="cuda")[:, None] + n - Nq
                    logits = torch.where(ahead, -math.inf, logits)
                lse[b, h] = torch.logsumexp(logits, -1)
                w = torch.where(torch.isfinite(lse[b, h])[:, None], torch.exp(logits - lse[b, h][:, None]), 0.0)
                o[b, h] = w @ v[h // (H // Hkv), :n]
        return {"o": o, "lse": lse}
    k_out, v_out = (torch.zeros((B, Hkv, case["N"], d), dtype=torch.float64, device="cuda") for _ in range(2))
    for b in range(B):
        n, first = lens[b], case["start"]
        if n == 0:
            continue
        if case["op"] == "write":
            k, v = (_exact_quantised(st[x][b, :, :n]) for x in ("k", "v"))
        else:
            last = -(-(first + n) // page)
            k, v = (x[:, first:first + n] for x in _exact_values(st["cache"][st["table"][b, :last].long()], Hkv, d))
        k_out[b, :, :n], v_out[b, :, :n] = k, v
    return {"k": k_out, "v": v_out}
