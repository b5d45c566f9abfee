"""CPU oracle of the 4-bit key/value cache: TEST INFRASTRUCTURE ONLY.

A plain restatement, in float64 and byte by byte, of the format that
include/fa.h defines: quantising a group of 32 channels, where a token's
codes and scales lie in a page, writing, reading back, and attention over
the held values (``oracle.attention`` on each sequence).  It shares no code
with the CUDA library.
"""

from __future__ import annotations

import numpy as np

from . import attention as att

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
GROUP = 32
BLOCK = 16
NAN_BITS = 0x7FFF


def to_bf16(x):
    """float64 rounded to bf16 (nearest, ties to even), as float64."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(all="ignore"):
        _, e = np.frexp(np.where(np.isfinite(x), x, 0.0))
        step = np.exp2(np.maximum(e - 8, -133).astype(np.float64))  # 8 significant bits; subnormals share a step
        out = np.where(np.isfinite(x), np.rint(x / step) * step, x)
    return np.where(np.abs(out) > 3.3895313892515355e38, np.copysign(np.inf, out), out)


def bf16_bits(x):
    """Bits of a float64 array that holds bf16 values."""
    return (np.asarray(x, dtype=np.float32).view(np.uint32) >> 16).astype(np.uint16)


def bits_value(b):
    return (np.asarray(b, dtype=np.uint32) << 16).view(np.float32).astype(np.float64)


def quantise(x):
    """x float64 [..., d] (bf16 values) -> codes uint8 [..., d], scale bits
    uint16 [..., d/32]."""
    x = np.asarray(x, dtype=np.float64)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    finite = np.isfinite(g).all(-1)
    a = np.where(np.isfinite(g), np.abs(g), 0.0)
    s = to_bf16(a.max(-1) / 6.0)
    s = np.where(s < 2.0 ** -126, 0.0, s)
    ratio = np.where(s[..., None] > 0, a / np.where(s > 0, s, 1.0)[..., None], 0.0)
    # Nearest level; of two equally near ones the even code.
    dist = np.abs(ratio[..., None] - LEVELS)
    best = dist.min(-1, keepdims=True)
    tied = dist == best
    order = np.where(tied, np.arange(8) % 2, 2)  # even codes first among the tied
    code = order.argmin(-1)
    code = np.where(ratio >= 6.0, 7, code).astype(np.uint8)
    code |= ((g < 0) & (code > 0)).astype(np.uint8) << 3
    code = np.where(finite[..., None], code, 0).astype(np.uint8)
    bits = np.where(finite, bf16_bits(s), NAN_BITS).astype(np.uint16)
    return code.reshape(x.shape), bits


def held(x):
    """The values the cache holds for x, in float64."""
    code, bits = quantise(x)
    return values(code, bits)


def values(code, bits):
    v = LEVELS[code & 7] * np.where(code & 8, -1.0, 1.0)
    with np.errstate(invalid="ignore"):
        g = v.reshape(*v.shape[:-1], v.shape[-1] // GROUP, GROUP) * bits_value(bits)[..., None]
    return g.reshape(v.shape)


def key_place(d, p, c):
    """(byte, shift) of channel c of token p's key in a block."""
    ng = d // GROUP
    g, r = divmod(c, GROUP)
    t, i = divmod(r, 8)
    byte = ((g // 4) * 16 + t * min(ng, 4) + g % 4) * 4 + i // 2
    if d == 256:
        byte ^= 64 * (p & 1)
    return p * (d // 2) + byte, 4 * (i % 2)


def value_place(d, p, c):
    ng = d // GROUP
    g, r = divmod(c, GROUP)
    u, i = divmod(r, 4)
    row = 4 * ((p & 1) + 2 * (p >> 3)) + ((p >> 1) & 3)
    byte = (u * ng + g) * 2 + i // 2
    if d == 128:
        byte ^= 32 * ((row >> 1) & 1)
    if d == 256:
        byte ^= 32 * (row & 3)
    return 8 * d + row * (d // 2) + byte, 4 * (i % 2)


def scale_place(d, p, which, g):
    return 16 * d + (p * 2 * (d // GROUP) + which * (d // GROUP) + g) * 2


def _token(cache, d, page_size, page, head, pos):
    """View of the block bytes that hold a position, and the place in it."""
    at = pos % page_size
    lo = (at // BLOCK) * 18 * d
    return cache[page, head, lo:lo + 18 * d], at % BLOCK


def _places(d):
    """Index arrays of a whole block: key and value (byte, shift) [16, d], scale bytes [16, 2, NG]."""
    k = np.array([[key_place(d, p, c) for c in range(d)] for p in range(BLOCK)])
    v = np.array([[value_place(d, p, c) for c in range(d)] for p in range(BLOCK)])
    s = np.array([[[scale_place(d, p, w, g) for g in range(d // GROUP)] for w in range(2)] for p in range(BLOCK)])
    return k, v, s


def write(cache, table, start, count, k, v, page_size):
    """Writes float64 k, v [B, Hkv, N, d] (bf16 values) into cache uint8
    [pages, Hkv, bytes], in place."""
    B, Hkv, N, d = k.shape
    places = _places(d)
    for b in range(B):
        for i in range(N if count is None else count[b]):
            pos = start[b] + i
            for h in range(Hkv):
                blk, p = _token(cache, d, page_size, table[b][pos // page_size], h, pos)
                for which, x in enumerate((k, v)):
                    code, bits = quantise(x[b, h, i])
                    at = places[which][p]
                    for nib in (0, 4):
                        pick = at[:, 1] == nib
                        blk[at[pick, 0]] = (blk[at[pick, 0]] & (0xF0 if nib == 0 else 0x0F)) | (code[pick] << nib)
                    sb = places[2][p, which]
                    blk[sb] = bits & 0xFF
                    blk[sb + 1] = bits >> 8


def read(cache, table_row, n, page_size, d, first=0):
    """Held keys and values, float64 [Hkv, n, d], of a sequence's positions
    first .. first + n - 1."""
    Hkv = cache.shape[1]
    kp, vp, sp = _places(d)
    out = np.zeros((2, Hkv, n, d))
    for i in range(n):
        pos = first + i
        for h in range(Hkv):
            blk, p = _token(cache, d, page_size, table_row[pos // page_size], h, pos)
            for which, at in enumerate((kp[p], vp[p])):
                code = (blk[at[:, 0]] >> at[:, 1]) & 15
                sb = sp[p, which]
                bits = blk[sb].astype(np.uint16) | (blk[sb + 1].astype(np.uint16) << 8)
                out[which, h, i] = values(code, bits)
    return out[0], out[1]


def canonical(cache, d):
    """The cache's bytes with the sign of zero codes dropped (a zero may carry
    either sign)."""
    blocks = cache.reshape(-1, 18 * d).copy()
    codes = blocks[:, :16 * d]
    low, high = codes & 0x0F, codes & 0xF0
    blocks[:, :16 * d] = np.where(low == 0x08, 0, low) | np.where(high == 0x80, 0, high)
    return blocks


def attend(q, k, v, n, scale, causal):
    """One sequence: q [H, Nq, d], held k, v [Hkv, >= n, d], its length n and
    a causal name -> O [H, Nq, d], L [H, Nq]."""
    H, Nq, d = q.shape
    group = H // k.shape[0]
    o, lse = np.zeros((H, Nq, d)), np.full((H, Nq), -np.inf)
    if n == 0:
        return o, lse
    kk, vv = np.repeat(k[:, :n], group, 0), np.repeat(v[:, :n], group, 0)
    off = 0 if causal == "none" else att.causal_offset(Nq, n, causal)
    o, lse = att.forward(q[None], kk[None], vv[None], scale, causal != "none", offset=off)
    return o[0], lse[0]
