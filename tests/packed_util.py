"""Inputs and bounds of the tests of packed sequences.

Bounds, before any run.  A logit is a sum of d products of bf16 values in fp32: d additions and the scaling, each off by
at most 2^-23 of the sum of the terms' sizes (`logit`): dS = (d + 8) 2^-23 logit.  L is off by dS, and by the rounding of
fp32 exponentials, logarithm and sums: 2^-20 (1 + |L|).  The weights of O are rounded to bf16 (2^-8 each, and their sum
with them), and follow the logits (2 dS): O is off by 2 (2^-8 + dS) of sum w |v|, and by its own rounding 2^-8 |O|; 2^-16 of
the same for fp32 sums and exponentials.
"""

import math

import numpy as np

from gpu_util import host, torch_cuda


def starts(lengths):
    return [0, *np.cumsum(lengths).tolist()]


def make(lq, lk, H, Hkv, d, seed, pad=0, strong=True):
    """q [Tq, H, d], k, v [Tk, Hkv, d] bf16 on the device; `pad` rows behind the last sequence."""
    torch = torch_cuda()
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(sum(lq) + pad, H, d, generator=g)
    k = torch.randn(sum(lk) + pad, Hkv, d, generator=g)
    v = torch.randn(sum(lk) + pad, Hkv, d, generator=g)
    if strong:
        k = k * (1.0 + 2.0 * (torch.rand(d, generator=g) < 0.1))
    return [x.to(torch.bfloat16).cuda() for x in (q, k, v)]


def i32(values):
    torch = torch_cuda()
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def check_forward(o, lse, want, d, rows=None):
    """o [Tq, H, d], lse [H, Tq] against the oracle's dict, over the rows of sequences (a list of indices)."""
    rows = slice(None) if rows is None else rows
    ds = (d + 8) * 2.0 ** -23 * want["logit"]
    L, got = want["lse"][:, rows], lse.double().cpu().numpy()[:, rows]
    empty = np.isneginf(L)
    assert np.array_equal(np.isneginf(got), empty)
    over = np.where(empty, 0.0, np.abs(np.where(empty, 0, got) - np.where(empty, 0, L))
                    - ds[:, rows] - 2.0 ** -20 * (1 + np.abs(np.where(empty, 0, L))))
    assert over.size == 0 or float(over.max()) <= 0.0, f"L off by {float(over.max()):.3e} more than its bound"
    O, got = want["o"][rows], host(o)[rows]
    bound = (2.0 ** -8 * (1 + 2.0 ** -8) * np.abs(O)
             + (2 * (2.0 ** -8 + ds.T[rows][..., None]) + 2.0 ** -16) * want["mass"][rows])
    over = np.abs(got - O) - bound
    bad = ~(over <= 1e-30)
    assert not bad.any(), f"O off by {np.nanmax(np.abs(got - O)):.3e}, {int(bad.sum())} beyond bound or not finite"


def scale_of(d):
    return 1.0 / math.sqrt(d)
