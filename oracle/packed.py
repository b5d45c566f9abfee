"""Attention over packed sequences in fp64 on the CPU, sequence by sequence and head by head.

Beside O and L (and the gradients) come the sizes that bound the rounding of an implementation with bf16 weights:
``mass`` = sum_j w_j |v_j| (the weighted magnitude behind each element of O) and ``logit`` = the largest
scale * sum_c |q_c k_c| that a row sees.
"""

import numpy as np


def visible(nq, nk, causal):
    """[nq, nk] truth values; causal "none", "top_left" or "bottom_right"."""
    if causal == "none":
        return np.ones((nq, nk), dtype=bool)
    off = nk - nq if causal == "bottom_right" else 0
    return np.arange(nk)[None] <= np.arange(nq)[:, None] + off


def forward(q, k, v, cu_q, cu_k, scale, causal, used=None, prefix=None):
    """q [Tq, H, d], k, v [Tk, Hkv, d], prefix (k, v) [P, Hkv, d] or None -> dict of o, lse [H, Tq], mass, logit [H, Tq];
    rows of no sequence are 0 (lse -inf)."""
    Tq, H, d = q.shape
    G = H // k.shape[1]
    out = {"o": np.zeros((Tq, H, d)), "mass": np.zeros((Tq, H, d)), "lse": np.full((H, Tq), -np.inf),
           "logit": np.zeros((H, Tq))}
    for b in range(len(cu_q) - 1):
        rows = slice(cu_q[b], cu_q[b + 1])
        nq, nk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        if used is not None:
            nk = used[b]
        seen = visible(nq, nk, causal)
        if prefix is not None:
            seen = np.concatenate([np.ones((nq, prefix[0].shape[0]), dtype=bool), seen], 1)
        for h in range(H):
            kk, vv = (x[cu_k[b]:cu_k[b] + nk, h // G] for x in (k, v))
            if prefix is not None:
                kk, vv = (np.concatenate([x[:, h // G], y]) for x, y in zip(prefix, (kk, vv)))
            s = np.where(seen, scale * (q[rows, h] @ kk.T), -np.inf)
            if s.size == 0:
                continue
            top = s.max(1, keepdims=True)
            w = np.exp(s - np.where(np.isfinite(top), top, 0.0))
            total = w.sum(1, keepdims=True)
            w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
            out["o"][rows, h] = w @ vv
            out["mass"][rows, h] = w @ np.abs(vv)
            with np.errstate(divide="ignore"):
                out["lse"][h, rows] = (np.log(total) + np.where(np.isfinite(top), top, 0.0))[:, 0]
            out["logit"][h, rows] = np.where(seen, scale * (np.abs(q[rows, h]) @ np.abs(kk).T), 0.0).max(1)
    return out


def backward(q, k, v, dout, cu_q, cu_k, scale, causal):
    """Gradients in fp64, and for each what bounds its rounding in an implementation that rounds the weights and dS to bf16
    (u = 2^-8) and takes D from an O of its own in bf16: dict of dq, dk, dv and dq_bound, dk_bound, dv_bound."""
    Tq, H, d = q.shape
    G = H // k.shape[1]
    out = {n: np.zeros(x.shape) for n, x in (("dq", q), ("dk", k), ("dv", v))}
    bound = {n: np.zeros(x.shape) for n, x in (("dq", q), ("dk", k), ("dv", v))}
    u = 2.0 ** -8
    for b in range(len(cu_q) - 1):
        rows, cols = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        nq, nk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        if nq == 0 or nk == 0:
            continue
        seen = visible(nq, nk, causal)
        for h in range(H):
            Q, K, V, dO = q[rows, h], k[cols, h // G], v[cols, h // G], dout[rows, h]
            s = np.where(seen, scale * (Q @ K.T), -np.inf)
            top = s.max(1, keepdims=True)
            w = np.exp(s - np.where(np.isfinite(top), top, 0.0))
            total = w.sum(1, keepdims=True)
            P = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
            O = P @ V
            dP = dO @ V.T
            dS = P * (dP - (dO * O).sum(1, keepdims=True))
            out["dq"][rows, h] = scale * (dS @ K)
            out["dk"][cols, h // G] += scale * (dS.T @ Q)
            out["dv"][cols, h // G] += P.T @ dO
            # A logit is off by ds, a weight by eP of itself, then by its rounding.
            logit = np.where(seen, scale * (np.abs(Q) @ np.abs(K).T), 0.0).max(1, keepdims=True)
            ds = (d + 8) * 2.0 ** -23 * logit
            eP = 2 * ds + 2.0 ** -18
            off_O = u * np.abs(O) + 2 * (u + ds + 2.0 ** -16) * (P @ np.abs(V))
            off_D = (np.abs(dO) * (off_O + d * 2.0 ** -23 * np.abs(O))).sum(1, keepdims=True)
            off_dP = (d + 8) * 2.0 ** -23 * (np.abs(dO) @ np.abs(V).T)
            off_S = (u + eP) * np.abs(dS) + (1 + u) * P * (off_D + off_dP)
            sums = 2.0 ** -16  # fp32 sums of up to 2^7 products a step
            bound["dv"][cols, h // G] += ((u + eP + sums) * P).T @ np.abs(dO)
            bound["dk"][cols, h // G] += scale * ((off_S + sums * np.abs(dS)).T @ np.abs(Q))
            bound["dq"][rows, h] = scale * ((off_S + sums * np.abs(dS)) @ np.abs(K))
    for n in bound:
        out[n + "_bound"] = bound[n] * (1 + u) + u * np.abs(out[n]) + 1e-30
    return out
