"""Float64 definition of sliding-window attention with sinks and shared key/value heads, its gradients, and what
rounding may do to a kernel that computes them from bf16 operands.

Query row i sits at position p = i + (Nk - Nq); key j is visible to it iff j <= p and (j > p - window or j < sinks).
Query head h reads key/value head h // (H // Hkv).  Rows that see no key have O = 0, LSE = -inf and no gradient.

Bounds (``*_bound``) count half a rounding step (2^-8 relative for bf16) for every value a kernel may round to
bf16, and SLACK relative for its fp32 arithmetic (products accumulated over at most a few thousand terms of mixed
sign, exp2 to 2^-22, exponents of up to a few tens of units in the last place).
"""
from __future__ import annotations

import numpy as np

HALF = 2.0 ** -8    # half a bf16 step, relative
SLACK = 2.0 ** -11  # fp32 arithmetic, relative to the sums of absolute values


def visible(Nq: int, Nk: int, window: int, sinks: int) -> np.ndarray:
    """Boolean [Nq, Nk]."""
    p = np.arange(Nq)[:, None] + (Nk - Nq)
    j = np.arange(Nk)[None, :]
    return (j <= p) & ((j > p - window) | (j < sinks))


def _weights(q, k, mask, scale):
    """(P [Nq, Nk], LSE [Nq]) of one head."""
    s = np.where(mask, scale * (q @ k.T), -np.inf)
    m = s.max(axis=1, initial=-np.inf)
    live = np.isfinite(m)
    e = np.exp(s - np.where(live, m, 0.0)[:, None])
    l = e.sum(axis=1)
    lse = np.full(m.shape, -np.inf)
    lse[live] = m[live] + np.log(l[live])
    return e / np.where(live, l, 1.0)[:, None], lse


def attention(q, k, v, window, sinks, scale, do=None):
    """Float64 arrays q, do [B, H, Nq, d], k, v [B, Hkv, Nk, d] -> dict with o, lse, their bounds, and with ``do``
    also dq, dk, dv and theirs."""
    B, H, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    G = H // Hkv
    mask = visible(Nq, Nk, window, sinks)
    r = {"o": np.zeros_like(q), "lse": np.zeros(q.shape[:3]), "o_bound": np.zeros_like(q),
         "lse_bound": np.zeros(q.shape[:3])}
    if do is not None:
        for n, like in (("dq", q), ("dk", k), ("dv", v)):
            r[n], r[n + "_bound"] = np.zeros_like(like), np.zeros_like(like)
    for b in range(B):
        for h in range(H):
            g = h // G
            Q, K, V = q[b, h], k[b, g], v[b, g]
            P, lse = _weights(Q, K, mask, scale)
            O = P @ V
            r["o"][b, h], r["lse"][b, h] = O, lse
            # Weights rounded once, normalised by their own rounded sum: the error is a weighted mean of
            # half a step of v - O; then O itself is rounded.
            A = P @ np.abs(V)
            ob = HALF * (A + 2 * np.abs(O)) + SLACK * A
            r["o_bound"][b, h] = ob
            # LSE: fp32 sums; an error of the largest score shifts it by as much (d terms, 2^-24 each).
            size = scale * np.where(mask, np.abs(Q) @ np.abs(K).T, 0.0).max(axis=1, initial=0.0)
            r["lse_bound"][b, h] = (d + 16) * 2.0 ** -24 * (size + np.where(np.isfinite(lse), np.abs(lse), 0.0)) + 2.0 ** -19
            if do is None:
                continue
            dO = do[b, h]
            dP = dO @ V.T
            D = (dO * O).sum(axis=1, keepdims=True)
            dS = P * (dP - D)
            r["dq"][b, h] = scale * dS @ K
            r["dk"][b, g] += scale * dS.T @ Q
            r["dv"][b, g] += P.T @ dO
            # P rounded for dV; dS rounded, from a D of the rounded O, for dQ and dK.
            dD = (np.abs(dO) * ob).sum(axis=1, keepdims=True)
            eS = HALF * np.abs(dS) + P * (dD + SLACK * (np.abs(dO) @ np.abs(V).T + np.abs(D)))
            r["dq_bound"][b, h] = scale * eS @ np.abs(K) + HALF * np.abs(r["dq"][b, h])
            r["dk_bound"][b, g] += scale * eS.T @ np.abs(Q)
            r["dv_bound"][b, g] += (HALF + SLACK) * P.T @ np.abs(dO)
    if do is not None:
        r["dk_bound"] += HALF * np.abs(r["dk"])
        r["dv_bound"] += HALF * np.abs(r["dv"])
    return r


def decode(q, k, v, lengths, window, sinks, scale):
    """Single-token form: q [B, H, d], caches [B, Hkv, Lmax, d]; sequence b's query sits at position
    lengths[b] - 1 (a length of 0 sees nothing).  Same dict as ``attention``, without the query axis."""
    B, H, d = q.shape
    out = None
    for b in range(B):
        L = int(lengths[b])
        r = attention(q[b:b + 1, :, None], k[b:b + 1, :, :L], v[b:b + 1, :, :L], window, sinks, scale)
        r = {n: x[:, :, 0] for n, x in r.items()}
        out = r if out is None else {n: np.concatenate((out[n], r[n])) for n in out}
    return out
