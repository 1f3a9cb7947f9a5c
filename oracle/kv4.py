"""Definition of the 4-bit KV cache, in numpy: groups of 32 channels with step = bf16(max |x| / 7) and codes
clamp(round_half_even(x / step), -7, 7) + 8, standing for step * (code - 8); a group holding an infinity or NaN has
step NaN.  In a stored row, unit u of group g (8 channels for K, 4 for V) sits at unit position u * (d / 32) + g,
its first channel in its lowest nibble.

Quotients are formed in float64: x and step have 8 significant bits each, so a quotient is a tie exactly or at least
2^-10 away from one, and float64 rounds it the right way.
"""
from __future__ import annotations

import numpy as np

GROUP = 32
UNIT = {"k": 8, "v": 4}


def bf16_bits(x) -> np.ndarray:
    """Float64 (or float32) -> bf16 bit patterns, rounding half to even (finite values; NaN -> 0x7fff)."""
    f = np.asarray(x, np.float32)
    u = f.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(f), np.uint16(0x7FFF), r)


def bf16_value(bits) -> np.ndarray:
    return (np.asarray(bits, np.uint32) << 16).view(np.float32).astype(np.float64)


def quantise(x):
    """Float64 array of bf16 values [..., d] -> (codes uint8 [..., d], one a channel; steps bf16 bits [..., d / 32])."""
    x = np.asarray(x, np.float64)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    amax = np.abs(g).max(axis=-1)   # NaN wins
    bad = ~np.isfinite(amax)
    q = np.where(bad, 0.0, amax) / 7
    # float64 -> bf16 directly: amax / 7 is never so near a bf16 tie that passing through float32 matters
    steps = np.where(bad, np.uint16(0x7FFF), bf16_bits(q))
    s = np.where(bad, 0.0, bf16_value(steps))[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        n = np.where(s > 0, np.rint(g / s), 0.0)
    n = np.where(bad[..., None], 0.0, np.clip(n, -7, 7))
    return (n + 8).astype(np.uint8).reshape(x.shape), steps.astype(np.uint16)


def values(codes, steps):
    """What codes (one a channel) and step bits stand for, float64."""
    c = codes.astype(np.float64).reshape(*codes.shape[:-1], -1, GROUP) - 8
    return (c * bf16_value(steps)[..., None]).reshape(codes.shape)


def _position(d, unit):
    pos = np.empty(d, np.int64)
    for ch in range(d):
        g, c = divmod(ch, GROUP)
        u, i = divmod(c, unit)
        pos[ch] = (u * (d // GROUP) + g) * unit + i
    return pos


def pack(codes, which):
    """Codes [..., d] -> stored bytes [..., d / 2] of a K ("k") or V ("v") row."""
    d = codes.shape[-1]
    nib = np.zeros_like(codes)
    nib[..., _position(d, UNIT[which])] = codes
    return nib[..., 0::2] | (nib[..., 1::2] << 4)


def unpack(stored, which):
    d = 2 * stored.shape[-1]
    nib = np.stack((stored & 15, stored >> 4), axis=-1).reshape(*stored.shape[:-1], d)
    return nib[..., _position(d, UNIT[which])]


def decode(q, k_codes, k_steps, v_codes, v_steps, lengths, window, sinks, scale):
    """Single-token attention over a cache given as codes (one a channel) and step bits; q [B, H, d] float64.  Dict of
    o, lse and bounds: weights times steps rounded once to fp16 (2^-11 relative; absolutely, where a product is small, half
    a subnormal step 2^-25 in units of which the largest product of the head and group has 2^3 or more, for codes up to
    7: below 2^-25 of that product a key), fp32 sums, the output rounded to bf16 (2^-8).  A group's bound holds nothing
    of other groups, and the LSE's nothing of V."""
    from . import windowed as W
    k, v = values(k_codes, k_steps), values(v_codes, v_steps)
    B, H, d = q.shape
    G = H // k.shape[1]
    r = {"o": np.zeros_like(q), "lse": np.full((B, H), -np.inf), "o_bound": np.zeros_like(q), "lse_bound": np.zeros((B, H))}
    for b in range(B):
        L = int(lengths[b])
        idx = np.nonzero(W.visible(1, L, window, sinks)[0])[0] if L else np.zeros(0, int)
        if idx.size == 0:
            continue
        for h in range(H):
            K, V = k[b, h // G, idx], v[b, h // G, idx]
            ks, vs = (bf16_value(s[b, h // G, idx]) for s in (k_steps, v_steps))
            s = scale * K @ q[b, h]
            m = s.max()
            p = np.exp(s - m)
            r["lse"][b, h] = m + np.log(p.sum())
            p /= p.sum()
            o = p @ V
            rep = lambda x: np.repeat(x, GROUP, axis=-1)  # noqa: E731
            terms = rep(p @ vs)
            largest = rep((p[:, None] * vs).max(axis=0))
            r["o"][b, h] = o
            r["o_bound"][b, h] = 2.0 ** -8 * np.abs(o) + 2.0 ** -10 * (p @ np.abs(V)) + 2.0 ** -12 * 8 * terms + \
                idx.size * 2.0 ** -25 * largest
            size = scale * (ks @ np.abs(q[b, h]).reshape(-1, GROUP).sum(1) * 15).max()
            r["lse_bound"][b, h] = 2.0 ** -19 * (1 + size + abs(r["lse"][b, h]))
    return r
