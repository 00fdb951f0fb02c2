"""Plain 64-bit forms of the rotary positions and of the 8-bit cache, for the tests (numpy,
written from the formulas, nothing of the library's)."""
from __future__ import annotations

import numpy as np

ZERO_PAGE_EXP = -160


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes."""
    out = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v = np.nan if (e, m) == (15, 7) else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        out[c] = -v if s else v
    return out


VALUES = e4m3_values()


def round_e4m3(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value, ties to the even code, saturating; NaN stays."""
    a = np.minimum(np.abs(x), 448.0)
    with np.errstate(divide="ignore", invalid="ignore"):
        step = 2.0 ** (np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6) - 3)
    return np.copysign(np.rint(a / step) * step, x)


def need_exp(amax: float) -> int:
    if amax == 0:
        return ZERO_PAGE_EXP
    if np.isinf(amax):
        return 0
    m, x = np.frexp(amax)
    return int(x) - (9 if m <= 0.875 else 8)


def turn(x, pos, inv_freq, axis, pairing, sign=1.0):
    """x [..., n, d] fp64 turned by pos [n, axes]; angles in extended precision."""
    n2 = len(inv_freq)
    theta = np.stack([pos[:, a].astype(np.longdouble) * np.longdouble(f) for f, a in zip(inv_freq, axis)], -1) * sign
    c, s = np.cos(theta).astype(np.float64), np.sin(theta).astype(np.float64)
    y = np.array(x, dtype=np.float64)
    ia, ib = (np.arange(n2) * 2, np.arange(n2) * 2 + 1) if pairing == "interleaved" else (np.arange(n2), np.arange(n2) + n2)
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y


def partner_size(x, n2, pairing):
    """|x_a| + |x_b| of the pair each channel is in (|x| of the channels that pass)."""
    y = np.abs(np.array(x, dtype=np.float64))
    ia, ib = (np.arange(n2) * 2, np.arange(n2) * 2 + 1) if pairing == "interleaved" else (np.arange(n2), np.arange(n2) + n2)
    y[..., ia] = y[..., ib] = np.abs(x[..., ia]) + np.abs(x[..., ib])
    return y


def append(pool, table, start, new, K, V):
    """pool: [values/codes as fp64 values in code units, exponents] for K and V (changed in
    place; code units are kept unrounded for the new tokens).  K, V fp64 [B, H, T, d]."""
    block = pool[0][0].shape[2]
    for X, (codes, exps) in ((K, pool[0]), (V, pool[1])):
        for b in range(X.shape[0]):
            t = 0
            while t < new[b]:
                pg, slot = divmod(int(start[b]) + t, block)
                page = int(table[b, pg])
                n = min(block - slot, int(new[b]) - t)
                for h in range(X.shape[1]):
                    part = X[b, h, t: t + n]
                    fin = np.abs(part[~np.isnan(part)])
                    need = need_exp(fin.max() if fin.size else 0.0)
                    e = max(need, int(exps[page, h])) if slot else need
                    if slot and e > exps[page, h]:
                        codes[page, h, :slot] = round_e4m3(codes[page, h, :slot] * 2.0 ** (int(exps[page, h]) - e))
                    codes[page, h, slot: slot + n] = part * 2.0 ** -e
                    exps[page, h] = e
                t += n


def attend(Q, kv, ke, vv, ve, table, lens, new, causal):
    """Q fp64 [B, Hq, M, d]; kv, vv fp64 code values [P, H, block, d].  Returns O, LSE (rows behind
    new[b] are zeros), and per element sum P|v|, per row the largest sum |q||k| / sqrt(d)."""
    B, Hq, M, d = Q.shape
    H, block = kv.shape[1], kv.shape[2]
    O, A = np.zeros(Q.shape), np.zeros(Q.shape)
    LSE, S = np.zeros((B, Hq, M)), np.zeros((B, Hq, M))
    for b in range(B):
        L = int(lens[b])
        ids = table[b, : -(-L // block)].astype(int)
        for h in range(H):
            k = (kv[ids, h] * 2.0 ** ke[ids, h].astype(float)[:, None, None]).reshape(-1, d)[:L]
            v = (vv[ids, h] * 2.0 ** ve[ids, h].astype(float)[:, None, None]).reshape(-1, d)[:L]
            for hq in range(h * Hq // H, (h + 1) * Hq // H):
                for m in range(int(new[b])):
                    n = min(max(L - int(new[b]) + m + 1, 0), L) if causal else L
                    if n == 0:
                        LSE[b, hq, m] = -np.inf
                        continue
                    s = k[:n] @ Q[b, hq, m] / np.sqrt(d)
                    mx = s.max()
                    p = np.exp(s - mx)
                    LSE[b, hq, m] = mx + np.log(p.sum())
                    p /= p.sum()
                    O[b, hq, m] = p @ v[:n]
                    A[b, hq, m] = p @ np.abs(v[:n])
                    S[b, hq, m] = (np.abs(k[:n]) @ np.abs(Q[b, hq, m])).max() / np.sqrt(d)
    return O, LSE, A, S
