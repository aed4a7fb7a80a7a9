"""fp64 / whole-number oracles of the operators on packed requests (test infrastructure).

``gdn``: the gated delta rule token by token.  ``tables``: block table, slots and offsets with
Python integers.  ``hold``: the value a 4-bit cache keeps for each element, by search over the
formats' own values.  ``attend``: causal grouped-query attention in fp64, row by row.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# every finite e4m3 value >= 0, in code order (exponent bias 7, 3 mantissa bits, 0x7f is NaN)
E4M3 = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)])


def gdn(q, k, v, alpha, beta, cu, S0=None):
    """Outputs [tokens, H, P] (NaN where no request owns the row) and states [B, H, P, N]."""
    T, H, N = q.shape
    P, B = v.shape[2], len(cu) - 1
    y = np.full((T, H, P), np.nan)
    S = np.zeros((B, H, P, N)) if S0 is None else np.array(S0, np.float64)
    for b in range(B):
        for t in range(cu[b], cu[b + 1]):
            X = S[b] * alpha[t][:, None, None]
            u = beta[t][:, None] * (v[t] - np.einsum("hpn,hn->hp", X, k[t]))
            S[b] = X + u[:, :, None] * k[t][:, None, :]
            y[t] = np.einsum("hpn,hn->hp", S[b], q[t])
    return y, S


def tables(cached, new, free, head, table, ps, max_tokens):
    """(table, cu, seq_len, slots, positions, next head), or None where the step is refused."""
    table = [list(r) for r in table]
    cu, slots, pos = [0], [], []
    for b, (c, n) in enumerate(zip(cached, new)):
        if c < 0 or n < 0 or c + n > len(table[b]) * ps:
            return None
        cu.append(cu[-1] + n)
        for p in range(-(-c // ps), -(-(c + n) // ps)):
            if head < 0 or head >= len(free):
                return None
            table[b][p] = free[head]
            head += 1
        for p in range(c, c + n):
            page = table[b][p // ps]
            slots.append(page * ps + p % ps if page >= 0 else -1)
            pos.append(p)
    if cu[-1] > max_tokens:
        return None
    pad = [-1] * (max_tokens - cu[-1])
    return table, cu, [c + n for c, n in zip(cached, new)], slots + pad, pos + pad, head


def nearest(x, values):
    """Index of the value nearest to each x >= 0, a tie going to the even index, past the end to the last."""
    hi = np.searchsorted(values, x).clip(1, len(values) - 1)
    lo = hi - 1
    dl, dh = x - values[lo], values[hi] - x
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def hold(x, scale):
    """Values kept for finite x [..., D] (float64 holding bf16 numbers): 16-channel blocks, e4m3 scale, e2m1 codes."""
    b = (np.asarray(x, np.float64) / scale).reshape(*x.shape[:-1], -1, 16)
    s = E4M3[nearest(np.abs(b).max(-1, keepdims=True) / 6, E4M3)]
    r = np.divide(np.abs(b), s, out=np.zeros_like(b), where=s > 0)
    return (np.sign(b) * E2M1[nearest(r, E2M1)] * s * scale).reshape(x.shape)


def attend(q, K, V, cu, scale):
    """q [tokens, Hq, D], K and V lists of [len_b, Hk, D]: outputs, and per row and head the sums that error bounds
    are made of: sum_j p_j |v_j|, the largest scale * sum_d |q_d k_jd| of a visible token, and sum_j |v_j|."""
    T, Hq, D = q.shape
    out, mean, big, flat = np.full((T, Hq, D), np.nan), np.zeros((T, Hq, D)), np.zeros((T, Hq)), np.zeros((T, Hq, D))
    for b in range(len(cu) - 1):
        n, L = cu[b + 1] - cu[b], len(K[b])
        for i in range(n):
            seen = L - n + i + 1
            for h in range(Hq):
                o = out[cu[b] + i, h]
                if seen <= 0:
                    o[:] = 0
                    continue
                j = h // (Hq // K[b].shape[1])
                qk = K[b][:seen, j] * q[cu[b] + i, h]
                s = scale * qk.sum(1)
                p = np.exp(s - s.max())
                p /= p.sum()
                o[:] = p @ V[b][:seen, j]
                mean[cu[b] + i, h] = p @ np.abs(V[b][:seen, j])
                big[cu[b] + i, h] = scale * np.abs(qk).sum(1).max()
                flat[cu[b] + i, h] = np.abs(V[b][:seen, j]).sum(0)
    return out, mean, big, flat
