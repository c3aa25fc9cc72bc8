"""Plain float64 attention, the oracle of the attention operators: one sequence at a time, every
score formed, from the formula

    out[t, h] = sum_j softmax_j(scale * q[t, h] . k[j, h']) v[j, h'],   j < keys(t),
    lse[t, h] = ln sum_j exp(scale * q[t, h] . k[j, h'])

with h' = h // (heads / kv_heads). Arrays are float64; a row that sees no key is zero, lse -inf.
"""
from __future__ import annotations

import numpy as np


def attend(q, k, v, scale: float):
    """q [n, H, D], k and v [m, Hk, D]: token t of n sees the first m - n + t + 1 keys.

    Returns out [n, H, D], lse [n, H], and what the error bounds need: mass = sum_j w_j |v_j|
    [n, H, D], dot = the largest scale * sum_d |q_d k_d| over the row's keys [n, H], and vsum =
    sum_j |v_j| over the row's keys [n, H, D].
    """
    n, H, D = q.shape
    m, Hk, _ = k.shape
    out = np.zeros((n, H, D))
    lse = np.full((n, H), -np.inf)
    mass, vsum = np.zeros((n, H, D)), np.zeros((n, H, D))
    dot = np.zeros((n, H))
    seen = np.arange(m)[None, :] <= (m - n + np.arange(n))[:, None]
    any_seen = seen.any(1)
    if m == 0 or not any_seen.any():
        return out, lse, mass, dot, vsum
    for h in range(H):
        c = h // (H // Hk)
        s = scale * (q[:, h] @ k[:, c].T)
        s = np.where(seen, s, -np.inf)
        top = np.where(any_seen, s.max(1), 0.0)
        e = np.exp(s - top[:, None])
        total = np.where(any_seen, e.sum(1), 1.0)
        w = e / total[:, None]
        out[:, h] = w @ v[:, c]
        lse[:, h] = np.where(any_seen, top + np.log(total), -np.inf)
        mass[:, h] = w @ np.abs(v[:, c])
        dot[:, h] = np.where(seen, scale * (np.abs(q[:, h]) @ np.abs(k[:, c]).T), 0.0).max(1)
        vsum[:, h] = seen @ np.abs(v[:, c])
    return out, lse, mass, dot, vsum
