"""The products around latent attention and its expanded form in float64 (oracle side)."""
from __future__ import annotations

import numpy as np


def absorb(q, w):
    """q [T, heads, 192], w [heads, 256, 512] -> [T, heads, 576]."""
    return np.concatenate([np.einsum("thd,hdc->thc", q[..., :128], w[:, :128]), q[..., 128:]], -1)


def project(o, w):
    """o [T, heads, 512] -> [T, heads, 128]."""
    return np.einsum("thc,hdc->thd", o, w[:, 128:])


def expand(c, w):
    """c [n, 512] -> keys and values [n, heads, 128]."""
    y = (c @ w.reshape(-1, w.shape[2]).T).reshape(len(c), len(w), 256)
    return y[..., :128], y[..., 128:]


def prefill(q, k, v, k_rope, q_lens, kv_lens, mask, sm_scale):
    """Attention of expanded rows, sequence by sequence.  q [T, heads, 192], k / v
    [N, heads, 128], k_rope [N, 64]; mask "causal", "full" or "cross" (then the rows hold
    kv_lens positions, else kv_lens + q_lens).  Returns out, lse and sum p |v|."""
    T, heads = q.shape[:2]
    out, mag = np.zeros((T, heads, v.shape[2])), np.zeros((T, heads, v.shape[2]))
    lse = np.full((T, heads), -np.inf)
    t = n = 0
    for ql, kv in zip(q_lens, kv_lens):
        held = kv + (0 if mask == "cross" else ql)
        for h in range(heads if held else 0):
            key = np.concatenate([k[n:n + held, h], k_rope[n:n + held]], 1)
            s = sm_scale * q[t:t + ql, h] @ key.T
            if mask == "causal":
                s[np.arange(held)[None] > kv + np.arange(ql)[:, None]] = -np.inf
            m = s.max(1, keepdims=True)
            e = np.exp(s - m)
            z = e.sum(1, keepdims=True)
            lse[t:t + ql, h] = (m + np.log(z))[:, 0]
            out[t:t + ql, h] = e / z @ v[n:n + held, h]
            mag[t:t + ql, h] = e / z @ np.abs(v[n:n + held, h])
        t, n = t + ql, n + held
    return out, lse, mag
