"""CPU oracle for the layers around RMA attention (test infrastructure only).

Plain FP64 restatements, token by token, of the query/key norm with the position rotation, the short
causal convolution and the gated delta rule, on values expanded exactly from their BF16 or FP32
storage.  Results stay FP64.  It shares no code with the CUDA library.
"""
from __future__ import annotations

import numpy as np


def norm_rope(x, w, positions, inv_freq, eps, interleaved=False):
    """x [B, n, H, D] f64, w [D], positions [B, n] or [B, n, H], inv_freq [pairs]: RMS norm, then rotation."""
    x = np.asarray(x, np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    pairs = len(inv_freq)
    if pairs == 0:
        return y
    pos = np.asarray(positions, np.float64)
    if pos.ndim == 2:
        pos = pos[:, :, None]
    angle = pos[..., None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(angle), np.sin(angle)
    i = np.arange(pairs)
    u, v = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
    out = y.copy()
    out[..., u] = y[..., u] * c - y[..., v] * s
    out[..., v] = y[..., v] * c + y[..., u] * s
    return out


def conv_silu(x, state, w, bias=None, lens=None):
    """x [B, n, C], state [B, 3, C], w [C, 4]: (out [B, n, C] with NaN past the lengths, new state)."""
    x, state, w = (np.asarray(t, np.float64) for t in (x, state, w))
    B, n, C = x.shape
    out = np.full((B, n, C), np.nan)
    new = state.copy()
    for b in range(B):
        m = n if lens is None else int(lens[b])
        seen = np.concatenate([state[b], x[b, :m]])
        for t in range(m):
            z = (seen[t:t + 4] * w.T).sum(0) + (0.0 if bias is None else np.asarray(bias, np.float64))
            out[b, t] = z / (1.0 + np.exp(-z))
        new[b] = seen[m:]
    return out, new


def delta_gates(a, b, a_log, dt_bias):
    """Log decay and beta from the projections a, b [..., HV]."""
    z = np.asarray(a, np.float64) + np.asarray(dt_bias, np.float64)
    with np.errstate(over="ignore"):
        g = -np.exp(np.asarray(a_log, np.float64)) * (np.maximum(z, 0) + np.log1p(np.exp(-np.abs(z))))
        return g, 1.0 / (1.0 + np.exp(-np.asarray(b, np.float64)))


def delta_rule(qkv, a, b, a_log, dt_bias, state, n_k_heads, l2norm=True, l2_eps=1e-6, scale=128 ** -0.5, lens=None):
    """The recurrence over qkv [B, n, C], a, b [B, n, HV] from state [B, HV, D, D].

    Returns (out [B, n, HV, D] with NaN past the lengths, new state, out_size, state_size): the sizes
    are the same sums over absolute values (what rounding errors are relative to)."""
    qkv, S = np.asarray(qkv, np.float64), np.array(state, np.float64)
    B, n, _ = qkv.shape
    HV, D = S.shape[1], S.shape[2]
    HK = n_k_heads
    heads = qkv.reshape(B, n, 2 * HK + HV, D)
    of = np.arange(HV) // (HV // HK)

    def unit(x):
        return x / np.sqrt((x * x).sum(-1, keepdims=True) + l2_eps) if l2norm else x

    q, k, v = unit(heads[:, :, :HK])[:, :, of] * scale, unit(heads[:, :, HK:2 * HK])[:, :, of], heads[:, :, 2 * HK:]
    g, beta = delta_gates(a, b, a_log, dt_bias)
    decay = np.exp(g)
    out = np.full((B, n, HV, D), np.nan)
    out_size = np.zeros_like(out)
    size = np.abs(S)
    for t in range(n):
        live = np.ones(B, bool) if lens is None else t < np.asarray(lens)
        d = np.where(live[:, None], decay[:, t], 1.0)[..., None, None]
        bt = np.where(live[:, None], beta[:, t], 0.0)[..., None]
        vt, kt, qt = (np.where(live[:, None, None], x[:, t], 0.0) for x in (v, k, q))
        S = S * d
        u = bt * (vt - np.einsum("bhkv,bhk->bhv", S, kt))
        S = S + kt[..., None] * u[:, :, None]
        size = size * d + np.abs(kt)[..., None] * np.abs(u)[:, :, None]
        o = np.einsum("bhkv,bhk->bhv", S, qt)
        out[live, t] = o[live]
        out_size[:, t] = np.einsum("bhkv,bhk->bhv", size, np.abs(qt))
    return out, S, out_size, size
