"""Float64 oracle of the delta rule over packed requests, the short convolution and the rotated append, with
the error that each number format leaves (TEST INFRASTRUCTURE ONLY; shares no code with the library).

The delta rule's recurrence is oracle/delta_rule.py's. For keys of at most unit length and strengths in [0, 1] a
token's map of a state column, s -> a (I - b k k^T) s + b v k, does not lengthen, so an error made at one token
reaches the end no larger than it was made; errors of different tokens are taken as independent (their sum grows
with the root of their number).
"""

from __future__ import annotations

import numpy as np

WINDOW = 32  # tokens that `near` looks back over
ETA = 2.0**-17  # of delta_causal


def delta(q, k, v, beta, alpha, state, scale):
    """One head: out [T, dv], the final state, and what the error bound needs.

    q, k [T, dk]; v [T, dv]; beta, alpha [T]; state [dk, dv], all as float64."""
    S = np.array(state, np.float64)
    T, dv = q.shape[0], v.shape[1]
    out = np.empty((T, dv))
    top = np.linalg.norm(S, axis=0)          # largest length of each state column so far
    reach = np.empty((T, dv))                # |q| times it
    near = np.empty((T, dv))                 # sum over the last WINDOW tokens of |q . k_j| |b_j u_j|
    us = np.zeros((T, dv))
    for t in range(T):
        u = beta[t] * (v[t] - alpha[t] * (S.T @ k[t]))
        S = alpha[t] * S + np.outer(k[t], u)
        us[t] = np.abs(u)
        out[t] = scale * (S.T @ q[t])
        top = np.maximum(top, np.linalg.norm(S, axis=0))
        lo = max(0, t + 1 - WINDOW)
        reach[t] = np.linalg.norm(q[t]) * top
        near[t] = np.abs(k[lo : t + 1] @ q[t]) @ us[lo : t + 1]
    return out, S, {"top": top, "reach": reach, "near": near}


def delta_bound(out, info, v, scale, dtype, q):
    """Tolerances (out [T, dv], state per column [dv]). They take in what a token cannot see (the largest value of all
    tokens, the longest that a state column has been): for values of like size. delta_causal's are the narrower ones.

    FP32 operands enter the products with 22 bits or more (half a step 2^-22), sums of FP32: each of a token's
    four products leaves up to 2^-21 of the column's length and value. For BF16 outputs there is room for products
    of 11-bit operands (half a step 2^-11), one with the state and two with the last WINDOW tokens: more than kernels
    need that take 22 bits for either type. And the sizes are those of all tokens, later ones among them, and of a
    column at its longest: delta_causal has the bound of what a token can see."""
    T = max(1, out.shape[0])
    size = info["top"] + np.abs(v).max(axis=0, initial=0)
    tol_state = 4 * 2.0**-21 * (1 + np.sqrt(T)) * size
    half, part = (2.0**-8, 2.0**-11) if dtype == "bf16" else (2.0**-11, 2.0**-21)
    tiny = 2.0**-134 if dtype == "bf16" else 2.0**-25  # half a step of subnormals
    made = part * (info["reach"] + 2 * info["near"]) + np.linalg.norm(q, axis=1, keepdims=True) * tol_state
    return half * np.abs(out) + (1 + half) * abs(scale) * made + tiny, tol_state


def delta_causal(q, k, v, beta, alpha, state, scale, dtype):
    """One head as `delta`, with tolerances that only what a token can see enters: out, state, tolerances of both.

    A column's size at token t is the largest it has had, as the gates since then leave it: the values', the state
    column's length. Each token adds an error of ETA of that size, earlier ones are shortened by the gates, and
    different tokens' are independent. ETA: four products of operands with 22 bits (2^-21 each), and two sets of
    values that share a power of two with others up to 2^20 larger (2^-39 of the largest, 2^-19 each):
    1.5 * 2^-18 < 2^-17. Both types alike: a 16-bit output adds half a step of its own, no more."""
    S = np.array(state, np.float64)
    T, dv = v.shape
    out, tol = np.empty((T, dv)), np.empty((T, dv))
    size, err = np.linalg.norm(S, axis=0), np.zeros(dv)
    half, tiny = (2.0**-8, 2.0**-134) if dtype == "bf16" else (2.0**-11, 2.0**-25)
    for t in range(T):
        S = alpha[t] * S
        S = S + np.outer(k[t], beta[t] * (v[t] - S.T @ k[t]))
        out[t] = scale * (S.T @ q[t])
        size = np.maximum(alpha[t] * size, np.maximum(np.abs(v[t]), np.linalg.norm(S, axis=0)))
        err = np.hypot(alpha[t] * err, ETA * size)
        tol[t] = half * np.abs(out[t]) + (1 + half) * abs(scale) * np.linalg.norm(q[t]) * err + tiny
    return out, S, tol, err


def conv(x, old, w, bias, silu, unit_heads, head_dim, eps):
    """One request: x [T, C], old [W - 1, C], w [C, W]; out, new state, tolerance before the last rounding."""
    T, W = x.shape[0], w.shape[1]
    line = np.concatenate([old, x])
    y, mag = np.zeros(x.shape), np.zeros(x.shape)
    for j in range(W):
        y += w[:, j] * line[j : j + T]
        mag += np.abs(w[:, j] * line[j : j + T])
    if bias is not None:
        y, mag = y + bias, mag + np.abs(bias)
    z, err = y, W * 2.0**-24 * mag           # W fused multiply-adds
    if silu:
        # exp is off by 2 + 1.173 |y| units of the last place, the quotient by 2, the sum by 1/2
        z = y / (1 + np.exp(-y))
        err = 1.1 * err + np.abs(z) * 2.0**-23 * (5 + 1.2 * np.abs(y))
    n = unit_heads * head_dim
    if n:
        h = z[:, :n].reshape(T, unit_heads, head_dim)
        e = err[:, :n].reshape(T, unit_heads, head_dim)
        length = np.sqrt((h * h).sum(-1, keepdims=True) + eps)
        # the length is off by what its entries are off, by its sums' roundings and those of the root
        rel = np.sqrt((e * e).sum(-1, keepdims=True)) / length + 2.0**-23 * (2 + np.log2(head_dim))
        err = np.concatenate([(e / length + np.abs(h) / length * rel).reshape(T, n), err[:, n:]], 1)
        z = np.concatenate([(h / length).reshape(T, n), z[:, n:]], 1)
    return z, line[T:], err


def rotate(x, positions, freq, interleaved):
    """x [T, H, D] turned; the tolerance before the last rounding is 2^-21 of the pair's length."""
    half = len(freq)
    angle = positions[:, None].astype(np.float64) * np.asarray(freq, np.float64)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    y, size = np.array(x, np.float64), np.zeros(x.shape)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    size[..., a] = size[..., b] = np.hypot(x[..., a], x[..., b])
    return y, 2.0**-21 * size
