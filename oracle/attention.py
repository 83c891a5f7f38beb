"""CPU oracle for the attention token mixer and its paged cache, in float64.

TEST INFRASTRUCTURE ONLY (like oracle/vq3_oracle.py): it shares no code with the CUDA library.

`attend` is the definition, one request at a time; `bound` an elementwise bound of the error that
the library's number formats allow, from arithmetic:

  u      half a step of the 16-bit type, relative: the output is rounded once, each probability once
  delta  relative error of a probability before that rounding: its exponent (base 2) is off by at most
         2^-24 times (D + 3) roundings of a sum of magnitude S = max_j sum_d |q_d k_jd| scale log2(e),
         the exponential itself by 2^-22
  n      terms summed in FP32: (n + 8) 2^-24 relative to the sum of magnitudes, in numerator and sum
  FP16   probabilities below 2^-14 of the format's window, which reaches 2^7 above the running maximum's
         1, are off by up to 2^-25 each: n 2^-32 max|v| relative to a sum of at least 1
"""

from __future__ import annotations

import numpy as np

HALF_STEP = {"f16": 2.0**-11, "bf16": 2.0**-8}


def attend(q, k, v, seen, scale):
    """q [n, H, D], k and v [L, Hkv, D], seen [n] keys per row -> out [n, H, D], lse [n, H], magnitudes
    A = sum p |v| / sum p [n, H, D] and S [n, H], all float64."""
    n, H, D = q.shape
    L, Hkv, _ = k.shape
    out = np.zeros((n, H, D))
    mag = np.zeros((n, H, D))
    lse = np.full((n, H), -np.inf)
    S = np.zeros((n, H))
    for h in range(H):
        kh, vh = k[:, h // (H // Hkv)], v[:, h // (H // Hkv)]
        s = q[:, h] @ kh.T * scale
        hidden = np.arange(L)[None] >= np.asarray(seen)[:, None]
        for i in range(n):
            if hidden[i].all():
                continue
            live = ~hidden[i]
            x = s[i, live]
            m = x.max()
            p = np.exp(x - m)
            lse[i, h] = m + np.log(p.sum())
            out[i, h] = p @ vh[live] / p.sum()
            mag[i, h] = p @ np.abs(vh[live]) / p.sum()
            S[i, h] = (np.abs(kh[live]) @ np.abs(q[i, h])).max() * scale * np.log2(np.e)
    return out, lse, mag, S


def bound(out, lse, mag, S, n, D, vmax, dtype):
    u = HALF_STEP[dtype]
    delta = np.log(2) * (D + 3) * 2.0**-24 * S + 2.0**-22
    sums = (n + 8) * 2.0**-24
    off = n * 2.0**-32 * vmax if dtype == "f16" else 0.0
    e = (u + 2 * delta[..., None] + 2 * sums) * mag * (1 + u) + off
    # the rounding of the output, with FP16's smallest step (2^-24) for tiny values
    return e + u * (np.abs(out) + e) + 2.0**-25, delta + 2 * sums + 2.0**-22 * (1 + np.where(np.isfinite(lse), np.abs(lse), 0))


def plan(cached, fresh, table, ring, head, count, page, max_tokens):
    """The page plan, token by token. Returns (status, table, q_start, kv_len, slots, positions, (head, count))."""
    R, width = table.shape
    status = 0
    need = [-(-(c + n) // page) for c, n in zip(cached, fresh)]
    held = [-(-c // page) for c in cached]
    if any(c < 0 or n < 0 or c + n > 0x3FFFFFFF for c, n in zip(cached, fresh)) or not 0 <= head < len(ring) or \
            not 0 <= count <= len(ring):
        return 8, None, None, None, None, None, None
    if sum(need) - sum(held) > count:
        status |= 1
    if any(n > width for n in need):
        status |= 2
    if sum(fresh) > max_tokens:
        status |= 4
    slots, positions = [-1] * max_tokens, [-1] * max_tokens
    if status:
        return status, table, [0] * (R + 1), [0] * R, slots, positions, (head, count)
    table = table.copy()
    q_start, t = [0], 0
    for r in range(R):
        for c in range(held[r], need[r]):
            table[r, c] = ring[head]
            head = (head + 1) % len(ring)
            count -= 1
        for i in range(fresh[r]):
            pos = cached[r] + i
            pg = int(table[r, pos // page])
            slots[t] = pg * page + pos % page if pg >= 0 else -1
            positions[t] = pos
            t += 1
        q_start.append(t)
    return 0, table, q_start, [c + n for c, n in zip(cached, fresh)], slots, positions, (head, count)
