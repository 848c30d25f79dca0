"""Plain 64-bit forms of the paged serving operators, and the error bounds the
kernels are held to.

Bounds count roundings: one rounding to type t is off by at most u(t) =
finfo(t).eps / 2 relative to the value (bf16 2^-8, fp32 2^-24).  For a row with
softmax weights p over n keys:
  * a logit is a sum of d products in fp32, scaled: it is off by at most
    e = (d + 4) 2^-24 scale sum_i |q_i k_i|, and the base-2 exponent it becomes
    by two more roundings of its own size;
  * the exponential adds 2^-21, so every weight is off by a factor of at most
    1 + w, w = 2 e + 2^-20 + 3 |logit - m| 2^-24 (m: the reference maximum; the
    weights that count are within 40 of it), and the weights' sum too;
  * bf16: each weight is rounded for its product with V (u = 2^-8);
  * products with V are summed in fp32 in some order: n roundings at most, each
    2^-23 (tensor cores may truncate) of sum_j p_j |v_j|;
  * the output is rounded once to its type.
So |dO| <= A (u_p + 2 w + n 2^-23 + 2^-20) + u_o |O| with A = sum_j p_j |v_j|,
and |dlse| <= e + w + (n / 32 + 40) 2^-24 + 4 |lse| 2^-24 (the sum of the
weights runs in at least 32 partial sums).
"""
from __future__ import annotations

import math

import numpy as np


def pages_of(n, ps):
    return -(-n // ps)


def plan(q_len, kv_len, free, n_free, table, ps, max_tokens):
    """(table, q_start, slot_map, positions, n_free), request by request."""
    table = table.copy()
    slots = np.full(max_tokens, -1, np.int64)
    pos = np.full(max_tokens, -1, np.int32)
    q_start = [0]
    t = 0
    for s, (q, kv) in enumerate(zip(q_len, kv_len)):
        for i in range(pages_of(kv - q, ps), pages_of(kv, ps)):
            n_free -= 1
            table[s, i] = free[n_free]
        for p in range(kv - q, kv):
            slots[t] = table[s, p // ps] * ps + p % ps
            pos[t] = p
            t += 1
        q_start.append(t)
    return table, np.array(q_start, np.int32), slots, pos, n_free


def release(kv_len, keep, table, free, n_free, ps):
    free = free.copy()
    for s, (kv, k) in enumerate(zip(kv_len, keep)):
        for i in range(pages_of(k, ps), pages_of(kv, ps)):
            free[n_free] = table[s, i]
            n_free += 1
    return free, n_free


def attention(Q, K, V, ps, table, q_start, kv_len, scale, causal, window, bf16):
    """O [T][H][d], lse [H][T] in 64 bits and their bounds, for rows that
    belong to a request; `mine` [T] marks those.  Q, K, V: 64-bit arrays of the
    rows and the pool."""
    T, H, d = Q.shape
    hk = K.shape[1]
    G = H // hk
    O = np.zeros((T, H, d))
    lse = np.full((H, T), -np.inf)
    tO = np.zeros((T, H, d))
    tl = np.zeros((H, T))
    mine = np.zeros(T, bool)
    u_p, u_o = (2.0 ** -8, 2.0 ** -8) if bf16 else (0.0, 2.0 ** -24)
    for s in range(len(kv_len)):
        a, b, kv = int(q_start[s]), int(q_start[s + 1]), int(kv_len[s])
        ids = table[s, :pages_of(kv, ps)]
        for t in range(a, b):
            mine[t] = True
            pos = kv - (b - a) + t - a
            hi = min(kv, pos + 1) if causal else kv
            lo = max(0, pos + 1 - window) if window else 0
            if hi <= lo:
                continue
            j = np.arange(lo, hi)
            pg, off = ids[j // ps], j % ps
            for g in range(hk):
                k, v = K[pg, g, off], V[pg, g, off]          # [n][d]
                q = Q[t, g * G:(g + 1) * G]                  # [G][d]
                x = q @ k.T * scale
                m = x.max(1, keepdims=True)
                p = np.exp(x - m)
                l = p.sum(1, keepdims=True)
                z = (m + np.log(l))[:, 0]
                p /= l
                o = p @ v
                e = ((d + 4) * 2.0 ** -24 * scale * (np.abs(q) @ np.abs(k).T)).max(1)
                w = 2 * e + 2.0 ** -20 + 3 * 40 * 2.0 ** -24
                n = hi - lo
                A = p @ np.abs(v)
                hs = slice(g * G, (g + 1) * G)
                O[t, hs], lse[hs, t] = o, z
                tO[t, hs] = A * (u_p + 2 * w + n * 2.0 ** -23 + 2.0 ** -20)[:, None] \
                    + u_o * np.abs(o) * 1.01 + 1e-30
                tl[hs, t] = e + w + (n / 32 + 40) * 2.0 ** -24 + 4 * np.abs(z) * 2.0 ** -24
    return O, lse, tO, tl, mine


def default_scale(d):
    return 1.0 / math.sqrt(d)
