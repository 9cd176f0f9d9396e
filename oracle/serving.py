"""The serving-loop steps, straight from their definitions.

recurrence  the layer over packed sequences, token by token in float64
            (canopy page, "The gated delta rule"; S is (dv, dk))
accept      the walk down a draft tree against the target's probabilities:
            float32 products and differences one at a time, and masses
            summed as whole numbers of 2^-46 in Python integers
"""

from __future__ import annotations

import numpy as np


def recurrence(q, k, v, g, beta, S0, starts, scale=1.0):
    """(o [N, HV, dv], S [B, HV, dv, dk]) in float64; q, k [N, H, dk], v
    [N, HV, dv], g, beta [N, HV], S0 [B, HV, dv, dk] or None."""
    q, k, v, g, beta = (np.asarray(x, np.float64) for x in (q, k, v, g, beta))
    N, HV, dv = v.shape
    B, dk = len(starts) - 1, q.shape[2]
    rep = HV // q.shape[1]
    S = np.zeros((B, HV, dv, dk)) if S0 is None else np.array(S0, np.float64)
    o = np.zeros((N, HV, dv))
    for b in range(B):
        for n in range(starts[b], starts[b + 1]):
            for h in range(HV):
                kk, qq, a = k[n, h // rep], q[n, h // rep], g[n, h]
                M = S[b, h]
                u = beta[n, h] * (v[n, h] - a * (M @ kk))
                S[b, h] = a * M + np.outer(u, kk)
                o[n, h] = scale * (S[b, h] @ qq)
    return o, S


def accept(p, tokens, parent, u, noise, q=None, lengths=None):
    """(accepted [B], out_tokens [B, T], counts [B]) for p, q [B, T, V]
    float32 (bf16 values given as float32), tokens in [0, V)."""
    f = np.float32
    B, T, V = p.shape
    accepted, out, counts = np.full(B, -1), np.full((B, T), -1), np.zeros(B, int)
    for b in range(B):
        n = T if lengths is None else int(lengths[b])
        if n == 0:
            continue
        cur, emitted = 0, []
        walking = True
        while walking:
            r, Z = p[b, cur].astype(f), f(1)
            walking = False
            for c in range(cur + 1, n):
                if parent[b, c] != cur:
                    continue
                x = tokens[b, c]
                qx = f(1) if q is None else f(q[b, cur, x])
                if f(f(f(u[b, c]) * Z) * qx) < r[x]:
                    emitted.append(int(x))
                    cur, walking = c, True
                    break
                if q is None:
                    Z = max(f(Z - r[x]), f(0))
                    r = r.copy()
                    r[x] = 0
                else:
                    r = np.maximum(r - Z * q[b, cur].astype(f), f(0))
                    units = [int(y) for y in np.ldexp(r.astype(np.float64), 46)]
                    Z = f(sum(units)) * f(2.0 ** -46)
        row = r if r.max() > 0 else p[b, cur].astype(f)
        emitted.append(int(np.argmax(row / noise[b].astype(f))))
        accepted[b], counts[b] = cur, len(emitted)
        out[b, :len(emitted)] = emitted
    return accepted, out, counts
