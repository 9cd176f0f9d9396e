"""Seeded inputs of the serving-loop operators' tests."""

import numpy as np
import torch

from synth.values import round_bf16


def layer_inputs(lens, H, HV, d, bf16, seed, kind="plain"):
    """q, k, v, g, beta of the packed tokens, S0 and starts, as numpy fp32.

    kind: "plain"; "aligned" (one key for all tokens of a sequence, beta near
    0.5, slow decay: every earlier token counts); "forget" (gates down to
    1e-30 beside gates of 1); "rates" (heads from fast to slow decay)."""
    rng = np.random.default_rng(seed)
    N, B = int(sum(lens)), len(lens)

    def unit(*s):
        x = rng.standard_normal(s)
        return (x / np.sqrt((x ** 2).sum(-1, keepdims=True))).astype(np.float32)

    q, k = unit(N, H, d), unit(N, H, d)
    v = rng.standard_normal((N, HV, d)).astype(np.float32)
    z = rng.standard_normal((N, HV))
    g = np.exp(-np.logaddexp(0.0, z)).astype(np.float32)
    beta = (1 / (1 + np.exp(-rng.standard_normal((N, HV))))).astype(np.float32)
    S0 = (0.1 * rng.standard_normal((B, HV, d, d))).astype(np.float32)
    starts = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    if kind == "aligned":
        for b in range(B):
            k[starts[b]:starts[b + 1]] = unit(1, H, d)
        beta = rng.uniform(0.4, 0.6, (N, HV)).astype(np.float32)
        g = rng.uniform(0.95, 1.0, (N, HV)).astype(np.float32)
    if kind == "forget":
        g = np.where(rng.random((N, HV)) < 0.1, np.float32(1e-30), np.float32(1)).astype(np.float32)
    if kind == "rates":
        g = np.exp(-np.logaddexp(0.0, z) * 2.0 ** -(8 * np.arange(HV) / max(1, HV - 1))).astype(np.float32)
    if bf16:
        q, k, v = round_bf16(q), round_bf16(k), round_bf16(v)
    return dict(q=q, k=k, v=v, g=g, beta=beta, S0=S0, starts=starts)


def to_cuda(x, bf16):
    dt = torch.bfloat16 if bf16 else torch.float32
    out = {n: torch.from_numpy(np.ascontiguousarray(x[n])).cuda() for n in x}
    for n in ("q", "k", "v"):
        out[n] = out[n].to(dt)
    return out


def random_tree(T, rng, kind="random"):
    parent = np.full(T, -1, np.int32)
    for i in range(1, T):
        parent[i] = {"chain": i - 1, "wide": (i - 1) // 4, "star": 0}.get(kind, rng.integers(i))
    return parent


def accept_inputs(B, T, V, seed, kind="random", draft=True, bf16=False, spread=2.0, ragged=False):
    """Target and draft rows, tokens drawn from the draft's rows (or its most
    likely tokens), and the random numbers, as numpy."""
    rng = np.random.default_rng(seed)
    parent = np.stack([random_tree(T, rng, kind) for _ in range(B)])

    def softmax(z):
        e = np.exp(z - z.max(-1, keepdims=True))
        return (e / e.sum(-1, keepdims=True)).astype(np.float32)

    z = spread * rng.standard_normal((B, T, V))
    zq = z + 0.7 * rng.standard_normal((B, T, V))
    p, q = softmax(z), softmax(zq)
    if bf16:
        p, q = round_bf16(p), round_bf16(q)
    tokens = np.zeros((B, T), np.int32)
    for b in range(B):
        seen = {}
        for c in range(1, T):
            i = parent[b, c]
            if draft:
                tokens[b, c] = np.argmax(q[b, i] / rng.exponential(size=V))
            else:
                m = seen[i] = seen.get(i, -1) + 1
                tokens[b, c] = np.argsort(-zq[b, i], kind="stable")[m % V]
    lengths = rng.integers(0, T + 1, B).astype(np.int32) if ragged else None
    return dict(p=p, q=q if draft else None, tokens=tokens, parent=parent, u=rng.random((B, T)).astype(np.float32),
                noise=np.maximum(rng.exponential(size=(B, V)), 1e-20).astype(np.float32), lengths=lengths)
