"""The serving-loop oracles against independent statements of the same
mathematics (CPU)."""

import numpy as np
import pytest

import oracle
from tests import serving_cases as sc


@pytest.mark.parametrize("lens", [[1], [0, 7, 3], [20]])
def test_recurrence_is_the_chain(lens):
    """Every sequence is a tree that is a chain: the replay oracle's outputs and last state."""
    x = sc.layer_inputs(lens, 2, 4, 16, False, seed=3)
    o, S = oracle.serving.recurrence(scale=0.5, **x)
    for b, n in enumerate(lens):
        s = slice(x["starts"][b], x["starts"][b + 1])
        if n == 0:
            assert np.array_equal(S[b], x["S0"][b].astype(np.float64))
            continue
        parent = np.arange(-1, n - 1, dtype=np.int32)[None]
        args = [np.repeat(x[m][s], 2, axis=1)[None] for m in ("q", "k")] + [x[m][s][None] for m in ("v", "g", "beta")]
        ro, rS = oracle.replay_batch(parent, *args, x["S0"][b:b + 1], keep_states=True, scale=0.5)
        assert np.allclose(o[s], ro[0], rtol=1e-12, atol=1e-12)
        assert np.allclose(S[b], rS[0, n - 1], rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("draft", [True, False])
def test_accepted_tokens_follow_the_target(draft):
    """The first emitted token is distributed as the target's row at the root,
    whatever the draft: 40,000 walks over a vocabulary of 5, every frequency
    within five standard deviations."""
    rng = np.random.default_rng(11)
    V, B, T = 5, 40000, 4
    p1, q1 = rng.dirichlet(np.ones(V)), rng.dirichlet(np.ones(V))
    parent = np.tile(np.array([-1, 0, 0, 1], np.int32), (B, 1))
    p = np.broadcast_to(p1.astype(np.float32), (B, T, V))
    if draft:
        q = np.broadcast_to(q1.astype(np.float32), (B, T, V))
        tokens = rng.choice(V, size=(B, T), p=q1).astype(np.int32)
    else:
        q = None
        tokens = np.tile(np.argsort(-q1)[[0, 0, 1, 0]].astype(np.int32), (B, 1))
    _, out, counts = oracle.serving.accept(p, tokens, parent, rng.random((B, T)).astype(np.float32),
                                           rng.exponential(size=(B, V)).astype(np.float32), q=q)
    assert (counts >= 1).all()
    freq = np.bincount(out[:, 0], minlength=V) / B
    assert (np.abs(freq - p1) < 5 * np.sqrt(p1 * (1 - p1) / B)).all()
    two = out[counts >= 2][:, 1]  # and so is the token after it
    freq = np.bincount(two, minlength=V) / two.size
    assert (np.abs(freq - p1) < 5 * np.sqrt(p1 * (1 - p1) / two.size)).all()
