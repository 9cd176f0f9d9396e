"""A Gated DeltaNet layer through a serving loop, on the GPU.

Prompts of different lengths go through the layer (prefill); rounds of tree
speculation follow (verify, accept, commit), then single tokens (step).  The
inputs are synthetic: the layer's activations and the target's and draft's
probabilities are random, with the draft near the target.  At the end the
states are compared with the layer run token by token over exactly the tokens
that each stream kept.

    python examples/serving_loop.py
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from gated_deltanet_linear_tree_gb300 import canopy  # noqa: E402

B, H, HV, D, T, V = 4, 16, 32, 128, 24, 4096
SCALE = D ** -0.5


def activations(n, gen):
    """q, k (unit rows), v, decay gates and write strengths of n tokens."""
    q, k = (torch.nn.functional.normalize(torch.randn(n, H, D, device="cuda", generator=gen), dim=-1).bfloat16()
            for _ in range(2))
    v = torch.randn(n, HV, D, device="cuda", generator=gen).bfloat16()
    g = torch.exp(-0.1 * torch.rand(n, HV, device="cuda", generator=gen))
    beta = torch.rand(n, HV, device="cuda", generator=gen)
    return [q, k, v, g, beta]


def main():
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    kept = [[] for _ in range(B)]  # per stream, the activations of the tokens that its state has taken in

    # prompts
    lens = [300, 17, 1025, 64]
    starts = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).int().cuda()
    x = activations(sum(lens), gen)
    ws = canopy.prefill_workspace(sum(lens), B, HV, D)
    o, S = canopy.prefill(*x, None, starts, ws, scale=SCALE, o_dtype=torch.bfloat16)
    for b in range(B):
        kept[b].append([y[starts[b]:starts[b + 1]] for y in x])
    print(f"prefill: {sum(lens)} tokens of {B} prompts, {canopy.prefill_plan(sum(lens), B, H, HV, True, D)}")

    # rounds of speculation over 24-node trees
    tree_ws = canopy.workspace(B, T, HV, D)
    parent = torch.tensor([-1] + [(i - 1) // 2 for i in range(1, T)], dtype=torch.int32, device="cuda").repeat(B, 1)
    for rnd in range(4):
        x = activations(B * T, gen)
        tree = [y.view(B, T, *y.shape[1:]) for y in x]
        o = canopy.verify(*tree, S, parent, tree_ws, scale=SCALE)
        logits = 3 * torch.randn(B, T, V, device="cuda", generator=gen)
        p = torch.softmax(logits, -1)
        q = torch.softmax(logits + 0.5 * torch.randn(B, T, V, device="cuda", generator=gen), -1)
        tokens = torch.zeros(B, T, dtype=torch.int32, device="cuda")
        for c in range(1, T):  # a node's children are drawn from its row of the draft
            tokens[:, c] = torch.multinomial(q[:, (c - 1) // 2], 1, generator=gen)[:, 0]
        u = torch.rand(B, T, device="cuda", generator=gen)
        noise = torch.empty(B, V, device="cuda").exponential_(generator=gen).clamp_min_(1e-20)
        accepted, out, counts = canopy.accept(p, tokens, parent, u, noise, q=q)
        S = canopy.commit(accepted, S, tree[1], parent, tree_ws)
        print(f"round {rnd}: tokens per stream {counts.tolist()}")
        for b in range(B):
            path, n = [], int(accepted[b])
            while n >= 0:
                path.insert(0, b * T + n)
                n = int(parent[b, n])
            kept[b].append([y[path] for y in x])

    # single tokens, the state in place
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(8):
        x = activations(B, gen)
        o, S = canopy.step(*x, S, S_out=S, scale=SCALE, err=err)
        for b in range(B):
            kept[b].append([y[b:b + 1] for y in x])
    assert int(err) == 0 and canopy.read_device_error(ws) == 0 and canopy.read_device_error(tree_ws) == 0

    # the same tokens one by one
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for b in range(B):
        y = [torch.cat(z).contiguous() for z in zip(*kept[b])]
        one[1] = y[0].shape[0]
        w = canopy.prefill_workspace(y[0].shape[0], 1, HV, D)
        _, ref = canopy.prefill(*y, None, one, w, scale=SCALE, force="scan")
        rel = float((S[b] - ref[0]).norm() / ref[0].norm())
        print(f"stream {b}: {y[0].shape[0]} tokens, state off by {rel:.1e}")
        assert rel < 1e-3


if __name__ == "__main__":
    main()
