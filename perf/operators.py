"""Timed cases of the serving-loop operators around the tree verify.

A stream served by Gated DeltaNet layers passes through three more steps next
to the draft tree's verify and commit:

  prefill  the layer over whole prompts (packed sequences of different
           lengths): outputs o and the state that the first verify starts from;
  step     the layer's recurrence for one token of every stream;
  accept   which node of the draft tree the target model's probabilities
           accept, the emitted tokens, and the token sampled after them.

The layer's rule, per sequence and value head, with the state S [dv][dk]:
    S_t = g_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T,
    o_t = scale S_t q_t.

``run`` computes a case in plain torch (``own`` false) or through the
library's entry points (``own`` true).
"""

import numpy as np
import torch

own = False

CHUNK = 64  # tokens per chunk of the plain prefill


# ---------------------------------------------------------------------------
# Cases.


def listed():
    return [
        # One token for a single stream: a lone user's next token, where the call's latency is everything.
        {"name": "step_1", "op": "step", "B": 1, "H": 16, "HV": 32, "bf16": True, "o_bf16": True},
        # A batch of 16 streams of the 16/32-head layer.
        {"name": "step_16", "op": "step", "B": 16, "H": 16, "HV": 32, "bf16": True, "o_bf16": True},
        # fp32 activations, one q/k head per value head, an odd batch.
        {"name": "step_33_fp32", "op": "step", "B": 33, "H": 16, "HV": 16, "bf16": False, "o_bf16": False},
        # A full decode batch: the states alone are 0.8 GB in and out.
        {"name": "step_200", "op": "step", "B": 200, "H": 16, "HV": 32, "bf16": True, "o_bf16": True},
        # A short question, less than one chunk.
        {"name": "prompt_37", "op": "prefill", "B": 1, "N": 37, "H": 16, "HV": 16, "bf16": True, "o_bf16": True},
        # fp32 activations over a few prompts.
        {"name": "prompts_600_fp32", "op": "prefill", "B": 4, "N": 600, "H": 16, "HV": 16, "bf16": False,
         "o_bf16": False},
        # Sixteen prompts of very different lengths packed together, an odd total, one of them empty; fp32 o.
        {"name": "prompts_8191", "op": "prefill", "B": 16, "N": 8191, "H": 16, "HV": 32, "bf16": True,
         "o_bf16": False},
        # One long document: the chunks follow one another, the heads alone are parallel.
        {"name": "document_16384", "op": "prefill", "B": 1, "N": 16384, "H": 16, "HV": 32, "bf16": True,
         "o_bf16": True},
        # The largest: a prefill batch of eight prompts.
        {"name": "prompts_32768", "op": "prefill", "B": 8, "N": 32768, "H": 16, "HV": 32, "bf16": True,
         "o_bf16": True},
        # A drafted chain of seven tokens behind the last one, for one stream.
        {"name": "accept_chain_8", "op": "accept", "B": 1, "T": 8, "V": 32000, "tree": "chain", "draft": True,
         "ragged": False, "bf16": False},
        # The bench's batch of 64-node trees, candidates taken as the draft's most likely tokens.
        {"name": "accept_16x64", "op": "accept", "B": 16, "T": 64, "V": 131072, "tree": "random", "draft": False,
         "ragged": False, "bf16": False},
        # Ragged trees sampled from the draft's probabilities, an odd vocabulary.
        {"name": "accept_48x33", "op": "accept", "B": 48, "T": 33, "V": 50021, "tree": "random", "draft": True,
         "ragged": True, "bf16": False},
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread evenly over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["step", "prefill", "accept"])
    if op == "accept":
        return {"op": op, "B": _log_int(rng, 1, 48), "T": _log_int(rng, 2, 64), "V": _log_int(rng, 1000, 131072),
                "tree": rng.choice(["chain", "random", "wide"]), "draft": rng.random() < 0.5,
                "ragged": rng.random() < 0.5, "bf16": rng.random() < 0.3}
    heads = rng.choice([(16, 32), (16, 16), (8, 32), (4, 8), (3, 6), (16, 48)])
    bf16 = rng.random() < 0.8
    o_bf16 = bf16 and rng.random() < 0.6
    if op == "step":
        return {"op": op, "B": _log_int(rng, 1, 130), "H": heads[0], "HV": heads[1], "bf16": bf16, "o_bf16": o_bf16}
    most = 20000 if bf16 else 1000
    n = _log_int(rng, 1, most)
    return {"op": op, "B": min(n, _log_int(rng, 1, 24)), "N": n, "H": heads[0], "HV": heads[1], "bf16": bf16,
            "o_bf16": o_bf16}


def work(case):
    if case["op"] == "accept":
        # the last accepted node's row of the target (and the draft), and the noise; one probability per node
        es = 2 if case["bf16"] else 4
        B, T, V = case["B"], case["T"], case["V"]
        rows = 2 if case["draft"] else 1
        return {"bytes": B * V * (rows * es + 4) + B * T * (16 + rows * es), "flops": 3.0 * B * V}
    d, es, eo = 128, 2 if case["bf16"] else 4, 2 if case["o_bf16"] else 4
    n = case["N"] if case["op"] == "prefill" else case["B"]
    io = n * (2 * case["H"] * d * es + case["HV"] * (d * (es + eo) + 8))
    states = 2 * case["B"] * case["HV"] * d * d * 4
    # S k, the rank-one update and S q, two operations per element each
    return {"bytes": io + states, "flops": 6.0 * d * d * n * case["HV"]}


# ---------------------------------------------------------------------------
# Inputs.


def _lengths_of(case, seed):
    """B sequence lengths with the given sum: uneven, and one of them empty in larger batches."""
    B, N = case["B"], case["N"]
    rng = np.random.RandomState(seed % (1 << 31))
    if B == 1:
        return [N]
    share = rng.gamma(1.5, size=B)
    if B >= 4:
        share[rng.randint(B)] = 0.0
    cuts = np.floor(np.cumsum(share / share.sum()) * N + 0.5).astype(int)
    cuts[-1] = N
    return np.diff(np.concatenate([[0], cuts])).tolist()


def _layer_inputs(case, n, gen):
    """q, k (unit rows per head), v, decay gates and write strengths for n tokens, and B states."""
    H, HV, d = case["H"], case["HV"], 128
    dt = torch.bfloat16 if case["bf16"] else torch.float32

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    q, k = normal(n, H, d), normal(n, H, d)
    q = (q / q.norm(dim=-1, keepdim=True)).to(dt)
    k = (k / k.norm(dim=-1, keepdim=True)).to(dt)
    v = normal(n, HV, d).to(dt)
    # heads forget at different rates, from within a few tokens to over hundreds
    rate = 2.0 ** -(7.0 * torch.arange(HV, device="cuda") / max(1, HV - 1))
    g = torch.exp(-torch.nn.functional.softplus(normal(n, HV)) * rate)
    beta = torch.sigmoid(normal(n, HV))
    S0 = 0.1 * normal(case["B"], HV, d, d)
    return {"q": q, "k": k, "v": v, "g": g, "beta": beta, "S0": S0}


def _trees(case, rng):
    """Parent arrays [B, T] in topological order, and each node's rank among its siblings."""
    B, T = case["B"], case["T"]
    parent = np.full((B, T), -1, np.int32)
    rank = np.zeros((B, T), np.int64)
    for b in range(B):
        children = np.zeros(T, np.int64)
        for i in range(1, T):
            if case["tree"] == "chain":
                p = i - 1
            elif case["tree"] == "wide":
                p = (i - 1) // 4
            else:
                p = rng.randint(i)
                while children[p] >= 8:
                    p = rng.randint(i)
            parent[b, i] = p
            rank[b, i] = children[p]
            children[p] += 1
    return parent, rank


def _accept_inputs(case, seed, gen):
    B, T, V = case["B"], case["T"], case["V"]
    dt = torch.bfloat16 if case["bf16"] else torch.float32
    rng = np.random.RandomState(seed % (1 << 31))
    parent_h, rank_h = _trees(case, rng)
    parent = torch.from_numpy(parent_h).cuda()
    z = 4.0 * torch.randn(B, T, V, device="cuda", generator=gen)
    p = torch.softmax(z, -1).to(dt)
    z += 1.0 * torch.randn(B, T, V, device="cuda", generator=gen)
    rows = torch.arange(B, device="cuda")[:, None].expand(B, T)
    pp = parent.long().clamp_min(0)
    if case["draft"]:  # a node's children are independent samples of its row of the draft
        q = torch.softmax(z, -1).to(dt)
        tokens = torch.empty(B, T, dtype=torch.int32, device="cuda")
        for c in range(T):
            race = torch.empty(B, V, device="cuda").exponential_(generator=gen).clamp_min_(1e-20)
            tokens[:, c] = (q[rows[:, c], pp[:, c]].float() / race).argmax(-1).int()
    else:  # a node's children are its draft's most likely tokens in order
        q = None
        best = torch.topk(z, 1 + int(rank_h.max()), dim=-1).indices
        tokens = best[rows, pp, torch.from_numpy(rank_h).cuda()].int()
    del z
    lengths = None
    if case["ragged"]:
        lengths = torch.from_numpy(rng.randint(1, T + 1, size=B).astype(np.int32)).cuda()
    return {"p": p, "q": q, "tokens": tokens.contiguous(), "parent": parent, "lengths": lengths,
            "u": torch.rand(B, T, device="cuda", generator=gen),
            "noise": torch.empty(B, V, device="cuda").exponential_(generator=gen).clamp_min_(1e-20)}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    if case["op"] == "accept":
        s = _accept_inputs(case, seed, gen)
    elif case["op"] == "step":
        s = _layer_inputs(case, case["B"], gen)
        s["S_new"] = torch.empty_like(s["S0"])  # the other of the two state buffers that the loop alternates
    else:
        s = _layer_inputs(case, case["N"], gen)
        s["lens"] = _lengths_of(case, seed)
        starts = np.concatenate([[0], np.cumsum(s["lens"])]).astype(np.int32)
        s["starts"] = torch.from_numpy(starts).cuda()
    s["case"] = case
    s["scale"] = 128 ** -0.5
    s["o_dtype"] = torch.bfloat16 if case.get("o_bf16") else torch.float32
    if own and case["op"] == "prefill":
        from gated_deltanet_linear_tree_gb300 import canopy

        s["ws"] = canopy.prefill_workspace(case["N"], case["B"], case["HV"], 128)
    return s


# ---------------------------------------------------------------------------
# Plain forms.


def _plain_step(s):
    rep = s["v"].shape[1] // s["q"].shape[1]
    q = s["q"].float().repeat_interleave(rep, 1)
    k = s["k"].float().repeat_interleave(rep, 1)
    S = s["S0"] * s["g"][..., None, None]
    u = s["beta"][..., None] * (s["v"].float() - (S @ k[..., None])[..., 0])
    S = S + u[..., None] * k[..., None, :]
    o = s["scale"] * (S @ q[..., None])[..., 0]
    return o.to(s["o_dtype"]), S


def _plain_prefill(s):
    """Chunks of 64 tokens of the sequences padded to one length: within a chunk, with l the running
    sum of log g, G_ij = beta_i exp(l_i - l_j) k_i.k_j (j < i) and C_ij = exp(l_i - l_j) q_i.k_j (j <= i),
        (I + G) U = beta (V - exp(l) K S^T),  o = exp(l) Q S^T + C U,
        S <- exp(l_last) S + sum_j exp(l_last - l_j) u_j k_j^T."""
    starts, N, B = s["starts"].long(), s["q"].shape[0], s["starts"].numel() - 1
    HV, d = s["v"].shape[1:]
    rep = HV // s["q"].shape[1]
    nc = max(1, -(-max(s["lens"]) // CHUNK))
    pos = torch.arange(nc * CHUNK, device="cuda")
    at = starts[:-1, None] + pos
    valid = at < starts[1:, None]
    at = at.clamp_max(N - 1)

    def lay(x, fill):  # [N, heads, ...] -> [nc, B, heads, CHUNK, ...]
        x = x[at].float()
        x = torch.where(valid.reshape(valid.shape + (1,) * (x.dim() - 2)), x, torch.full_like(x, fill))
        x = x.reshape((B, nc, CHUNK) + x.shape[2:]).transpose(0, 1).transpose(2, 3)
        return x.repeat_interleave(HV // x.shape[2], 2) if x.shape[2] != HV else x

    q, k, v = lay(s["q"], 0.0), lay(s["k"], 0.0), lay(s["v"], 0.0)
    g, beta = lay(s["g"], 1.0), lay(s["beta"], 0.0)[..., None]
    l = torch.log(g).cumsum(-1)
    i = torch.arange(CHUNK, device="cuda")
    below = i[:, None] >= i[None, :]
    decay = torch.exp(torch.where(below, l[..., :, None] - l[..., None, :], torch.full((), -torch.inf, device="cuda")))
    eye = torch.eye(CHUNK, device="cuda")
    A = beta * decay * (k @ k.transpose(-1, -2))
    A = torch.where(i[:, None] == i[None, :], eye, A)
    W = torch.linalg.solve_triangular(A, eye.expand_as(A).contiguous(), upper=False, unitriangular=True)
    C = decay * (q @ k.transpose(-1, -2))
    gamma = torch.exp(l)[..., None]
    last = decay[..., -1, :, None]
    S = s["S0"]
    o = torch.empty_like(v)
    for c in range(nc):  # the state passes from chunk to chunk
        U = W[c] @ (beta[c] * (v[c] - gamma[c] * (k[c] @ S.transpose(-1, -2))))
        o[c] = gamma[c] * (q[c] @ S.transpose(-1, -2)) + C[c] @ U
        S = gamma[c][..., -1:, :] * S + (last[c] * U).transpose(-1, -2) @ k[c]
    o = o.transpose(2, 3).transpose(0, 1).reshape(B * nc * CHUNK, HV, d)
    n = torch.arange(N, device="cuda")
    b = torch.searchsorted(starts, n, right=True) - 1
    return (s["scale"] * o[b * (nc * CHUNK) + n - starts[b]]).to(s["o_dtype"]), S


def _plain_accept(s):
    """Every stream walks from its root.  At node i with target row p and draft row q, the children are
    tried in index order against the row r (p at first) of mass Z (1 at first): child c with token x is
    accepted if u_c Z q(x) < r(x); a rejected one leaves r <- max(r - Z q, 0) and Z its sum (in units of
    2^-46, so that the sum does not depend on its order).  Without draft probabilities q is the token
    itself: accepted if u_c Z < r(x), else r(x) <- 0 and Z <- max(Z - r(x), 0).  Where no child is
    accepted, the next token is the lowest index with the largest r / noise (of p where r is all zero)."""
    p, q, tokens, parent, u, noise = s["p"], s["q"], s["tokens"].long(), s["parent"], s["u"], s["noise"]
    B, T, V = p.shape
    rows = torch.arange(B, device="cuda")
    n = s["lengths"] if s["lengths"] is not None else torch.full((B,), T, dtype=torch.int32, device="cuda")
    cur = torch.where(n > 0, 0, -1)
    r, Z = p[:, 0].float(), torch.ones(B, device="cuda")
    out = torch.full((B, T), -1, dtype=torch.int32, device="cuda")
    count = torch.zeros(B, dtype=torch.int64, device="cuda")
    for c in range(1, T):  # a node's children come after it, and siblings in order
        tried = (parent[:, c] == cur) & (c < n)
        x = tokens[:, c:c + 1]
        rx = r.gather(1, x)[:, 0]
        if q is not None:
            qrow = q[rows, cur.clamp_min(0)].float()
            accepted = tried & (u[:, c] * Z * qrow.gather(1, x)[:, 0] < rx)
            left = (r - Z[:, None] * qrow).clamp_min(0)
            mass = (left * 2.0 ** 46).to(torch.int64).sum(1).float() * 2.0 ** -46
        else:
            accepted = tried & (u[:, c] * Z < rx)
            left = r.scatter(1, x, 0.0)
            mass = (Z - rx).clamp_min(0)
        refused = tried & ~accepted
        r = torch.where(accepted[:, None], p[:, c].float(), torch.where(refused[:, None], left, r))
        Z = torch.where(accepted, torch.ones_like(Z), torch.where(refused, mass, Z))
        cur = torch.where(accepted, c, cur)
        out[rows, count.clamp_max(T - 1)] = torch.where(accepted, x[:, 0].int(), -1)
        count += accepted
    score = r / noise
    score = torch.where(score.max(1, keepdim=True).values > 0, score, p[rows, cur.clamp_min(0)].float() / noise)
    best = torch.where(score == score.max(1, keepdim=True).values, torch.arange(V, device="cuda"), V).min(1).values
    out[rows, count.clamp_max(T - 1)] = torch.where(n > 0, best.int(), -1)
    return cur.int(), out, (count + (n > 0)).int()


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"step": _plain_step, "prefill": _plain_prefill, "accept": _plain_accept}[op](s)
    from gated_deltanet_linear_tree_gb300 import canopy

    if op == "step":
        return canopy.step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["S0"], S_out=s["S_new"], o_dtype=s["o_dtype"],
                           scale=s["scale"])
    if op == "prefill":
        return canopy.prefill(s["q"], s["k"], s["v"], s["g"], s["beta"], s["S0"], s["starts"], s["ws"],
                              o_dtype=s["o_dtype"], scale=s["scale"])
    return canopy.accept(s["p"], s["tokens"], s["parent"], s["u"], s["noise"], q=s["q"], lengths=s["lengths"])


# ---------------------------------------------------------------------------
# The definition in 64 bits: the recurrence, token by token.


def exact(case, seed):
    if case["op"] == "accept":
        return None  # whole numbers throughout
    s = prepare(case, seed)
    B, HV = case["B"], case["HV"]
    lens = s["lens"] if case["op"] == "prefill" else [1] * B
    if max(lens) * (1 + B * HV / 512) > 100000:
        return None
    first = torch.tensor([sum(lens[:b]) for b in range(B)], device="cuda")
    n = torch.tensor(lens, device="cuda")
    head = torch.arange(HV, device="cuda") // (HV // case["H"])
    S = s["S0"].double()
    out = torch.zeros(sum(lens), HV, 128, dtype=torch.float64, device="cuda")
    order = torch.tensor(sorted(range(B), key=lambda b: -lens[b]), device="cuda")
    for t in range(max(lens)):
        m = sum(x > t for x in lens)  # the streams, longest first, that still have a token
        at, who = first[order[:m]] + t, order[:m]
        qt, kt = s["q"][at][:, head].double(), s["k"][at][:, head].double()
        vt, gt, bt = s["v"][at].double(), s["g"][at].double(), s["beta"][at].double()
        P = S[who]
        u = bt[..., None] * (vt - gt[..., None] * torch.matmul(P, kt[..., None])[..., 0])
        P = gt[..., None, None] * P + u[..., :, None] * kt[..., None, :]
        out[at] = s["scale"] * torch.matmul(P, qt[..., None])[..., 0]
        S[who] = P
    return out, S
