"""Timed cases of the attention layers that stand between Gated DeltaNet layers.

Models that stack Gated DeltaNet layers put a softmax attention layer between
every few of them.  Its keys and values stay in pages of a cache, and a draft
tree passes through it as it passes through the other layers:

  qk_prep       the norm of every head's query and key, the rotation by the
                token's position (one or several axes) in the same pass, and
                the keys and values put into the cache's pages;
  attend        the new tokens' attention over the paged cache: one token of
                every stream, the nodes of a draft tree along their root paths,
                or chunks of prompts; whole, or through a sliding window with a
                few first tokens that stay visible;
  cache_commit  the accepted path's keys and values moved together in the
                pages, and the streams' new lengths.

For row i of a sequence with n new rows behind c tokens in the cache, at
position t_i = c + depth_i (depth_i = i without a tree):
    x -> w x / sqrt(mean x^2 + eps)  (rms)  or  x / sqrt(sum x^2 + eps)  (l2),
    (x_a, x_b) -> (x_a cos f - x_b sin f, x_b cos f + x_a sin f) with f the
        position times the pair's frequency, for the first R of the d columns;
    o_i = sum_j p_ij v_j, p_i the softmax of scale q_i.k_j over the tokens j
        that i sees: the cache's and its root path's (itself among them), those
        with t_i - t_j < window or t_j < sinks where there is a window.

``run`` computes a case in plain torch (``own`` false) or through the
library's entry points (``own`` true).
"""

import math

import numpy as np
import torch

own = False

EPS = 1e-6


# ---------------------------------------------------------------------------
# Cases.


def listed():
    return [
        # A lone user's next token: queries and keys normed and rotated, the key and value put into the cache.
        {"name": "prep_step_1", "op": "qk_prep", "B": 1, "N": 1, "HQ": 16, "HKV": 4, "d": 128, "bf16": True,
         "norm": "rms", "rot": 64, "axes": 1, "pairs": "half", "cache": True, "page": 64, "ctx": 700},
        # The unit queries and keys that the tree verify takes, for the bench's batch of 16 trees of 64 nodes.
        {"name": "prep_unit_16x64", "op": "qk_prep", "B": 16, "N": 1024, "HQ": 16, "HKV": 16, "d": 128, "bf16": True,
         "norm": "l2", "rot": 0, "axes": 1, "pairs": "half", "cache": False, "page": 64, "ctx": 0},
        # Five prompts with images in them: rotation by time, height and width, an odd total, into pages of 16.
        {"name": "prep_images_16383", "op": "qk_prep", "B": 5, "N": 16383, "HQ": 32, "HKV": 8, "d": 128, "bf16": True,
         "norm": "rms", "rot": 128, "axes": 3, "pairs": "half", "cache": True, "page": 16, "ctx": 900},
        # A lone user's next token behind a short conversation, where the call's latency is everything.
        {"name": "attend_step_1", "op": "attend", "rows": "step", "B": 1, "N": 1, "HQ": 16, "HKV": 4, "d": 128,
         "bf16": True, "page": 64, "ctx": 700, "window": 0, "sinks": 0},
        # A decode batch of conversations of very different lengths.
        {"name": "attend_step_64", "op": "attend", "rows": "step", "B": 64, "N": 64, "HQ": 32, "HKV": 8, "d": 128,
         "bf16": True, "page": 16, "ctx": 16000, "window": 0, "sinks": 0},
        # One stream behind a very long document: the work is split along the cache.
        {"name": "attend_step_long", "op": "attend", "rows": "step", "B": 1, "N": 1, "HQ": 16, "HKV": 2, "d": 128,
         "bf16": True, "page": 128, "ctx": 262143, "window": 0, "sinks": 0},
        # The bench's batch of 16 trees of up to 64 nodes, ragged, behind some thousand tokens.
        {"name": "attend_tree_16x64", "op": "attend", "rows": "tree", "B": 16, "N": 1024, "HQ": 16, "HKV": 4,
         "d": 128, "bf16": True, "page": 64, "ctx": 6001, "window": 0, "sinks": 0},
        # fp32 activations and cache, small trees, narrow heads.
        {"name": "attend_tree_4x33_fp32", "op": "attend", "rows": "tree", "B": 4, "N": 132, "HQ": 8, "HKV": 2,
         "d": 64, "bf16": False, "page": 32, "ctx": 1000, "window": 0, "sinks": 0},
        # Prompts packed together in a layer with a sliding window and four sinks, seven queries a key head.
        {"name": "attend_window_8191", "op": "attend", "rows": "packed", "B": 6, "N": 8191, "HQ": 28, "HKV": 4,
         "d": 128, "bf16": True, "page": 32, "ctx": 5000, "window": 1024, "sinks": 4},
        # The largest: a chunk of 4,096 tokens of a long prompt behind what the cache already holds of it.
        {"name": "attend_chunk_4096", "op": "attend", "rows": "packed", "B": 1, "N": 4096, "HQ": 32, "HKV": 8,
         "d": 128, "bf16": True, "page": 64, "ctx": 28672, "window": 0, "sinks": 0},
        # A drafted chain of eight tokens of one stream, prepared into the cache and its accepted part kept.
        {"name": "commit_chain_8", "op": "cache_commit", "tree": "chain", "B": 1, "T": 8, "HQ": 16, "HKV": 4,
         "d": 128, "bf16": True, "norm": "rms", "rot": 64, "axes": 1, "pairs": "half", "page": 64, "ctx": 700},
        # Forty-eight trees of 64 nodes, prepared into the cache and the accepted paths moved together.
        {"name": "commit_48x64", "op": "cache_commit", "tree": "random", "B": 48, "T": 64, "HQ": 32, "HKV": 8,
         "d": 128, "bf16": True, "norm": "rms", "rot": 128, "axes": 1, "pairs": "half", "page": 16, "ctx": 500},
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread evenly over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["qk_prep", "attend", "attend", "cache_commit"])
    HQ, HKV = rng.choice([(16, 4), (32, 8), (16, 16), (32, 2), (28, 4), (24, 8), (8, 1), (5, 5)])
    bf16 = rng.random() < 0.8
    case = {"op": op, "HQ": HQ, "HKV": HKV, "d": rng.choice([64, 128, 128]), "bf16": bf16,
            "page": rng.choice([16, 32, 64, 128, 256])}
    if op == "attend":
        rows = rng.choice(["step", "tree", "packed"])
        B = _log_int(rng, 1, 64 if rows == "step" else 16)
        n = 1 if rows == "step" else _log_int(rng, 2, 256) if rows == "tree" else 0
        N = B * n if n else max(B, _log_int(rng, 20, 4096 if bf16 else 600))
        most = 260000 // B if rows == "step" else 16000 if rows == "tree" else 28000
        window = _log_int(rng, 16, 4096) if rng.random() < 0.3 else 0
        return {**case, "rows": rows, "B": B, "N": N, "ctx": _log_int(rng, 1, most if bf16 else min(most, 4000)),
                "window": window, "sinks": rng.choice([0, 1, 4, 130]) if window else 0}
    d = case["d"]
    case.update(norm=rng.choice(["rms", "rms", "l2"]), rot=rng.choice([0, d // 4, d // 2, d]),
                axes=rng.choice([1, 1, 3]), pairs=rng.choice(["half", "half", "adjacent"]))
    if op == "cache_commit":
        return {**case, "tree": rng.choice(["chain", "random", "wide"]), "B": _log_int(rng, 1, 48),
                "T": _log_int(rng, 2, 128), "ctx": _log_int(rng, 1, 1500)}
    N = _log_int(rng, 1, 16383)
    cache = rng.random() < 0.7
    return {**case, "B": min(N, _log_int(rng, 1, 40)), "N": N, "cache": cache,
            "ctx": _log_int(rng, 1, 3000) if cache else 0}


def _spread(b):
    """Fractions of [0, 1) that are far apart for successive b."""
    return (b + 1) * 0.6180339887498949 % 1.0


def _contexts(case):
    """Tokens that each sequence already has in the cache: ctx for one, from a quarter of it for many."""
    B, ctx = case["B"], case["ctx"]
    return [ctx] if B == 1 else [int(ctx * (0.25 + 0.75 * _spread(b))) for b in range(B)]


def _lens(case):
    """New rows of every sequence."""
    B = case["B"]
    if case["op"] == "cache_commit" or case.get("rows") == "tree":
        T = case["T"] if "T" in case else case["N"] // B
        return [T if B == 1 else T - int(0.4 * T * _spread(b)) for b in range(B)]
    if case.get("rows") == "step" or B == 1:
        return [case["N"] // B] * B
    share = [0.05 + _spread(b + 7) ** 2 for b in range(B)]
    cuts = [round(case["N"] * sum(share[:b]) / sum(share)) for b in range(B + 1)]
    return [cuts[b + 1] - cuts[b] for b in range(B)]


def _tree_parents(T, shape, rng):
    return [-1] + [i - 1 if shape == "chain" else (i - 1) // 4 if shape == "wide" else int(rng.randint(i))
                   for i in range(1, T)]


def work(case):
    es, d, HQ, HKV = 2 if case["bf16"] else 4, case["d"], case["HQ"], case["HKV"]
    lens, ctxs = _lens(case), _contexts(case)
    n = sum(lens)
    if case["op"] != "attend":
        # queries in and out, keys in and out, and values where they go into the cache
        cached = case["op"] == "cache_commit" or case["cache"]
        total = 2 * n * (HQ + HKV + (HKV if cached else 0)) * d * es
        if case["op"] == "cache_commit":  # half a tree's depth of keys and values moves
            depth = {"chain": lambda t: t / 2, "wide": lambda t: math.log(t, 4)}.get(case["tree"], math.log)
            total += sum(4 * HKV * d * es * max(0.0, depth(t)) for t in lens if t > 1) * (case["tree"] != "chain")
        return {"bytes": total, "flops": 8.0 * n * (HQ + HKV) * d}
    window, sinks = case["window"] or 1 << 40, case["sinks"]
    pairs = keys = 0.0
    for m, c in zip(lens, ctxs):
        if case["rows"] == "tree":
            m_seen = sum(math.log(i + 1) + 1 for i in range(m))  # nodes on a random tree's root paths
            near = min(c, window)
            pairs += m * (near + min(sinks, c - near)) + m_seen
            keys += near + min(sinks, c - near) + m
        else:
            for i in range(m):
                near = min(c + i + 1, window)
                pairs += near + min(sinks, c + i + 1 - near)
            near = min(c + m, window + m - 1)
            keys += near + min(sinks, c + m - near)
    return {"bytes": 2 * n * HQ * d * es + 2 * keys * HKV * d * es, "flops": 4.0 * pairs * HQ * d}


# ---------------------------------------------------------------------------
# Inputs.


def _positions(case, lens, ctxs, rng):
    """Positions [axes, n] of the new tokens: text counts all axes on alike, an image's tokens share their time
    and carry their row and column."""
    rows = []
    for m, c in zip(lens, ctxs):
        if case["axes"] == 1:
            rows.append(np.arange(c, c + m)[None])
            continue
        at, t, parts = 0, c, [np.zeros((3, 0), int)]
        while at < m:
            text = int(rng.randint(20, 200))
            parts.append(np.repeat(np.arange(t, t + text)[None], 3, 0))
            t += text
            h, w = (int(x) for x in rng.randint(8, 40, size=2))
            y, x = np.divmod(np.arange(h * w), w)
            parts.append(np.stack([np.full(h * w, t), t + y, t + x]))
            t += max(h, w)
            at += text + h * w
        rows.append(np.concatenate(parts, 1)[:, :m])
    return np.concatenate(rows, 1).astype(np.int32)


def _pages(case, lens, ctxs, gen):
    """A cache of shuffled pages with the tokens before the call in it (and room for the new ones), and the
    sequences' page tables."""
    ps = case["page"]
    need = [-(-(c + m) // ps) for c, m in zip(ctxs, lens)]
    total = sum(need) + 3
    order = torch.randperm(total, device="cuda", generator=gen).int()
    table = torch.full((len(need), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    dt = torch.bfloat16 if case["bf16"] else torch.float32
    shape = (total, case["HKV"], ps, case["d"])
    return {"k_cache": torch.randn(shape, device="cuda", generator=gen, dtype=dt),
            "v_cache": torch.randn(shape, device="cuda", generator=gen, dtype=dt), "page_table": table}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    rng = np.random.RandomState(seed % (1 << 31))
    HQ, HKV, d = case["HQ"], case["HKV"], case["d"]
    dt = torch.bfloat16 if case["bf16"] else torch.float32
    lens, ctxs = _lens(case), _contexts(case)
    tree = case["op"] == "cache_commit" or case.get("rows") == "tree"
    B = case["B"]
    T = (case["T"] if "T" in case else case["N"] // B) if tree else None
    n = B * T if tree else sum(lens)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    def ints(x):
        return torch.from_numpy(np.asarray(x, np.int32)).cuda()

    s = {"case": case, "lens": lens, "ctxs": ctxs, "T": T, "starts": None, "lengths": None, "context": ints(ctxs)}
    if tree:
        s["parent_h"] = [_tree_parents(T, case.get("tree", "random"), rng) for _ in range(B)]
        s["parent"] = ints(s["parent_h"])
        s["lengths"] = ints(lens)
    elif lens != [1] * B:
        s["starts"] = ints(np.concatenate([[0], np.cumsum(lens)]))
    lead = (B, T) if tree else (n,)
    if case["op"] == "attend":
        # queries and keys as a layer with normed heads has them; some heads look sharply, some evenly
        sharp = torch.linspace(0.5, 2.0, HQ, device="cuda")[:, None]
        s["q"] = (normal(*lead, HQ, d) * sharp).to(dt)
        s.update(_pages(case, lens, ctxs, gen))
        s["scale"] = d ** -0.5
        if tree:  # the loop's buffer of outputs: rows behind a tree's end stay as they are
            s["out"] = torch.zeros_like(s["q"])
        if own:
            from gated_deltanet_linear_tree_gb300 import canopy

            s["ws"] = canopy.attend_workspace(n, B, HQ, HKV, d)
        return s
    # what a projection gives, scales differing from token to token; one row in some hundreds is a pad's zeros
    size = torch.exp(normal(*lead, 1, 1))
    size = torch.where(torch.rand(*lead, 1, 1, device="cuda", generator=gen) < 0.003, torch.zeros_like(size), size)
    s["q"], s["k"] = ((normal(*lead, H, d) * size).to(dt) for H in (HQ, HKV))
    s["q_weight"] = s["k_weight"] = None
    if case["norm"] == "rms":
        s["q_weight"], s["k_weight"] = 1 + 0.2 * normal(d), 1 + 0.2 * normal(d)
    s["freqs"] = s["positions"] = s["axis"] = None
    if case["rot"]:
        half = case["rot"] // 2
        s["freqs"] = (1e6 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).float()
        if tree:
            depth = [[0] * T for _ in range(B)]
            for b in range(B):
                for i in range(1, T):
                    depth[b][i] = depth[b][s["parent_h"][b][i]] + 1
            pos = np.asarray(depth) + np.asarray(ctxs)[:, None]
            pos = np.broadcast_to(pos, (case["axes"], B, T)).astype(np.int32)
        else:
            pos = _positions(case, lens, ctxs, rng)
        if case["axes"] == 1:
            s["positions"] = ints(pos[0])
        else:
            s["positions"] = ints(pos)
            # a frequency's axis: time for the first half, then height and width by turns
            s["axis"] = ints([0 if i < half // 2 else 1 + i % 2 for i in range(half)])
    if case["op"] == "cache_commit" or case["cache"]:
        s["v"] = normal(*lead, HKV, d).to(dt)
        s.update(_pages(case, lens, ctxs, gen))
    if case["op"] == "cache_commit":
        s["q_out"] = torch.zeros_like(s["q"])  # the loop's buffer: rows behind a tree's end stay as they are
        s["accepted"] = ints([rng.randint(m) for m in lens])
    return s


# ---------------------------------------------------------------------------
# Plain forms.


def _rows_of(s):
    """(sequence, index in it, row) of every new row, as index tensors."""
    b = np.repeat(np.arange(len(s["lens"])), s["lens"])
    i = np.concatenate([np.arange(m) for m in s["lens"]])
    row = b * s["T"] + i if s["T"] else np.arange(len(b))
    return (torch.from_numpy(x).cuda() for x in (b, i, row))


def _plain_norm_rotate(x, weight, s):
    case = s["case"]
    y = x.float()
    y2 = (y * y).sum(-1, keepdim=True)
    y = y / torch.sqrt(y2 / case["d"] + EPS) * weight if case["norm"] == "rms" else y / torch.sqrt(y2 + EPS)
    half = case["rot"] // 2
    if half:
        pos = s["positions"].double()
        angle = pos[..., None] * s["freqs"].double()  # the product of a far position is long
        if case["axes"] > 1:
            angle = angle.gather(0, s["axis"].long().expand(angle.shape[1:])[None])[0]
        cos, sin = torch.cos(angle).float()[..., None, :], torch.sin(angle).float()[..., None, :]
        a, b = (y[..., :half], y[..., half:2 * half]) if case["pairs"] == "half" else \
            (y[..., 0:2 * half:2], y[..., 1:2 * half:2])
        ra, rb = a * cos - b * sin, b * cos + a * sin
        turned = torch.cat([ra, rb], -1) if case["pairs"] == "half" else torch.stack([ra, rb], -1).flatten(-2)
        y = torch.cat([turned, y[..., 2 * half:]], -1)
    return y.to(x.dtype)


def _plain_prep(s):
    q = _plain_norm_rotate(s["q"], s["q_weight"], s)
    k = _plain_norm_rotate(s["k"], s["k_weight"], s)
    if "k_cache" not in s:
        return q, k
    b, i, row = _rows_of(s)
    at = s["context"].long()[b] + i
    ps = s["case"]["page"]
    page = s["page_table"].long()[b, at // ps]
    for cache, x in ((s["k_cache"], k), (s["v_cache"], s["v"])):
        cache[page, :, at % ps] = x.flatten(0, -3)[row]
    if s["T"]:  # rows behind a tree's end are not prepared
        q = torch.where((torch.arange(s["T"], device="cuda") < s["lengths"][:, None])[..., None, None], q, 0)
    return q, s["k_cache"], s["v_cache"]


def _reach(s):
    """[B, T, T]: whether node j is on node i's root path (i itself among them), by squaring: after r rounds the
    nodes up to 2^r steps above."""
    B, T = s["parent"].shape
    node = torch.arange(T, device="cuda")
    reach = ((s["parent"][..., None] == node) | torch.eye(T, dtype=torch.bool, device="cuda")).float()
    for _ in range((T - 1).bit_length()):
        reach = ((reach @ reach) > 0).float()
    return reach > 0


def _softmax_of(q, K, V, seen, s):
    """q [b, n, HQ, d] over K, V [b, HKV, m, d], where seen [b, n, m] (a row at least sees one); fp32."""
    b, n, HQ, d = q.shape
    HKV, m = K.shape[1:3]
    x = q.float().reshape(b, n, HKV, HQ // HKV, d).permute(0, 2, 3, 1, 4).reshape(b, HKV, -1, d)
    z = (s["scale"] * (x @ K.transpose(-1, -2))).reshape(b, HKV, HQ // HKV, n, m)
    z = torch.where(seen[:, None, None], z, -torch.inf)
    p = torch.exp(z - z.amax(-1, keepdim=True))
    y = (p.reshape(b, HKV, -1, m) @ V).reshape(b, HKV, HQ // HKV, n, d) / p.sum(-1, keepdim=True)
    return y.permute(0, 3, 1, 2, 4).reshape(b, n, HQ, d).to(q.dtype)


def _near(at, place, case):
    """Whether a row at position `at` sees one at position `place` before it."""
    if not case["window"]:
        return at >= place
    return (at >= place) & ((at - place < case["window"]) | (place < case["sinks"]))


def _plain_attend_even(s):
    """Single tokens and trees: every stream's rows at once, the caches filled up to one length."""
    case = s["case"]
    B, ps = case["B"], case["page"]
    q = s["q"].reshape(B, -1, case["HQ"], case["d"])
    T = q.shape[1]
    lens = s["lengths"].long() if s["T"] else torch.ones(B, dtype=torch.int64, device="cuda")
    c = s["context"].long()[:, None]
    reach = _reach(s) if s["T"] else torch.ones(B, 1, 1, dtype=torch.bool, device="cuda")
    depth = reach.sum(-1) - 1
    m = max(x + y for x, y in zip(s["lens"], s["ctxs"]))
    key = torch.arange(m, device="cuda").expand(B, m)
    node = (key - c).clamp(0, T - 1)
    new = key >= c
    place = torch.where(new, c + depth.gather(1, node), key)
    seen = ~new[:, None] | reach.gather(2, node[:, None].expand(B, T, m))
    seen &= _near((c + depth)[..., None], place[:, None], case) & (key < c + lens[:, None])[:, None]
    seen[..., 0] |= ~seen.any(-1)  # a row behind its tree's end (not returned)
    table = s["page_table"][:, :-(-m // ps)].long()
    there = (key < c + lens[:, None])[:, None, :, None]
    K, V = (torch.where(there, x[table.clamp_min(0)].transpose(1, 2).flatten(2, 3)[:, :, :m].float(), 0)
            for x in (s["k_cache"], s["v_cache"]))
    o = _softmax_of(q, K, V, seen, s)
    return torch.where((torch.arange(T, device="cuda") < lens[:, None])[..., None, None], o, 0).reshape(s["q"].shape)


def _plain_attend_packed(s):
    """Prompts: sequence by sequence, some hundred rows at a time."""
    case = s["case"]
    ps = case["page"]
    o = torch.empty_like(s["q"])
    first = 0
    for b, (m, c) in enumerate(zip(s["lens"], s["ctxs"])):
        pages = s["page_table"][b, :-(-(c + m) // ps)].long()
        K, V = (x[pages].transpose(0, 1).flatten(1, 2)[None, :, :c + m].float() for x in (s["k_cache"], s["v_cache"]))
        place = torch.arange(c + m, device="cuda")
        for r in range(0, m, 512):
            rows = slice(r, min(m, r + 512))
            seen = _near(place[c:][rows, None], place, case)
            o[first:first + m][rows] = _softmax_of(s["q"][first:first + m][rows][None], K, V, seen[None], s)[0]
        first += m
    return o


def _plain_attend(s):
    return (_plain_attend_packed if s["starts"] is not None else _plain_attend_even)(s)


def _plain_commit(s):
    q, K, V = _plain_prep(s)
    reach = _reach(s)
    depth = reach.sum(-1) - 1
    path = reach.gather(1, s["accepted"].long()[:, None, None].expand(-1, 1, reach.shape[2]))[:, 0]
    context = s["context"] + path.sum(1).int()
    b, node = path.nonzero(as_tuple=True)
    c, ps = s["context"].long()[b], s["case"]["page"]
    src, dst = c + node, c + depth[b, node]
    for cache in (K, V):
        moved = cache[s["page_table"].long()[b, src // ps], :, src % ps]
        cache[s["page_table"].long()[b, dst // ps], :, dst % ps] = moved
    return q, K, V, context


def run(s):
    op, case = s["case"]["op"], s["case"]
    if not own:
        return {"qk_prep": _plain_prep, "attend": _plain_attend, "cache_commit": _plain_commit}[op](s)
    from gated_deltanet_linear_tree_gb300 import canopy

    if op == "attend":
        return canopy.attend(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["context"], s["ws"],
                             starts=s["starts"], parent=s.get("parent"), lengths=s["lengths"], window=case["window"],
                             sinks=case["sinks"], scale=s["scale"], out=s.get("out"))
    args = {"norm": case["norm"], "q_weight": s["q_weight"], "k_weight": s["k_weight"], "eps": EPS,
            "freqs": s["freqs"], "positions": s["positions"], "axis": s["axis"], "pairs": case["pairs"]}
    if "k_cache" not in s:
        return canopy.qk_prep(s["q"], s["k"], **args)
    q, _ = canopy.qk_prep(s["q"], s["k"], v=s["v"], k_cache=s["k_cache"], v_cache=s["v_cache"],
                          page_table=s["page_table"], context=s["context"], starts=s["starts"], lengths=s["lengths"],
                          q_out=s.get("q_out"), **args)
    if op == "qk_prep":
        return q, s["k_cache"], s["v_cache"]
    context = canopy.cache_commit(s["accepted"], s["parent"], s["k_cache"], s["v_cache"], s["page_table"],
                                  s["context"], lengths=s["lengths"])
    return q, s["k_cache"], s["v_cache"], context


# ---------------------------------------------------------------------------
# The definitions in 64 bits.


def _exact_rotated(x, weight, s):
    """Norm and rotation as complex numbers, pair by pair."""
    case = s["case"]
    x = x.double()
    if case["norm"] == "rms":
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.double()
    else:
        x = x * torch.rsqrt(x.square().sum(-1, keepdim=True) + EPS)
    half = case["rot"] // 2
    for i in range(half):
        at = (i, i + half) if case["pairs"] == "half" else (2 * i, 2 * i + 1)
        pos = s["positions"] if case["axes"] == 1 else s["positions"][int(s["axis"][i])]
        angle = pos.double() * s["freqs"][i].double()
        z = torch.complex(x[..., at[0]], x[..., at[1]]) * torch.polar(torch.ones_like(angle), angle)[..., None]
        x[..., at[0]], x[..., at[1]] = z.real, z.imag
    return x


def _exact_prep(s):
    q = _exact_rotated(s["q"], s["q_weight"], s)
    k = _exact_rotated(s["k"], s["k_weight"], s)
    if "k_cache" not in s:
        return q, k
    K, V = s["k_cache"].double(), s["v_cache"].double()
    table, ps, first = s["page_table"].cpu(), s["case"]["page"], 0
    for b, (m, c) in enumerate(zip(s["lens"], s["ctxs"])):
        at = 0
        while at < m:  # page by page
            page, slot = int(table[b, (c + at) // ps]), (c + at) % ps
            cnt = min(ps - slot, m - at)
            src = (b, slice(at, at + cnt)) if s["T"] else slice(first + at, first + at + cnt)
            K[page, :, slot:slot + cnt] = k[src].transpose(0, 1)
            V[page, :, slot:slot + cnt] = s["v"][src].double().transpose(0, 1)
            at += cnt
        if s["T"]:
            q[b, m:] = 0
        first += m
    return q, K, V


def _exact_attend(s):
    case = s["case"]
    HQ, HKV, d, ps, T = case["HQ"], case["HKV"], case["d"], case["page"], s["T"]
    window = case["window"] or 1 << 40
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda").reshape(-1, HQ, d)
    qs = s["q"].reshape(-1, HQ, d)
    first = 0
    for b, (m, c) in enumerate(zip(s["lens"], s["ctxs"])):
        lo = b * T if T else first
        first += m
        table = s["page_table"][b].long()
        depth, above = list(range(m)), None
        if T:
            parent, above = s["parent_h"][b], np.zeros((m, m), bool)
            for i in range(m):
                if i:
                    above[i] = above[parent[i]]
                    depth[i] = depth[parent[i]] + 1
                else:
                    depth[i] = 0
                above[i, i] = True
            above = torch.from_numpy(above).cuda()
        place = torch.cat([torch.arange(c), c + torch.tensor(depth, dtype=torch.int64)]).cuda()
        for r in range(0, m, 256):
            i = torch.arange(r, min(m, r + 256), device="cuda")
            # without a tree nothing behind the last row of the block is seen
            last = c + (m if T else int(i[-1]) + 1)
            j = torch.arange(last, device="cuda")
            far = place[c + i][:, None] - place[None, :last]
            hidden = (far >= window) & (place[None, :last] >= case["sinks"])
            if T:
                hidden[:, c:] |= ~above[i]
            else:
                hidden |= far < 0
            seen = (~hidden).any(0).nonzero()[:, 0]  # the others need not be read
            for h in range(HKV):
                K = s["k_cache"][table[j[seen] // ps], h, j[seen] % ps].double()
                V = s["v_cache"][table[j[seen] // ps], h, j[seen] % ps].double()
                for g in range(h * HQ // HKV, (h + 1) * HQ // HKV):
                    z = (qs[lo + i, g].double() @ K.T) * s["scale"]
                    z.masked_fill_(hidden[:, seen], -torch.inf)
                    out[lo + i, g] = torch.exp(z - torch.logsumexp(z, 1, keepdim=True)) @ V
    return out.reshape(s["q"].shape)


def _exact_commit(s):
    q, K, V = _exact_prep(s)
    table, ps = s["page_table"].tolist(), s["case"]["page"]
    for b, node in enumerate(s["accepted"].tolist()):
        path = []
        while node >= 0:
            path.append(node)
            node = s["parent_h"][b][node]
        c = s["ctxs"][b]
        for at, node in enumerate(reversed(path)):  # a node's place is never before its depth's
            if at != node:
                to, fro = c + at, c + node
                for cache in (K, V):
                    cache[table[b][to // ps], :, to % ps] = cache[table[b][fro // ps], :, fro % ps]
    return q, K, V, None


def exact(case, seed):
    if case["op"] == "attend" and work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    return {"qk_prep": _exact_prep, "attend": _exact_attend, "cache_commit": _exact_commit}[case["op"]](s)
