"""attend where every CTA works on twenty and more tiles of keys, as it does for a user: rings of stages that go
round several times, maxima that grow late in a piece, CTAs that walk many pieces.  Sampled rows against the
definition in 64 bits; the rest by their repetition, bit for bit."""

import numpy as np
import pytest
import torch

from attention_cases import attend_bound

pytestmark = pytest.mark.gpu

# name -> type, (HQ, HKV, d), page, sequences as (new rows, context), rows a stream (trees or tokens) or None for
# packed ones, window, sinks
CASES = {
    "tokens": (True, (32, 8, 128), 16, [(1, 4000 + 700 * b) for b in range(8)], 1, 0, 0),
    "tokens_d64": (True, (16, 16, 64), 64, [(1, 4000 + 900 * b) for b in range(5)], 1, 0, 0),
    "token_long": (True, (16, 2, 128), 128, [(1, 199999)], 1, 0, 0),
    "tokens_window": (True, (32, 8, 128), 32, [(1, 9000 + 100 * b) for b in range(16)], 1, 3500, 200),
    "few_trees": (True, (16, 4, 128), 64, [(4 - b % 2, 5000 + 300 * b) for b in range(16)], 4, 0, 0),
    "few_mixed": (True, (16, 4, 128), 16, [(1, 3000 + 100 * b) for b in range(40)] + [(90, 5000)], None, 0, 0),
    "packed": (True, (16, 4, 128), 64, [(300, 3000), (1, 700), (700, 4500), (64, 3333)], None, 0, 0),
    "packed_d64": (True, (16, 8, 64), 256, [(200, 9000), (0, 50), (600, 8111)], None, 0, 0),
    "packed_heads": (True, (48, 1, 128), 32, [(50, 4000), (131, 9001)], None, 0, 0),
    "window": (True, (28, 4, 128), 32, [(4100, 100), (31, 2000), (1, 1500)], None, 1000, 4),
    "window_d64": (True, (16, 16, 64), 16, [(5000, 300), (3001, 4000)], None, 900, 140),
    "trees": (True, (16, 4, 128), 64, [(64 - 2 * b, 3000 + 300 * b) for b in range(16)], 64, 0, 0),
    "trees_window": (True, (16, 4, 128), 16, [(64 - b, 6000 + 100 * b) for b in range(16)], 64, 4500, 10),
    "fp32_tokens": (False, (32, 8, 128), 16, [(1, 4000 + 700 * b) for b in range(8)], 1, 0, 0),
    "fp32_packed": (False, (16, 4, 128), 64, [(100, 5000), (201, 5100)], None, 0, 0),
    "fp32_trees": (False, (8, 4, 64), 32, [(33 - b, 6000) for b in range(20)], 33, 5000, 9),
}


def units_of_a_cta(lib, bf16, HQ, HKV, d, seqs, N, window, sinks):
    g = HQ // HKV
    plan = lib.attend_plan(N, len(seqs), HQ, HKV, bf16, d)
    if plan == "tiles":
        rows, keys, ctas = 2 * (128 // g), 80 if d == 128 else 128, 152
    else:
        rows, keys, ctas = (16 if N * g <= 16 * len(seqs) else 64) // g, 64, 304
    total = 0
    for n, c in seqs:
        for r in range(0, n, rows):
            total += HKV * (min(c + r, window + sinks if window else c + r) // keys)
    return total / ctas


def inputs(name):
    bf16, (HQ, HKV, d), page, seqs, T, window, sinks = CASES[name]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(sorted(CASES).index(name))
    rng = np.random.RandomState(len(name))
    dt = torch.bfloat16 if bf16 else torch.float32
    normal = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    B, N = len(seqs), len(seqs) * T if T else sum(n for n, _ in seqs)
    need = [-(-(c + n) // page) for n, c in seqs]
    order = torch.randperm(sum(need) + 2, device="cuda", generator=gen).int()
    table = torch.full((B, max(need) + 1), -1, dtype=torch.int32, device="cuda")
    # every third head's keys look more and more, every third less and less along a direction of the queries
    u = torch.nn.functional.normalize(normal(HKV, d), dim=-1)
    q = 0.5 * normal(N, HQ, d) + 20 * u.repeat_interleave(HQ // HKV, 0)
    k, v = normal(len(order), HKV, page, d), normal(len(order), HKV, page, d)
    at = 0
    for b, ((n, c), m) in enumerate(zip(seqs, need)):
        mine = order[at:at + m]
        table[b, :m], at = mine, at + m
        ramp = 25 * torch.arange(m * page, device="cuda").view(m, 1, page, 1) / (m * page)
        kind = torch.arange(HKV, device="cuda").view(1, HKV, 1, 1) % 3
        k[mine.long()] += torch.where(kind == 1, ramp, torch.where(kind == 2, 25 - ramp, 0)) * u[:, None]
    x = {"q": q.to(dt), "k": k.to(dt), "v": v.to(dt), "table": table, "N": N,
         "context": torch.tensor([c for _, c in seqs], dtype=torch.int32, device="cuda"), "starts": None,
         "parent": None, "lengths": None}
    if not T:
        x["starts"] = torch.tensor(np.concatenate([[0], np.cumsum([n for n, _ in seqs])]), dtype=torch.int32,
                                   device="cuda")
    elif T > 1:
        x["q"] = x["q"].view(B, T, HQ, d)
        x["lengths"] = torch.tensor([n for n, _ in seqs], dtype=torch.int32, device="cuda")
        x["parent"] = torch.tensor([[-1] + [rng.randint(max(0, i - 5), i) for i in range(1, T)] for _ in range(B)],
                                   dtype=torch.int32, device="cuda")
    return x


def definition(x, name, b, i):
    """Row i of sequence b in 64 bits: (its row of q, o, sum p |v|)."""
    bf16, (HQ, HKV, d), page, seqs, T, window, sinks = CASES[name]
    n, c = seqs[b]
    row = b * T + i if T else sum(m for m, _ in seqs[:b]) + i
    places, times = list(range(c)), list(range(c))
    if x["parent"] is None:
        places, times, t = list(range(c + i + 1)), list(range(c + i + 1)), c + i
    else:
        path, node = [], i
        while node >= 0:
            path, node = [node] + path, int(x["parent"][b, node])
        places, times, t = places + [c + j for j in path], times + [c + j for j in range(len(path))], c + len(path) - 1
    places, times = torch.tensor(places, device="cuda"), torch.tensor(times, device="cuda")
    if window:
        places = places[(t - times < window) | (times < sinks)]
    pages = x["table"][b].long()[places // page]
    K, V = (y[pages, :, places % page].double().repeat_interleave(HQ // HKV, 1) for y in (x["k"], x["v"]))
    z = d ** -0.5 * torch.einsum("hd,mhd->hm", x["q"].view(-1, HQ, d)[row].double(), K)
    p = torch.exp(z - z.amax(1, keepdim=True))
    p /= p.sum(1, keepdim=True)
    return row, torch.einsum("hm,mhd->hd", p, V), torch.einsum("hm,mhd->hd", p, V.abs())


@pytest.mark.parametrize("name", CASES)
def test_many_tiles_a_cta(lib, name):
    bf16, (HQ, HKV, d), page, seqs, T, window, sinks = CASES[name]
    x = inputs(name)
    assert units_of_a_cta(lib, bf16, HQ, HKV, d, seqs, x["N"], window, sinks) >= 20
    ws = lib.attend_workspace(x["N"], len(seqs), HQ, HKV, d)

    def run():
        return lib.attend(x["q"], x["k"], x["v"], x["table"], x["context"], ws, starts=x["starts"],
                          parent=x["parent"], lengths=x["lengths"], window=window, sinks=sinks,
                          out=torch.full_like(x["q"], 7.0)).view(-1, HQ, d)

    o = run()
    assert lib.read_device_error(ws) == 0
    rng = np.random.RandomState(0)
    norms = x["k"].double().square().sum(-1)
    top = x["k"].view(-1, d)[norms.argmax()].double().cpu().numpy()[None]
    got, ref, weight, rows = [], [], [], []
    for b, (n, c) in enumerate(seqs):
        for i in sorted({0, n - 1, *rng.randint(0, n, size=min(n, 7))} if n else ()):
            row, r, w = definition(x, name, b, int(i))
            rows.append(row)
            got.append(o[row].double())
            ref.append(r)
            weight.append(w)
    got, ref, weight = (torch.stack(y).cpu().numpy() for y in (got, ref, weight))
    c = dict(q=x["q"].view(-1, HQ, d)[rows].double().cpu().numpy(), k=top, scale=d ** -0.5, bf16=bf16)
    # (the largest sum of magnitudes of a score is that of the longest row and key: their norms' product)
    bound = attend_bound(c, ref, weight, max(n + m for n, m in seqs))
    off = np.abs(got - ref)
    assert (off <= bound).all(), f"{(off / bound).max():.3g} of the bound"
    if T and T > 1:  # rows behind a tree's end
        for b, (n, _) in enumerate(seqs):
            assert (o[b * T + n:(b + 1) * T] == 7).all()
    for _ in range(3):
        assert torch.equal(run(), o)
