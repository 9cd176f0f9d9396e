"""Inputs of the attention layers' tests, and the bounds that their errors are held to."""

import numpy as np
import torch

import oracle
import synth

U32, U16 = 2.0 ** -24, 2.0 ** -8  # half a step of fp32 and bf16, relative


def rounded(x, bf16):
    """x as the type holds it."""
    t = torch.from_numpy(np.asarray(x, np.float32))
    return (t.bfloat16().float() if bf16 else t).numpy()


def tensor(x, bf16=False):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t.bfloat16() if bf16 else t).cuda()


def cache(rng, need, HKV, d, page, bf16, spare=2):
    """(k, v, table): shuffled pages for sequences of `need` places, all places filled; table entries that are
    not needed are -1."""
    count = [-(-n // page) for n in need]
    order = rng.permutation(sum(count) + spare)
    table = np.full((len(need), max(1, max(count)) + 1), -1, np.int32)
    at = 0
    for b, c in enumerate(count):
        table[b, :c] = order[at:at + c]
        at += c
    k, v = (rounded(rng.standard_normal((len(order), HKV, page, d)), bf16) for _ in range(2))
    return k, v, table


def attend_case(seed, lens, ctxs, HQ, HKV, d, page, bf16, T=None, tree=None, sharp=1.5):
    """Rows of sequences with `lens` new tokens behind `ctxs`: packed, or with T rows a stream.  tree: a
    function (T, rng) -> parent array."""
    rng = np.random.RandomState(seed)
    B = len(lens)
    N = B * T if T else sum(lens)
    first = [b * T for b in range(B)] if T else np.concatenate([[0], np.cumsum(lens)])[:-1]
    rows = [range(int(f), int(f) + n) for f, n in zip(first, lens)]
    k, v, table = cache(rng, [c + n for c, n in zip(ctxs, lens)], HKV, d, page, bf16)
    q = rounded(sharp * rng.standard_normal((N, HQ, d)), bf16)
    parent = None if tree is None else np.stack([tree(T, rng) for _ in range(B)]).astype(np.int32)
    return dict(q=q, k=k, v=v, table=table, ctxs=np.asarray(ctxs, np.int32), lens=np.asarray(lens, np.int32),
                rows=rows, parent=parent, T=T, bf16=bf16, scale=d ** -0.5)


def attend_reference(c, window=0, sinks=0):
    return oracle.attention.attend(c["q"], c["k"], c["v"], c["table"], c["ctxs"], c["rows"], c["parent"], window,
                                   sinks, c["scale"])


def attend_bound(c, o, weight, keys):
    """How far an element of o may be off: scores are fp32 sums of d products (each of the scaled sum's terms off
    by at most (d + 4) half steps of the largest sum of magnitudes), the exponential is off by 2^-21, the sums
    over `keys` keys by a half step a term, relative to sum p |v|; bf16 rounds the weights once before the second
    product, and o once."""
    d = c["q"].shape[-1]
    size = c["scale"] * d * np.abs(c["q"]).max() * np.abs(c["k"]).max()
    # the sum of magnitudes of any row and key, by Cauchy-Schwarz, if that is less
    size = min(size, c["scale"] * np.sqrt((c["q"].astype(np.float64) ** 2).sum(-1).max()
                                          * (c["k"].astype(np.float64) ** 2).sum(-1).max()))
    fp32 = 2 * (d + 4) * U32 * size + 2 * 2.0 ** -21 + 2 * (keys + 64) * U32
    half = U16 if c["bf16"] else U32
    return (fp32 + (U16 if c["bf16"] else 0)) * weight + half * np.abs(o) * (1 + fp32 + U16) + 1e-30


TREES = {"chain": lambda T, rng: synth.trees.chain(T), "wide": lambda T, rng: synth.trees.topk(T, 4),
         "random": lambda T, rng: np.array([-1] + [rng.randint(i) for i in range(1, T)], np.int32)}


def run_attend(canopy, c, window=0, sinks=0, ws=None, fill=7.0):
    """The library's output [N, HQ, d] as float64 numpy, the error word, and which rows it left as they were."""
    N, HQ, d = c["q"].shape
    B, HKV = len(c["lens"]), c["k"].shape[1]
    shape = (B, c["T"], HQ, d) if c["T"] and not (c["T"] == 1 and c["parent"] is None) else (N, HQ, d)
    q = tensor(c["q"], c["bf16"]).view(shape)
    out = torch.full_like(q, fill)
    ws = canopy.attend_workspace(N, B, HQ, HKV, d) if ws is None else ws
    starts = lengths = None
    if not c["T"]:
        starts = tensor(np.concatenate([[0], np.cumsum(c["lens"])]).astype(np.int32))
    elif len(shape) == 4:
        lengths = tensor(c["lens"])
    canopy.attend(q, tensor(c["k"], c["bf16"]), tensor(c["v"], c["bf16"]), tensor(c["table"]), tensor(c["ctxs"]), ws,
                  starts=starts, parent=None if c["parent"] is None else tensor(c["parent"]), lengths=lengths,
                  window=window, sinks=sinks, scale=c["scale"], out=out)
    err = canopy.read_device_error(ws)
    return out.view(N, HQ, d).double().cpu().numpy(), err


def check_attend(canopy, c, window=0, sinks=0, ws=None):
    o, err = run_attend(canopy, c, window, sinks, ws)
    assert err == 0, hex(err)
    ref, weight = attend_reference(c, window, sinks)
    mine = np.concatenate([np.asarray(r, int) for r in c["rows"]])
    bound = attend_bound(c, ref[mine], weight[mine], int((c["ctxs"] + c["lens"]).max()))
    off = np.abs(o[mine] - ref[mine])
    assert (off <= bound).all(), f"{(off / bound).max():.3g} of the bound at {np.unravel_index((off / bound).argmax(), off.shape)}"
    rest = np.setdiff1d(np.arange(len(o)), mine)
    assert (o[rest] == 7.0).all()
    return o
