"""Plain fp64 forms of the speculative-decoding operators, and random steps to try them on."""
from __future__ import annotations

import dataclasses
import math

import numpy as np
import torch


def ancestors(parents):
    """Boolean [n, n]: draft i sees draft j (itself and its ancestors)."""
    n = len(parents)
    a = np.zeros((n, n), dtype=bool)
    for i in range(n):
        j = i
        while j >= 0:
            a[i, j] = True
            j = parents[j]
    return a


def pack(bools, words, garbage=None):
    """int32 [n, words]; bits past n are random where ``garbage`` is a Generator."""
    n = bools.shape[0]
    wide = np.zeros((n, words * 32), dtype=bool)
    if garbage is not None:
        wide[:] = garbage.random(wide.shape) < 0.5
    wide[:, :n] = bools
    return np.packbits(wide, axis=1, bitorder="little").view(np.int32).reshape(n, words)


@dataclasses.dataclass
class Step:
    """One verification step (CPU tensors)."""
    q: torch.Tensor
    k_cache: torch.Tensor
    v_cache: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor
    block_tables: torch.Tensor
    context_lens: torch.Tensor
    query_start: torch.Tensor
    tree_mask: torch.Tensor
    sees: list            # per sequence boolean [n, n]
    max_query_len: int
    scale: float
    fp8: bool


def make_step(seed, base, nodes, hq, hkv, d, bs, fp8=False, scale=None, kind="tree", words=None, tail_rows=0,
              spare_blocks=3):
    """A step over ``base`` committed tokens and ``nodes`` drafts per sequence. kind: "tree", "chain" or "any"
    (random bits, among them rows that see nothing). Slots that hold no token are NaN."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    base, nodes = np.asarray(base), np.asarray(nodes)
    lens = base + nodes
    need = -(-lens // bs)
    width = max(int(need.max()) if len(need) else 1, 1)
    nb = int(need.sum()) + spare_blocks
    perm = rng.permutation(nb)
    tables = np.full((len(lens), width), -1, dtype=np.int32)
    at = 0
    for s, k in enumerate(need):
        tables[s, :k] = perm[at:at + k]
        at += k
    mq = int(nodes.max()) if len(nodes) else 0
    words = words or max(-(-mq // 32), 1)
    sees, rows = [], []
    for n in nodes:
        if kind == "any":
            a = rng.random((n, n)) < 0.4
            a[rng.random(n) < 0.25] = False
        else:
            parents = [i - 1 if kind == "chain" else int(rng.integers(-1, i)) if i else -1 for i in range(n)]
            a = ancestors(parents)
        sees.append(a)
        rows.append(pack(a, words, rng))
    total = int(nodes.sum()) + tail_rows
    mask = np.concatenate(rows + [np.zeros((tail_rows, words), dtype=np.int32)])
    shape = (nb, bs, hkv, d)
    live = torch.zeros(nb * bs, dtype=torch.bool)
    for s, L in enumerate(lens):
        t = np.arange(L)
        live[torch.from_numpy(tables[s, t // bs].astype(np.int64) * bs + t % bs)] = True
    dead = ~live.view(nb, bs)
    if fp8:
        pools = []
        for _ in range(2):
            c = (torch.randint(0, 2, shape, generator=gen) << 7) | torch.randint(32, 96, shape, generator=gen)
            c = c.to(torch.uint8)
            c[dead] = 0x7F
            pools.append(c)
    else:
        pools = []
        for _ in range(2):
            c = torch.randn(shape, generator=gen).to(torch.bfloat16)
            c[dead] = float("nan")
            pools.append(c)
    h = torch.arange(hkv, dtype=torch.float32)
    return Step(q=torch.randn(total, hq, d, generator=gen).to(torch.bfloat16), k_cache=pools[0], v_cache=pools[1],
                k_scale=2.0 ** -4 * (1 + h / hkv), v_scale=2.0 ** -4 * (1 + h / (2 * hkv)),
                block_tables=torch.from_numpy(tables), context_lens=torch.from_numpy(lens.astype(np.int32)),
                query_start=torch.from_numpy(np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)),
                tree_mask=torch.from_numpy(mask), sees=sees, max_query_len=mq,
                scale=1.0 / math.sqrt(d) if scale is None else scale, fp8=fp8)


def attention(step, skip=()):
    """(out, sum_j p_j |v_j|) in fp64, both [T][Hq][D]; rows of no sequence stay NaN."""
    hkv, d = step.k_cache.shape[2:]
    bs, hq = step.k_cache.shape[1], step.q.shape[1]
    g = hq // hkv
    out = torch.full(step.q.shape, float("nan"), dtype=torch.float64)
    spread = torch.zeros_like(out)
    for s in range(len(step.sees)):
        if s in skip:
            continue
        q0, q1, L = int(step.query_start[s]), int(step.query_start[s + 1]), int(step.context_lens[s])
        n = q1 - q0
        if n == 0:
            continue
        t = torch.arange(L)
        slot = step.block_tables[s].long()[t // bs] * bs + t % bs
        rows = []
        for pool, scale in ((step.k_cache, step.k_scale), (step.v_cache, step.v_scale)):
            x = pool.reshape(-1, hkv, d)[slot]
            rows.append(x.view(torch.float8_e4m3fn).double() * scale.double()[None, :, None] if step.fp8
                        else x.double())
        sees = torch.cat([torch.ones(n, L - n, dtype=torch.bool), torch.from_numpy(step.sees[s])], dim=1)
        for i in range(n):
            j = torch.nonzero(sees[i])[:, 0]
            for h in range(hq):
                if len(j) == 0:
                    out[q0 + i, h] = 0
                    continue
                x = rows[0][j, h // g] @ step.q[q0 + i, h].double() * step.scale
                p = torch.softmax(x, 0)
                out[q0 + i, h] = p @ rows[1][j, h // g]
                spread[q0 + i, h] = p @ rows[1][j, h // g].abs()
    return out.numpy(), spread.numpy()


def assert_close(got, ref, spread, fp8, what=""):
    """bf16 results against fp64. The output is rounded once (half a step: 2^-8 of it). The weights are rounded to
    bf16 (2^-8 each; over an e4m3 cache to fp16, 2^-11), which moves the weighted sum by that share of
    sum_j p_j |v_j| and the normaliser by the same share of the result. Logits come from exact products summed in
    fp32, and the base-2 exponential is good to about 2^-22: a quarter on top covers both and second orders."""
    got = np.asarray(got, dtype=np.float64)
    assert not np.isnan(got).any(), f"{what}: NaN in the output"
    w = 2.0 ** -11 if fp8 else 2.0 ** -8
    bound = 1.25 * (2.0 ** -8 * np.abs(ref) + w * (spread + np.abs(ref))) + 1e-6
    err = np.abs(got - ref)
    bad = err > bound
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} off, worst {np.max(err / bound):.2f} of the bound "
                           f"at {np.argwhere(bad)[0].tolist()}")
