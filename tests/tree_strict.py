"""A comparison for drafted-tree attention that notices a lost run of tokens or a wrong mask bit in a long context."""
from __future__ import annotations

import numpy as np
import torch


def moments(step, lost=None, sees=None):
    """fp64 (out, sum_j p_j^2 v_j^2), both [T][Hq][D]. ``lost`` (sequence -> positions that nobody sees) and ``sees`` (in
    place of the step's) make a wrong result on purpose."""
    hkv, d = step.k_cache.shape[2:]
    bs, hq = step.k_cache.shape[1], step.q.shape[1]
    g = hq // hkv
    out = torch.full(step.q.shape, float("nan"), dtype=torch.float64)
    square = torch.zeros_like(out)
    for s, own in enumerate(sees or step.sees):
        q0, q1, L = int(step.query_start[s]), int(step.query_start[s + 1]), int(step.context_lens[s])
        n = q1 - q0
        if n == 0:
            continue
        t = torch.arange(L)
        slot = step.block_tables[s].long()[t // bs] * bs + t % bs
        visible = torch.cat([torch.ones(n, L - n, dtype=torch.bool), torch.from_numpy(np.array(own))], dim=1)
        if lost and s in lost:
            visible[:, lost[s]] = False
        for h in range(hkv):
            rows = []
            for pool, scale in ((step.k_cache, step.k_scale), (step.v_cache, step.v_scale)):
                x = pool.reshape(-1, hkv, d)[slot, h]
                rows.append(x.view(torch.float8_e4m3fn).double() * scale.double()[h] if step.fp8 else x.double())
            q = step.q[q0:q1, h * g:(h + 1) * g].double()
            x = (q @ rows[0].T * step.scale).masked_fill(~visible[:, None, :], -float("inf"))
            p = torch.softmax(x, 2).nan_to_num(0.0)
            out[q0:q1, h * g:(h + 1) * g] = p @ rows[1]
            square[q0:q1, h * g:(h + 1) * g] = (p * p) @ (rows[1] * rows[1])
    return out.numpy(), square.numpy()


def excess(got, ref, square, fp8):
    """Largest root mean square error of a row (a draft's head: D elements), over what roundings can make of it.

    Every weight is rounded on its own, by u = 2^-8 of itself at most (bf16; 2^-11 in f16 over e4m3 pools), its square
    by u^2 / 3 on average; the normaliser sums them unrounded. An element's error has the variance u^2 / 3 sum_j p_j^2
    v_j^2 then, and the output's rounding adds (2^-8)^2 / 3 of its own square. Over the D elements of a row the squares
    average out but for the weights they share: if one weight is nearly all, its error may be u instead of u / sqrt(3).
    Twice the root covers that. Logits and sums are in fp32: 2^-20 of the result."""
    got = np.asarray(got, dtype=np.float64)
    assert not np.isnan(got).any(), "NaN in the output"
    u = 2.0 ** -11 if fp8 else 2.0 ** -8
    var = (u * u * square + 2.0 ** -16 * ref * ref) / 3
    bound = 2 * np.sqrt(var.mean(axis=-1)) + 2.0 ** -20 * np.sqrt((ref * ref).mean(axis=-1)) + 1e-7
    return float((np.sqrt(((got - ref) ** 2).mean(axis=-1)) / bound).max())


def rounded_as_the_kernel_does(step):
    """The result with every weight rounded to bf16 or f16, against a reference between 1 and 2^-8 (bf16) or 2^-7 and
    2^-15 (f16) of the largest weight, normalised by the unrounded sum, and rounded to bf16."""
    hkv, d = step.k_cache.shape[2:]
    bs, hq = step.k_cache.shape[1], step.q.shape[1]
    g, rng = hq // hkv, np.random.default_rng(5)
    out = torch.zeros(step.q.shape, dtype=torch.float64)
    for s, own in enumerate(step.sees):
        q0, q1, L = int(step.query_start[s]), int(step.query_start[s + 1]), int(step.context_lens[s])
        if q1 == q0:
            continue
        t = torch.arange(L)
        slot = step.block_tables[s].long()[t // bs] * bs + t % bs
        visible = torch.cat([torch.ones(q1 - q0, L - q1 + q0, dtype=torch.bool), torch.from_numpy(np.array(own))], dim=1)
        for h in range(hkv):
            k, v = (x.reshape(-1, hkv, d)[slot, h] for x in (step.k_cache, step.v_cache))
            if step.fp8:
                k, v = (x.view(torch.float8_e4m3fn).double() * c.double()[h]
                        for x, c in ((k, step.k_scale), (v, step.v_scale)))
            x = (step.q[q0:q1, h * g:(h + 1) * g].double() @ k.double().T * step.scale).masked_fill(~visible[:, None, :], -float("inf"))
            top = x.amax(2, keepdim=True)
            lag = torch.from_numpy(rng.uniform(0, 8, size=tuple(top.shape))) + (7 if step.fp8 else 0)
            e = torch.exp(x - top.nan_to_num(neginf=0.0)) * 2.0 ** lag
            r = e.to(torch.float16 if step.fp8 else torch.bfloat16).double()
            o = (r @ v.double()) / e.sum(2, keepdim=True)
            out[q0:q1, h * g:(h + 1) * g] = o.nan_to_num(0.0).to(torch.bfloat16).double()
    return out.numpy()
