"""The speculative-decoding entry points on a host without a GPU: bad arguments are
rejected before any CUDA call, and the plain forms the GPU tests use are themselves right."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_377_b200 as pkv
from paged_kv_cache_377_b200 import tree
from tree_reference import ancestors, attention, make_step, pack

P = ctypes.c_void_p(4096)  # a non-null, aligned address: argument checks never dereference it
ODD = ctypes.c_void_p(4098)


def err():
    return pkv.library().pkv_last_error().decode()


def _tree(fp8=False, **kw):
    a = dict(out=P, q=P, k=P, v=P, ks=P, vs=P, bt=P, cl=P, qs=P, mask=P, words=1, S=4, T=20, mq=8, Hq=4, Hkv=2, D=64,
             bs=16, scale=0.125, MB=4, NB=16, ws=P, wsb=1 << 30)
    a.update(kw)
    head = [a["out"], a["q"], a["k"], a["v"]] + ([a["ks"], a["vs"]] if fp8 else [])
    rest = [a[x] for x in ("bt", "cl", "qs", "mask", "words", "S", "T", "mq", "Hq", "Hkv", "D", "bs", "scale", "MB", "NB",
                           "ws", "wsb")]
    lib = tree._lib()
    return (lib.paged_attn_tree_fp8 if fp8 else lib.paged_attn_tree)(*head, *rest, None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,code,msg", [
    (dict(q=None), -1, "NULL"), (dict(mask=None), -1, "NULL"), (dict(ws=None), -1, "NULL"), (dict(S=-1), -1, "num_seqs"),
    (dict(mq=-1), -1, "max_query_len"), (dict(words=0), -1, "mask_words"), (dict(mq=33), -1, "mask_words"),
    (dict(mq=4097, words=1000), -2, "exceeds"), (dict(Hq=5), -1, "multiple"), (dict(Hq=18), -2, "exceeds"),
    (dict(D=96), -2, "head_dim"), (dict(bs=8), -2, "block_size"), (dict(scale=float("nan")), -1, "scale"),
    (dict(q=ODD), -1, "aligned"), (dict(ws=ctypes.c_void_p(4112)), -1, "aligned"), (dict(wsb=16), -1, "workspace_bytes"),
    (dict(NB=1 << 28), -1, "2^31"), (dict(MB=1 << 28), -1, "2^31")])
def test_tree_attention_rejects_bad_arguments(kw, code, msg, fp8):
    assert _tree(fp8, **kw) == code and msg in err(), err()


@pytest.mark.parametrize("kw", [dict(ks=None), dict(vs=None)])
def test_the_scales_are_required_over_e4m3_pools(kw):
    assert _tree(True, **kw) == -1 and "NULL" in err()


@pytest.mark.parametrize("kw", [dict(S=0), dict(T=0), dict(mq=0)])
def test_empty_steps_are_no_ops(kw):
    assert _tree(**kw) == 0


def test_workspace_sizes():
    assert pkv.tree_workspace_bytes(128) >= pkv.tree_workspace_bytes(64) >= 256
    with pytest.raises(pkv.PagedKVError, match="head_dim"):
        pkv.tree_workspace_bytes(96)


@pytest.mark.parametrize("at,bad,msg", [(0, None, "NULL"), (3, None, "NULL"), (4, -1, "num_seqs"), (6, 64, "mask_words"),
                                        (6, 5000, "exceeds"), (7, 0, "mask_words"), (8, None, "NULL")])
def test_mask_rejects_bad_arguments(at, bad, msg):
    args = [P, P, P, P, 4, 20, 8, 1, P, None]
    args[at] = bad
    assert tree._lib().paged_tree_mask(*args) < 0 and msg in err(), err()


@pytest.mark.parametrize("at,bad,msg", [(0, None, "NULL"), (4, None, "NULL"), (9, -1, "num_seqs"), (10, -1, "num_s"),
                                        (10, (1 << 30) + 1, "num_slots"), (11, 0, "positive"), (12, 0, "positive"),
                                        (13, 0, "positive"), (13, 1 << 28, "2^31"), (14, None, "NULL")])
def test_grow_rejects_bad_arguments(at, bad, msg):
    args = [P] * 9 + [4, 20, 8, 16, 64, P, None]
    args[at] = bad
    assert tree._lib().kv_tables_grow(*args) == -1 and msg in err(), err()


@pytest.mark.parametrize("at,bad,msg", [(0, None, "NULL"), (5, None, "NULL"), (6, -1, "num_seqs"), (7, 0, "positive"),
                                        (8, 0, "positive"), (9, 1 << 28, "2^31"), (10, None, "NULL")])
def test_trim_rejects_bad_arguments(at, bad, msg):
    args = [P] * 6 + [4, 8, 16, 64, P, None]
    args[at] = bad
    assert tree._lib().kv_tables_trim(*args) == -1 and msg in err(), err()


@pytest.mark.parametrize("at,bad,msg", [(0, None, "NULL"), (5, None, "NULL"), (8, -1, "num_seqs"), (9, -1, "max_accepted"),
                                        (10, 0, "positive"), (11, 4, "16 bytes"), (12, 4, "elem_bytes"), (1, ODD, "aligned"),
                                        (7, P, "new_lens"), (15, 1 << 28, "2^31"), (10, 1 << 20, "2^26")])
def test_keep_rejects_bad_arguments(at, bad, msg):
    args = [P, P, P, P, P, P, P, ctypes.c_void_p(8192), 4, 8, 2, 64, 2, 16, 8, 64, P, None]
    args[at] = bad
    assert tree._lib().kv_cache_keep(*args) < 0 and msg in err(), err()


def test_wrappers_refuse_host_tensors():
    t = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_attn_tree(t, t, t, t, t, t, t, t, 1, 1.0, t)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.kv_tables_trim(i.view(2, 2), i, i, i, i, i, 16, i)


# ---------------------------------------------------------------- the plain forms themselves

def test_ancestors_of_a_small_tree():
    #   0        3
    #   |- 1
    #   |- 2 - 4
    a = ancestors([-1, 0, 0, -1, 2])
    assert a.astype(int).tolist() == [[1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 0, 1, 0, 0], [0, 0, 0, 1, 0], [1, 0, 1, 0, 1]]
    assert pack(a, 1)[:, 0].tolist() == [1, 3, 5, 8, 21]


@pytest.mark.parametrize("fp8", [False, True])
def test_plain_attention_of_a_chain_is_causal_attention(fp8):
    step = make_step(3, [20, 0, 33], [5, 7, 1], 4, 2, 64, 16, fp8=fp8, kind="chain")
    out, spread = attention(step)
    for s in range(3):
        q0, q1, L = int(step.query_start[s]), int(step.query_start[s + 1]), int(step.context_lens[s])
        t = torch.arange(L)
        rows = []
        for pool, sc in ((step.k_cache, step.k_scale), (step.v_cache, step.v_scale)):
            x = pool[step.block_tables[s].long()[t // 16], t % 16]
            rows.append((x.view(torch.float8_e4m3fn).double() * sc.double()[:, None] if fp8 else x.double())
                        .transpose(0, 1).repeat_interleave(2, 0))
        mask = torch.ones(q1 - q0, L, dtype=torch.bool).tril(L - (q1 - q0))
        want = torch.nn.functional.scaled_dot_product_attention(
            step.q[q0:q1].double().transpose(0, 1), *rows, attn_mask=mask, scale=step.scale).transpose(0, 1)
        np.testing.assert_allclose(out[q0:q1], want.numpy(), rtol=1e-12, atol=1e-12)
    assert (spread >= np.abs(out) - 1e-12).all()


def test_plain_rows_that_see_nothing_are_zero():
    step = make_step(5, [0, 3], [6, 2], 2, 1, 64, 16, kind="any")
    step.sees[0][2] = False
    out, _ = attention(step)
    assert (out[2] == 0).all() and np.abs(out[6:]).max() > 0
