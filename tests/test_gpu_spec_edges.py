"""Speculative-decoding operators at the edges of what their documentation allows.
References and tolerances as in test_gpu_spec."""
import numpy as np
import pytest
import torch

import spec_ref
from long_context_fp8_b200 import dsa
from test_gpu_spec import _run_tree, _tree_case

pytestmark = pytest.mark.gpu

TIMEOUT = 5


# ------------------------------------------------------------------ queries that are not finite

@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("ns,ctxs,H", [
    ([1, 1, 1], [1, 2, 40], 16),               # a row's only logits lie beside masked ones
    ([4, 3], [60, 64], 16),                    # within the first step of 64 positions
    ([9], [70], 128),                          # pairs of tiles
    ([2, 3], [129, 3000], 256),                # a token of two tiles; cut items
    ([40], [5000], 16),
])
def test_tree_attn_queries_that_are_not_finite(ns, ctxs, H, kv8):
    """NaN, +inf, and -inf against K of one sign, whose logits are all -inf: NaN in their own row and head
    (softmax of nothing but -inf is 0 / 0), zeros in a padding row, and the same bits everywhere else."""
    rng = np.random.default_rng(31 + sum(ctxs))
    inp, vals = _tree_case(rng, ns, ctxs, H, 1, 128, 32, kv8)
    K = inp["k_cache"]
    if kv8:
        K[..., 7] = (K[..., 7] & 0x37) | 8                   # positive and not zero
    else:
        K[..., 7] = 1.5
    N = sum(ns)
    if N > 3:
        inp["parents"][3] = -2                               # a padding row (and rows under it)
    pad = torch.zeros(N, dtype=torch.bool)
    at = 0
    for n in ns:
        pad[at:at + n] = torch.tensor([a is None for a in spec_ref.ancestors(inp["parents"][at:at + n].numpy())])
        at += n
    base, base_lse = _run_tree(inp)
    assert torch.isfinite(base).all() and torch.isfinite(base_lse[~pad]).all()
    for value, where in ((float("nan"), (0, 5)), (float("-inf"), (0, 7)), (float("inf"), (0, 7)), (float("-inf"), (1, 7))):
        bad = dict(inp, q=inp["q"].clone())
        hit = torch.zeros(N, H, dtype=torch.bool)
        hit[:, where[0]::3] = True
        bad["q"][..., where[1]] = torch.where(hit, torch.tensor(value, dtype=torch.bfloat16), bad["q"][..., where[1]])
        out, lse = (x.cpu() for x in _run_tree(bad))
        nan = hit & ~pad[:, None]
        assert torch.isnan(out[nan]).all() and torch.isnan(lse[nan]).all(), (value, where)
        assert torch.equal(out[~nan], base.cpu()[~nan]) and torch.equal(lse[~nan], base_lse.cpu()[~nan]), (value, where)
        assert torch.all(out[pad] == 0) and torch.isneginf(lse[pad]).all()


# ------------------------------------------------------------------ bounded waits

@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("items", ["short", "long", "pair"])
def test_tree_attn_waits_run_out_then_the_next_call_is_exact(items, d, kv8):
    """The library's hook withholds copies in CTA 0, so that its roles wait for what never comes: every wait gives
    up, the call reports DSA_ERR_TIMEOUT, and the next one on the same workspace returns the bits of an
    undisturbed call.  Single tiles (whose two sets exchange statistics) in several items and in one, and pairs."""
    rng = np.random.default_rng(51)
    ns, ctxs, H = {"short": ([2] * 600, [int(v) for v in rng.integers(2, 200, 600)], 16),
                   "long": ([3], [70000], 16), "pair": ([9], [70000], 32)}[items]
    inp, _ = _tree_case(rng, ns, ctxs, H, 1, d, 64, kv8)
    ws = dsa.workspace(dsa.tree_attn_workspace_size(len(ns), sum(ns), H, 1, d), "cuda")
    out, lse = _run_tree(inp, ws=ws)
    assert dsa.dsa_stream_status(ws) == 0
    dsa.test_stall_next(dsa.STALL_TREE_ATTN)
    _run_tree(inp, ws=ws)
    assert dsa.dsa_stream_status(ws) == TIMEOUT
    again, again_lse = _run_tree(inp, ws=ws)
    assert dsa.dsa_stream_status(ws) == 0
    assert torch.equal(again, out) and torch.equal(again_lse, lse)


def test_tree_attn_stall_can_be_disarmed():
    inp, _ = _tree_case(np.random.default_rng(52), [3], [70000], 16, 1, 128, 64, False)
    ws = dsa.workspace(dsa.tree_attn_workspace_size(1, 3, 16, 1, 128), "cuda")
    dsa.test_stall_next(dsa.STALL_TREE_ATTN)
    dsa.test_stall_next(dsa.STALL_NONE)
    _run_tree(inp, ws=ws)
    assert dsa.dsa_stream_status(ws) == 0
