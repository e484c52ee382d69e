"""Speculative-decoding operators at the edges of what their documentation allows.
References and tolerances as in test_gpu_spec."""
import numpy as np
import pytest
import torch

from long_context_fp8_b200 import dsa
from test_gpu_spec import _run_tree, _tree_case

pytestmark = pytest.mark.gpu

TIMEOUT = 5


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
