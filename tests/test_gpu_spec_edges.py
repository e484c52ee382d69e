"""Speculative-decoding operators at the edges of what their documentation allows.
References and tolerances as in test_gpu_spec."""
import numpy as np
import pytest
import torch

import spec_ref
from long_context_fp8_b200 import dsa
from test_gpu_spec import _check_tree, _check_verify, _dev, _run_tree, _run_verify, _tree_case

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


# ------------------------------------------------------------------ peaked targets

def _peaked(V, left, depth, ratio, u_last, rng):
    """A root whose first `depth` children are point masses that each take all but `left` of what is left of the
    target; one more child takes `ratio` of the rest."""
    tokens = rng.permutation(V)[:depth + 1]
    P = np.zeros((depth + 2, V))
    rest = 1.0
    for x in tokens[:depth]:
        P[0, x] = rest * (1.0 - left)
        rest *= left
    others = np.setdiff1d(np.arange(V), tokens)
    w = rng.random(len(others)) + 0.1
    P[0, others] = rest * (1.0 - ratio) * w / w.sum()
    P[0, tokens[depth]] = rest * ratio
    P[1:] = 1.0 / V
    n = depth + 2
    u = np.full(n, 1.0 - 2.0 ** -24)                         # above 1 - left: rejected
    u[depth + 1] = u_last
    return P.astype(np.float32), np.append([0], tokens), np.array([-1] + [0] * (n - 1)), u.astype(np.float32)


@pytest.mark.parametrize("B", [1, 9, 60, 500])
@pytest.mark.parametrize("left", [6e-6, 2.0 ** -12, 0.1])
def test_verify_peaked_targets_with_point_masses(left, B):
    """Siblings that each leave little of the target: the sums after them keep their 64 bits, so the next child is
    accepted or not as the definition has it, in batches of any size."""
    V = 1003
    rng = np.random.default_rng(5)
    for depth in range(1, 8):
        if left ** depth < 1e-30:
            break
        # the child's weight is `ratio` of the rest up to the roundings of P to fp32 (2^-24 each): u a few of them
        # below and above it decides
        for u_last in (0.5 - 2.0 ** -18, 0.5 + 2.0 ** -18):
            P, tokens, parents, u = _peaked(V, left, depth, 0.5, u_last, rng)
            n = len(tokens)
            case = (np.tile(P, (B, 1)), None, np.tile(tokens, B), np.tile(parents, B), np.arange(B + 1) * n,
                    np.tile(u, B), np.linspace(0.0, 0.999, B).astype(np.float32))
            got = _run_verify(*case)
            _check_verify(case, 128, got)
            want = [0, depth + 1] if u_last < 0.5 else [0]
            assert [int(v) for v in got[0][0] if v >= 0] == want


# ------------------------------------------------------------------ idle sequences

def _ms(call, times=5):
    call()
    best = float("inf")
    for _ in range(times):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@pytest.mark.parametrize("B,max_tokens", [(1000, 64), (1000, 5000), (60000, 64), (200000, 5000)])
def test_blocks_extend_over_idle_sequences(B, max_tokens):
    """Runs of sequences that do not grow lie between the tokens of one group of four."""
    new = np.zeros(B, int)
    new[[0, 1, B // 2, B - 2, B - 1]] = [3, 2, 1, 4, 2]
    pool = dict(block_table=np.full((B, 1), -1), context_lens=np.zeros(B, int), pages_held=np.zeros(B, int),
                free_pages=np.arange(20), free_count=np.array([20]))
    dev = {k: _dev(v) for k, v in pool.items()}
    first = {k: v.clone() for k, v in dev.items()}
    plan = dsa.dsa_blocks_extend(dev, _dev(new), 16, 20, max_tokens)
    ref_plan, err = spec_ref.extend(pool, new, 16, 20, max_tokens)
    assert not err
    for got, ref in ((dev, pool), (plan, ref_plan)):
        for k, v in ref.items():
            assert np.array_equal(got[k].cpu().numpy(), v), k

    def call(lens):
        for k, v in first.items():
            dev[k].copy_(v)
        dsa.dsa_blocks_extend(dev, lens, 16, 20, max_tokens, plan=plan)

    # the same tokens in one run of sequences: the gaps cost a search each, no walk
    near = np.zeros(B, int)
    near[:5] = new[new > 0]
    near_dev, far_dev = _dev(near), _dev(new)
    ms_near, ms_far = _ms(lambda: call(near_dev)), _ms(lambda: call(far_dev))
    assert ms_far < 2.0 * ms_near + 0.02, (ms_near, ms_far)


@pytest.mark.parametrize("kv8", [False, True])
def test_tree_attn_over_many_idle_sequences(kv8):
    """Tens of thousands of sequences of which three have drafts, far apart."""
    rng = np.random.default_rng(41)
    inp, vals = _tree_case(rng, [3, 2, 4], [300, 700, 90], 16, 1, 128, 64, kv8)
    B, at = 60000, [0, 29999, 59999]
    n = np.zeros(B, int)
    n[at] = [3, 2, 4]
    ctx = np.full(B, -5)                                     # nothing is checked where there are no drafts
    ctx[at] = [300, 700, 90]
    bt = np.full((B, inp["block_table"].shape[1]), -1)
    bt[at] = inp["block_table"].numpy()
    dev = {k: v.cuda() for k, v in inp.items()}
    dev.update(block_table=_dev(bt), context_lens=_dev(ctx), token_start=_dev(np.append([0], np.cumsum(n))))
    ws = dsa.workspace(dsa.tree_attn_workspace_size(B, 9, 16, 1, 128), "cuda")
    out, lse = dsa.dsa_tree_attn(dev, 4, 700, ws=ws)
    assert dsa.dsa_stream_status(ws) == 0
    _check_tree(inp, vals, out, lse, 128 ** -0.5)
    ms = _ms(lambda: dsa.dsa_tree_attn(dev, 4, 700, out=out, lse=lse, ws=ws))
    assert ms < 2.0, ms


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
