"""Speculative-decoding operators at the edges of what their documentation allows.
References and tolerances as in test_gpu_spec."""
import numpy as np
import pytest
import torch

import spec_ref
from long_context_fp8_b200 import dsa
from test_gpu_spec import (INVALID, WORKSPACE, _check_tree, _check_verify, _dev, _run_pool, _run_tree, _run_verify, _status,
                           _Step, _tree_case)

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

# ------------------------------------------------------------------ steps of fixed buffers over ragged drafts

class _Ragged(_Step):
    """A step whose buffers hold the most tokens that any step may have: sequences bring 0 to n drafts, and the rows
    behind the last token are padding."""

    def fill_ragged(self, seed):
        self.fill(seed)
        rng = np.random.default_rng(100 + seed)
        self.ns = rng.integers(0, self.n + 1, self.B)
        self.ns[seed % self.B], self.ns[(seed + 1) % self.B] = 0, self.n
        parents, depth = np.full(self.N, 99), np.full(self.N, -7)
        at = 0
        for n in self.ns:
            for i in range(n):
                parents[at + i] = -1 if i == 0 else rng.integers(max(0, i - 3), i)
                depth[at + i] = 0 if i == 0 else depth[at + parents[at + i]] + 1
            at += n
        self.start = np.append([0], np.cumsum(self.ns))
        self.new.copy_(_dev(self.ns))
        self.parents.copy_(_dev(parents))
        self.depth.copy_(_dev(depth))
        self.q[at:] = float("nan")
        self.target[at:] = float("nan")

    def run(self):
        start, pool = self.plan["token_start"], self.pool
        dsa.dsa_blocks_extend(pool, self.new, self.ps, self.P, self.N, plan=self.plan, status=self.status)
        prefix = (pool["context_lens"] - (start[1:] - start[:-1]))[self.plan["seq_ids"].long().clamp(min=0)]
        dsa.dsa_rope(self.q, prefix + self.depth, self.table, k=self.k, rot_begin=64, interleaved=True, q_out=self.qr,
                     k_out=self.kr)
        bt = pool["block_table"]
        self.append(self.caches, self.kidx, self.kr.view(self.N, -1), self.v, self.plan["seq_ids"],
                    self.plan["positions"], bt, status=self.status)
        inp = dict(q=self.qr, block_table=bt, context_lens=pool["context_lens"], token_start=start, parents=self.parents,
                   **{k: v for k, v in self.caches.items() if k[0] in "kv" and k[1] == "_"})
        dsa.dsa_tree_attn(inp, self.n, self.max_context, out=self.out, lse=self.lse, ws=self.ws)
        dsa.dsa_verify_tree(self.target, self.draft, self.tokens, self.parents, start, self.ua, self.us, path=self.path,
                            accept_len=self.acc, next_token=self.next, status=self.status)
        dsa.dsa_cache_compact(self.caches, bt, pool["context_lens"], start, self.path, self.acc, N=self.N,
                              keep_lens=self.keep, status=self.status)
        dsa.dsa_blocks_trim(pool, self.keep, self.ps, self.P, status=self.status)


@pytest.mark.parametrize("kv8", [False, True])
def test_steps_of_fixed_buffers_over_ragged_drafts(kv8):
    """One graph for every step, with as many rows as the largest: padding rows are no tokens to any operator, and
    none of them is reported."""
    B, ps, n, H, V = 5, 16, 7, 16, 300
    s = _Ragged(B, ps, 12, 70, n, H, V, kv8)
    rows = [[] for _ in range(B)]
    graph = None
    for seed in range(6):
        s.fill_ragged(seed)
        s.out.fill_(3.0)
        s.lse.fill_(3.0)
        if graph is None:
            s.run()                                          # the library loads its kernels before the capture
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert int(s.status.item()) == 0 and dsa.dsa_stream_status(s.ws) == 0
        total, start = int(s.start[-1]), s.start
        assert torch.all(s.plan["seq_ids"][total:] == -1) and torch.all(s.plan["positions"][total:] == -1)
        assert torch.all(s.out[total:] == 3.0) and torch.all(s.lse[total:] == 3.0)
        _check_verify((s.target.cpu().numpy(), s.draft.cpu().numpy(), s.tokens.cpu().numpy(), s.parents.cpu().numpy(),
                       start, s.ua.cpu().numpy(), s.us.cpu().numpy()), n, (s.path, s.acc, s.next))
        acc, path = s.acc.cpu().numpy(), s.path.cpu().numpy()
        for b in range(B):
            t = slice(int(start[b]), int(start[b + 1]))
            assert (acc[b] == 0) == (s.ns[b] == 0)
            if s.ns[b]:
                K, Vv = (torch.cat([torch.stack([r[j] for r in rows[b]]), new[t]]) if rows[b] else new[t]
                         for j, new in enumerate((s.kr[:, 0], s.v)))
                if kv8:
                    K, Vv = ((c.view(torch.float8_e4m3fn).double() * sc.double()[:, None]) for c, sc in
                             (dsa.dsa_quantize_e4m3(x.contiguous()) for x in (K, Vv)))
                ro, rl, to, tl = spec_ref.tree_attn(s.qr[t].double().cpu().numpy(), K.double().cpu().numpy()[:, None],
                                                    Vv.double().cpu().numpy()[:, None], len(K),
                                                    s.parents[t].cpu().numpy(), H, 128 ** -0.5)
                assert np.all(np.abs(s.out[t].double().cpu().numpy() - ro) <= to)
                assert np.all(np.abs(s.lse[t].double().cpu().numpy() - rl) <= tl)
            for i in range(acc[b]):
                at = int(start[b]) + int(path[b, i])
                rows[b].append((s.kr[at, 0].clone(), s.v[at].clone(), s.kidx[at].clone()))
        ctx, held, bt = (s.pool[k].cpu().numpy() for k in ("context_lens", "pages_held", "block_table"))
        count, free = int(s.pool["free_count"].item()), s.pool["free_pages"].cpu().numpy()
        assert [len(r) for r in rows] == list(ctx) and np.array_equal(held, -(-ctx // ps))
        pages = np.concatenate([free[:count]] + [bt[b, :held[b]] for b in range(B)])
        assert np.array_equal(np.sort(pages), np.arange(70))
        for b in range(B):
            at = np.arange(ctx[b])
            slot = torch.from_numpy(bt[b, at // ps].astype(np.int64) * ps + at % ps).cuda()
            if len(at):
                want = torch.stack([r[2] for r in rows[b]])
                assert torch.equal(s.caches["kidx_cache"].flatten(0, 1)[slot], dsa.dsa_quantize_e4m3(want)[0])
        if graph is None:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                s.run()


@pytest.mark.parametrize("kv8", [False, True])
def test_append_reports_tokens_that_may_not_be_beside_padding(kv8):
    """Only sequence -1 at position -1 is padding: one of the two alone is reported, as before."""
    s = _Step(2, 16, 4, 8, 4, 4, 10, kv8)
    s.pool["block_table"][:, 0] = torch.tensor([2, 5], dtype=torch.int32, device="cuda")
    s.fill(1)
    before = {k: v.clone() for k, v in s.caches.items()}
    for seq, pos, want in (([-1] * 8, [-1] * 8, 0), ([-1] * 7 + [0], [-1] * 8, INVALID), ([-1] * 8, [-1] * 7 + [0], INVALID),
                           ([-1] * 7 + [-2], [-1] * 8, INVALID)):
        st = _status()
        s.append(s.caches, s.kidx, s.k.view(8, -1), s.v, _dev(seq), _dev(pos), s.pool["block_table"], status=st)
        assert int(st.item()) == want
        assert all(torch.equal(s.caches[k], v) for k, v in before.items())

# ------------------------------------------------------------------ several K/V heads

def test_grouped_heads_through_append_attention_and_compaction():
    """bf16 caches of several K/V heads: appended as rows of H_kv * d, attended, compacted in their own shape, and
    attended again over what was accepted."""
    rng = np.random.default_rng(61)
    B, P, ps, H, Hkv, d = 3, 40, 16, 8, 4, 64
    ns, first = np.array([5, 3, 7]), np.array([30, 0, 61])
    N, start = int(ns.sum()), np.append([0], np.cumsum(ns))
    K, V = (torch.from_numpy(rng.standard_normal((B, 80, Hkv, d))).bfloat16() for _ in range(2))
    pool = dict(block_table=torch.full((B, 6), -1, dtype=torch.int32, device="cuda"), context_lens=_dev(np.zeros(B)),
                pages_held=_dev(np.zeros(B)), free_pages=_dev(rng.permutation(P)), free_count=_dev([P]))
    caches = dict(kidx_cache=torch.zeros((P, ps, 128), dtype=torch.uint8, device="cuda"),
                  kscale_cache=torch.zeros((P, ps), device="cuda"),
                  k_cache=torch.zeros((P, ps, Hkv, d), dtype=torch.bfloat16, device="cuda"),
                  v_cache=torch.zeros((P, ps, Hkv, d), dtype=torch.bfloat16, device="cuda"))
    rows = {**caches, "k_cache": caches["k_cache"].view(P, ps, Hkv * d), "v_cache": caches["v_cache"].view(P, ps, Hkv * d)}

    def append(lens):
        plan = dsa.dsa_blocks_extend(pool, _dev(lens), ps, P, int(np.sum(lens)))
        seq, pos = plan["seq_ids"].cpu().long(), plan["positions"].cpu().long()
        st = _status()
        dsa.dsa_cache_append(rows, torch.randn((len(seq), 128)).bfloat16().cuda(), K[seq, pos].flatten(1).cuda(),
                             V[seq, pos].flatten(1).cuda(), plan["seq_ids"], plan["positions"], pool["block_table"], status=st)
        assert int(st.item()) == 0
        return plan

    def attend(lens, parents, q):
        inp = dict(q=q.cuda(), k_cache=caches["k_cache"], v_cache=caches["v_cache"], block_table=pool["block_table"],
                   context_lens=pool["context_lens"], token_start=_dev(np.append([0], np.cumsum(lens))), parents=_dev(parents))
        return dsa.dsa_tree_attn(inp, 7, 96)

    def check(out, lse, kv, ctxs, lens, parents, q):
        at = 0
        for b, n in enumerate(lens):
            t = slice(at, at + n)
            ro, rl, to, tl = spec_ref.tree_attn(q[t].double().numpy(), kv[0][b].double().numpy(), kv[1][b].double().numpy(),
                                                int(ctxs[b]), parents[t], H // Hkv, d ** -0.5)
            assert np.all(np.abs(out[t].double().cpu().numpy() - ro) <= to)
            assert np.all(np.abs(lse[t].double().cpu().numpy() - rl) <= tl)
            at += n

    append(first)
    plan = append(ns)
    parents = np.concatenate([[-1] + [int(rng.integers(max(0, i - 2), i)) for i in range(1, n)] for n in ns])
    q = torch.from_numpy(rng.standard_normal((N, H, d))).bfloat16()
    check(*attend(ns, parents, q), [[x[b, :first[b] + n] for b, n in enumerate(ns)] for x in (K, V)], first + ns, ns,
          parents, q)
    path = np.array([[0, 2, 4], [0, 1, -1], [0, 3, 6]])
    acc = np.array([3, 2, 3])
    st = _status()
    keep = dsa.dsa_cache_compact(caches, pool["block_table"], pool["context_lens"], plan["token_start"], _dev(path),
                                 _dev(acc), N=N, status=st)
    assert int(st.item()) == 0 and np.array_equal(keep.cpu().numpy(), first + acc)
    dsa.dsa_blocks_trim(pool, keep, ps, P)
    # what was accepted, in order; one more token each
    kept = [[x[b, list(range(first[b])) + [first[b] + p for p in path[b, :acc[b]]]] for b in range(B)] for x in (K, V)]
    for b in range(B):
        for x, rest in zip((K, V), kept):
            x[b, :len(rest[b])] = rest[b]
    append(np.ones(B, int))
    q = torch.from_numpy(rng.standard_normal((B, H, d))).bfloat16()
    ctxs = first + acc + 1
    check(*attend(np.ones(B, int), np.full(B, -1), q), [[x[b, :ctxs[b]] for b in range(B)] for x in (K, V)], ctxs, [1] * B,
          np.full(B, -1), q)


def test_compaction_takes_the_attention_caches_of_one_head():
    """FP8 caches [P, page_size, 1, d] with their scales move like [P, page_size, d]; more heads are refused."""
    rng = np.random.default_rng(62)
    bt, ctx, start, path, acc = _dev([[3, 1]]), _dev([20]), _dev([0, 6]), _dev([[0, 2, 5]]), _dev([3])

    def caches(*heads):
        c = {x + "_cache": torch.from_numpy(rng.integers(0, 256, (5, 16, *heads, 64)).astype(np.uint8)).cuda() for x in "kv"}
        c.update({x + "_cache_scale": torch.from_numpy(rng.random((5, 16, *heads)).astype(np.float32)).cuda() for x in "kv"})
        return c

    four = caches(1)
    three = {k: v.squeeze(2).clone() for k, v in four.items()}
    keep = [dsa.dsa_cache_compact(c, bt, ctx, start, path, acc) for c in (four, three)]
    assert torch.equal(keep[0], keep[1]) and keep[0].tolist() == [17]
    for k, v in three.items():
        assert torch.equal(four[k].squeeze(2), v)
    with pytest.raises(ValueError, match="one K/V head"):
        dsa.dsa_cache_compact(caches(2), bt, ctx, start, path, acc)

# ------------------------------------------------------------------ a pool without a stack

def test_blocks_of_a_pool_whose_pages_are_all_in_the_tables():
    """No free pages and no room for any: sequences grow and shrink within what they hold, the rest is refused."""
    pool = dict(block_table=np.array([[3, 1, 4], [0, 5, -1], [2, -1, -1]]), context_lens=np.array([10, 0, 16]),
                pages_held=np.array([3, 2, 1]), free_pages=np.zeros(0, int), free_count=np.array([0]))
    dev, plan, st = _run_pool(pool, np.array([30, 32, 1]), 16, 6, 70)
    ref_plan, err = spec_ref.extend(pool, np.array([30, 32, 1]), 16, 6, 70)
    assert err and st == WORKSPACE
    for got, ref in ((dev, pool), (plan, ref_plan)):
        for k, v in ref.items():
            assert np.array_equal(got[k].cpu().numpy(), v), k
    keep, st = np.array([33, 30, 16]), _status()             # the third trim gives nothing back
    dsa.dsa_blocks_trim(dev, _dev(keep), 16, 6, status=st)
    assert not spec_ref.trim(pool, keep, 16, 6) and int(st.item()) == 0
    for k, v in pool.items():
        assert np.array_equal(dev[k].cpu().numpy(), v), k


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
