"""Parity of the speculative-decoding operators (rotary positions, block tables,
tree attention, verification, compaction; through the C ABI) with plain 64-bit
references.

Bars: whole numbers and moved bytes equal; rotary values within the fp32 roundings
of two products of sine and cosine, attention within the roundings of bf16 weights
and fp32 sums that spec_ref.tree_attn adds up row by row, plus one rounding of the
output type."""
import numpy as np
import pytest
import torch

import spec_ref
from long_context_fp8_b200 import dsa

pytestmark = pytest.mark.gpu

INVALID, WORKSPACE = 1, 3
F32_STEP, BF16_STEP = 2.0 ** -24, 2.0 ** -8


def _dev(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x)).to(dtype).cuda()


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ rotary positions

ROPE_CASES = [
    # rows, H_q, H_k, d, begin, rot, interleaved, scaling, dtype, inverse
    (1, 1, 0, 64, 0, 64, False, "none", torch.float32, False),
    (1, 1, 1, 64, 0, 64, True, "none", torch.bfloat16, False),
    (1, 128, 1, 128, 64, 64, True, "yarn", torch.bfloat16, False),
    (7, 3, 2, 128, 0, 64, False, "linear", torch.float32, True),
    (33, 16, 1, 192, 128, 64, True, "yarn", torch.float32, False),
    (300, 5, 5, 192, 0, 192, False, "none", torch.bfloat16, True),
    (1001, 1, 0, 128, 0, 32, True, "linear", torch.bfloat16, False),
    (3, 300, 0, 128, 64, 64, False, "yarn", torch.bfloat16, False),
    (5000, 1, 1, 64, 48, 16, False, "none", torch.float32, False),
    (2, 4, 1, 1024, 8, 256, True, "none", torch.float32, False),
    (130, 64, 1, 576, 512, 64, False, "none", torch.bfloat16, False),
]


def _rope_tol(mag, y, factor, dtype):
    """cos and sin: the angle to 2^-27 half turns, 0.4 steps of 2^-24, and 2 ulp; then the factor's
    product, and a product and a sum of fp32: 6 steps of the magnitudes; one more rounding of the output."""
    return 6 * F32_STEP * mag + np.abs(y) * (BF16_STEP if dtype == torch.bfloat16 else F32_STEP) * 1.01


@pytest.mark.parametrize("rows,H_q,H_k,d,begin,rot,inter,scaling,dtype,inverse", ROPE_CASES)
def test_rope(rows, H_q, H_k, d, begin, rot, inter, scaling, dtype, inverse):
    g = torch.Generator().manual_seed(rows + d)
    kw = dict(scaling=scaling, factor=1.0 if scaling == "none" else 8.0)
    table, f = dsa.dsa_rope_freqs(rot, **kw), float(np.float32(1.3))
    pos = torch.randint(0, 1 << 20, (rows,), generator=g, dtype=torch.int32)
    pos[0] = 0
    xs = [torch.randn((rows, h, d), generator=g).to(dtype) if h else None for h in (H_q, H_k)]
    q_out, k_out = dsa.dsa_rope(xs[0].cuda(), pos.cuda(), table, k=None if xs[1] is None else xs[1].cuda(),
                                rot_begin=begin, interleaved=inter, attn_factor=f, inverse=inverse)
    for x, got in zip(xs, (q_out, k_out)):
        if x is None:
            assert got is None
            continue
        ref, mag = spec_ref.rope(x.double().numpy(), pos.numpy(), spec_ref.rope_freqs(rot, **kw), begin, inter, f,
                                 inverse)
        got = got.double().cpu().numpy()
        keep = np.r_[0:begin, begin + rot:d]
        assert np.array_equal(got[..., keep], x.double().numpy()[..., keep])
        assert np.all(np.abs(got - ref) <= _rope_tol(mag, ref, f, dtype))


@pytest.mark.parametrize("positions", [[2 ** 31 - 1, 2 ** 31 - 2, -1, -2 ** 31, 2 ** 30 + 12345, 0]])
def test_rope_far_positions(positions):
    """The angle of the table's definition, in whole numbers: positions * turns mod 2^64."""
    table = dsa.dsa_rope_freqs(64)
    x = torch.randn((len(positions), 2, 64), generator=torch.Generator().manual_seed(1))
    got, _ = dsa.dsa_rope(x.cuda(), _dev(positions), table)
    turn = np.array([[float((p * int(t)) % 2 ** 64) / 2.0 ** 64 for t in table] for p in positions])[:, None, :]
    co, si = np.cos(2 * np.pi * turn), np.sin(2 * np.pi * turn)
    a, c = x.double().numpy()[..., :32], x.double().numpy()[..., 32:]
    ref = np.concatenate([a * co - c * si, c * co + a * si], -1)
    mag = np.concatenate([np.abs(a) + np.abs(c)] * 2, -1)
    assert np.all(np.abs(got.double().cpu().numpy() - ref) <= _rope_tol(mag, ref, 1.0, torch.float32))


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rope_strided_and_in_place(inter, dtype):
    """q and k as parts of one projection's output, rotated in place: the same bits, the rest untouched."""
    rows, H_q, H_k, d = 37, 6, 2, 128
    x = torch.randn((rows, (H_q + 2 * H_k) * d), generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    pos, table = torch.arange(rows, dtype=torch.int32, device="cuda") * 1000, dsa.dsa_rope_freqs(64)
    kw = dict(rot_begin=32, interleaved=inter)
    q, k = x[:, :H_q * d].view(rows, H_q, d), x[:, H_q * d:(H_q + H_k) * d].view(rows, H_k, d)
    want_q, want_k = dsa.dsa_rope(q.contiguous(), pos, table, k=k.contiguous(), **kw)
    old = x.clone()
    got_q, got_k = dsa.dsa_rope(q, pos, table, k=k, **kw)
    assert torch.equal(x, old) and torch.equal(got_q, want_q) and torch.equal(got_k, want_k)
    dsa.dsa_rope(q, pos, table, k=k, q_out=q, k_out=k, **kw)
    assert torch.equal(q, want_q) and torch.equal(k, want_k)
    assert torch.equal(x[:, (H_q + H_k) * d:], old[:, (H_q + H_k) * d:])
    # only one of the two in place
    y = old.clone()
    q2, k2 = y[:, :H_q * d].view(rows, H_q, d), y[:, H_q * d:(H_q + H_k) * d].view(rows, H_k, d)
    _, got_k = dsa.dsa_rope(q2, pos, table, k=k2, q_out=q2, **kw)
    assert torch.equal(q2, want_q) and torch.equal(got_k, want_k) and torch.equal(k2.contiguous(), old[:, H_q * d:(H_q + H_k) * d].view(rows, H_k, d))


def test_rope_gradient():
    """inverse is the transpose: against the formula's gradient and against differences of the forward call."""
    rows, H, d = 5, 3, 64
    g = torch.Generator().manual_seed(4)
    x, gy = torch.randn((rows, H, d), generator=g), torch.randn((rows, H, d), generator=g)
    pos, table = torch.arange(rows, dtype=torch.int32).mul(777).cuda(), dsa.dsa_rope_freqs(32)
    kw = dict(rot_begin=16, attn_factor=0.75)
    gx = dsa.dsa_rope(gy.cuda(), pos, table, inverse=True, **kw)[0].double().cpu().numpy()
    eye = np.eye(d)
    J = np.stack([spec_ref.rope(np.tile(e, (rows, 1, 1)), pos.cpu().numpy(), spec_ref.rope_freqs(32), 16, False, 0.75)[0]
                  [:, 0] for e in eye], -1)                       # [rows, out, in]
    ref = np.einsum("roi,rho->rhi", J, gy.double().numpy())
    mag = np.einsum("roi,rho->rhi", np.abs(J), np.abs(gy.double().numpy()))
    assert np.all(np.abs(gx - ref) <= 8 * F32_STEP * mag)
    # the map is linear, so a difference over a step of 1 is the directional derivative
    for seed in range(3):
        v = torch.randn((rows, H, d), generator=torch.Generator().manual_seed(50 + seed))
        y1 = dsa.dsa_rope((x + v).cuda(), pos, table, **kw)[0].double().cpu()
        y0 = dsa.dsa_rope(x.cuda(), pos, table, **kw)[0].double().cpu()
        lhs, rhs = float(((y1 - y0) * gy.double()).sum()), float((gx * v.double().numpy()).sum())
        assert abs(lhs - rhs) <= 32 * F32_STEP * float((gy.abs() * (x.abs() + v.abs() + 1) * 4).double().sum())


def test_rope_no_rows():
    q, k = dsa.dsa_rope(torch.empty((0, 4, 64), device="cuda"), _dev([]), dsa.dsa_rope_freqs(64))
    assert q.shape == (0, 4, 64) and k is None


# ------------------------------------------------------------------ block tables

def _pool(rng, B, ps, width, most, spare):
    ctx = rng.integers(0, most + 1, B)
    held = np.minimum(-(-ctx // ps) + rng.integers(0, 2, B), width)       # some hold a page more than they need
    total = int(held.sum()) + spare
    order = rng.permutation(total)
    bt = np.full((B, width), -1)
    bt[np.arange(width)[None, :] < held[:, None]] = order[:held.sum()]
    return dict(block_table=bt, context_lens=ctx, pages_held=held, free_pages=np.append(order[held.sum():], [-1] * 5),
                free_count=np.array([spare])), total


def _run_pool(pool, new, ps, num_pages, max_tokens):
    dev = {k: _dev(v) for k, v in pool.items()}
    st = _status()
    plan = dsa.dsa_blocks_extend(dev, _dev(new), ps, num_pages, max_tokens, status=st)
    return dev, plan, int(st.item())


def _same(dev, ref):
    for k, v in ref.items():
        assert np.array_equal(dev[k].cpu().numpy(), v), k


@pytest.mark.parametrize("B,ps,width,most,grow,spare,max_tokens", [
    (1, 16, 4, 0, 1, 5, 1), (1, 64, 9, 100, 300, 9, 300), (64, 64, 20, 1000, 16, 200, 1030), (7, 48, 30, 900, 200, 60, 1500),
    (1024, 16, 6, 60, 20, 3000, 21000), (2500, 16, 8, 60, 9, 4000, 30000),
    (2500, 16, 8, 60, 9, 700, 30000),          # pages run out in the second thousand
    (300, 32, 8, 100, 40, 900, 3001),          # max_tokens runs out
    (300, 32, 4, 100, 90, 900, 20000),         # sequences outgrow their tables
    (5, 16, 3, 20, 9, 0, 40),                  # nothing free
])
def test_blocks_extend_and_trim(B, ps, width, most, grow, spare, max_tokens):
    rng = np.random.default_rng(B + ps + spare)
    ref, num_pages = _pool(rng, B, ps, width, most, spare)
    new = rng.integers(0, grow + 1, B)
    new[0] = grow
    old = {k: v.copy() for k, v in ref.items()}
    dev, plan, st = _run_pool(ref, new, ps, num_pages, max_tokens)
    ref_plan, err = spec_ref.extend(ref, new, ps, num_pages, max_tokens)
    _same(dev, ref)
    _same(plan, ref_plan)
    assert (st != 0) == err
    keep = np.where(rng.random(B) < 0.2, 0, rng.integers(0, 10 ** 6, B) % (ref["context_lens"] + 1))
    for room in (0, num_pages):                  # a stack that may not hold what comes back, and one that does
        trimmed, ref2 = {k: v.clone() for k, v in dev.items()}, {k: v.copy() for k, v in ref.items()}
        ref2["free_pages"] = np.append(ref2["free_pages"], [-1] * room)
        trimmed["free_pages"] = _dev(ref2["free_pages"])
        st = _status()
        dsa.dsa_blocks_trim(trimmed, _dev(keep), ps, num_pages, status=st)
        refused = spec_ref.trim(ref2, keep, ps, num_pages)
        assert (int(st.item()) == WORKSPACE) == refused and not (room and refused)
        _same(trimmed, ref2)
    if not err and np.array_equal(old["pages_held"], -(-old["context_lens"] // ps)):
        dsa.dsa_blocks_trim(dev, _dev(old["context_lens"]), ps, num_pages)
        _same(dev, old)


def test_blocks_extend_refusals_leave_the_pool():
    ps, num_pages = 16, 40
    base = dict(block_table=np.array([[3, 4, -1, -1]] * 6), context_lens=np.array([20, 40, -1, 20, 20, 20]),
                pages_held=np.array([2, 2, 2, 5, -1, 2]), free_pages=np.arange(10, 20), free_count=np.array([10]))
    new = np.array([-3, 1, 1, 1, 1, 5])                    # five sequences that may not be; the last one grows
    dev, plan, st = _run_pool(base, new, ps, num_pages, 50)
    ref_plan, err = spec_ref.extend(base, new, ps, num_pages, 50)
    assert st == INVALID and err
    _same(dev, base)
    _same(plan, ref_plan)
    # page ids of the free stack that are out of range: reported, slot -1, nothing written elsewhere
    bad = dict(block_table=np.full((2, 3), -1), context_lens=np.zeros(2, int), pages_held=np.zeros(2, int),
               free_pages=np.array([5, 40, -7]), free_count=np.array([3]))
    dev, plan, st = _run_pool(bad, np.array([30, 10]), ps, num_pages, 64)
    ref_plan, _ = spec_ref.extend(bad, np.array([30, 10]), ps, num_pages, 64)
    assert st == INVALID
    _same(dev, bad)
    _same(plan, ref_plan)
    # a free count that is not one
    for count in (-1, 11):
        p = dict(block_table=np.full((2, 3), -1), context_lens=np.zeros(2, int), pages_held=np.zeros(2, int),
                 free_pages=np.arange(10), free_count=np.array([count]))
        dev, plan, st = _run_pool(p, np.array([1, 0]), ps, num_pages, 8)
        assert st in (INVALID, WORKSPACE) and int(plan["token_start"][-1]) == 0
        _same(dev, p)


def test_blocks_trim_refusals_leave_the_pool():
    ps, num_pages = 16, 40
    ref = dict(block_table=np.array([[3, 4, 5, -1]] * 3 + [[6, 99, 7, -1]] + [[8, 9, 1, -1]]),
               context_lens=np.array([40, 40, 40, 40, 40]), pages_held=np.array([3, 3, 7, 3, 3]),
               free_pages=np.array([20, 21, -1, -1, -1, -1]), free_count=np.array([2]))
    keep = np.array([41, -1, 3, 1, 0])          # too long, negative, pages_held out of range, a bad page, no room left
    dev = {k: _dev(v) for k, v in ref.items()}
    st = _status()
    dsa.dsa_blocks_trim(dev, _dev(keep), ps, num_pages, status=st)
    assert spec_ref.trim(ref, keep, ps, num_pages) and int(st.item()) in (INVALID, WORKSPACE)
    _same(dev, ref)


# ------------------------------------------------------------------ tree attention

def _tree_case(rng, ns, ctxs, H, Hkv, d, ps, kv8, q_mul=1.5, num_extra=3, rand_parent=True):
    """Inputs (numpy and device) of packed trees; what lies behind each context is poison."""
    B, N = len(ns), sum(ns)
    pages = [-(-max(c, 1) // ps) for c in ctxs]
    P = sum(pages) + num_extra
    order = rng.permutation(P)
    bt = np.full((B, max(pages) + 1), -1)
    at = 0
    for b, p in enumerate(pages):
        bt[b, :p] = order[at:at + p]
        at += p
    parents = []
    for n in ns:
        for i in range(n):
            parents.append(i - 1 if i == 0 or not rand_parent else int(rng.integers(-1, i)))
    start = np.concatenate([[0], np.cumsum(ns)])
    q = torch.from_numpy(q_mul * rng.standard_normal((N, H, d))).to(torch.bfloat16)
    inp, vals = {}, {}
    used = np.zeros((P, ps), bool)
    for b, c in enumerate(ctxs):
        for s in range(c):
            used[bt[b, s // ps], s % ps] = True
    for x in ("k", "v"):
        if kv8:
            codes = rng.integers(0, 256, (P, ps, Hkv, d)).astype(np.uint8)
            codes[(codes & 0x7F) == 0x7F] = 0x30
            scale = np.exp(rng.uniform(-6, -4, (P, ps, Hkv))).astype(np.float32)
            vals[x] = spec_ref.e4m3_values(codes) * scale[..., None].astype(np.float64)
            codes[~used] = 0x7F                              # NaN
            scale[~used] = np.inf
            inp[x + "_cache"], inp[x + "_cache_scale"] = torch.from_numpy(codes), torch.from_numpy(scale)
        else:
            t = torch.from_numpy(rng.standard_normal((P, ps, Hkv, d))).to(torch.bfloat16)
            vals[x] = t.double().numpy()
            poison = torch.from_numpy(rng.choice([np.inf, -np.inf, np.nan], t.shape)).to(torch.bfloat16)
            inp[x + "_cache"] = torch.where(torch.from_numpy(used)[..., None, None], t, poison)
    inp.update(q=q, block_table=torch.from_numpy(bt).int(), context_lens=torch.tensor(ctxs, dtype=torch.int32),
               token_start=torch.from_numpy(start).int(), parents=torch.tensor(parents, dtype=torch.int32))
    return inp, vals


def _tree_ref(inp, vals, b, sm):
    bt, ctx = inp["block_table"].numpy(), int(inp["context_lens"][b])
    t0, t1 = int(inp["token_start"][b]), int(inp["token_start"][b + 1])
    ps = inp["k_cache"].shape[1]
    s = np.arange(ctx)
    K, V = (vals[x][bt[b, s // ps], s % ps] for x in ("k", "v"))
    q = inp["q"][t0:t1].double().numpy()
    return spec_ref.tree_attn(q, K, V, ctx, inp["parents"][t0:t1].numpy(), q.shape[1] // K.shape[1], sm), slice(t0, t1)


def _check_tree(inp, vals, out, lse, sm, seqs=None):
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(len(inp["context_lens"])) if seqs is None else seqs:
        (ro, rl, to, tl), rows = _tree_ref(inp, vals, b, sm)
        assert np.array_equal(np.isneginf(lse[rows]), np.isneginf(rl)), b
        fin = np.isfinite(rl)
        err_o, err_l = np.abs(out[rows] - ro), np.abs(lse[rows][fin] - rl[fin])
        assert np.all(err_o <= to), (b, np.max(err_o / np.maximum(to, 1e-300)))
        assert np.all(err_l <= tl[fin]), (b, np.max(err_l / tl[fin]))
        assert np.all(out[rows][~fin] == 0)


def _run_tree(inp, max_tree=None, max_context=None, sm=None, **kw):
    dev = {k: v.cuda() for k, v in inp.items()}
    ns = (inp["token_start"][1:] - inp["token_start"][:-1]).clamp(min=0)
    return dsa.dsa_tree_attn(dev, int(ns.max()) if max_tree is None else max_tree,
                             int(inp["context_lens"].max()) if max_context is None else max_context, sm, **kw)


TREE_CASES = [
    # drafts of each sequence, contexts, H, H_kv, d, page
    ([1], [1], 1, 1, 128, 16),
    ([1], [1], 16, 1, 64, 64),
    ([3], [3], 16, 1, 128, 64),                      # no prefix
    ([5, 0, 2], [128, 0, 129], 8, 8, 128, 32),
    ([7, 1, 4], [127, 300, 256], 24, 2, 64, 48),
    ([9], [700], 128, 1, 128, 64),
    ([2, 3], [500, 130], 256, 1, 128, 128),          # a token takes two tiles
    ([2], [333], 200, 1, 64, 16),                    # and the second of them is not full
    ([3, 2], [200, 70], 300, 1, 64, 16),             # three tiles a token: a pair holds two tokens' tiles
    ([2, 1], [150, 40], 512, 4, 128, 16),            # one full tile a token
    ([5, 3], [260, 33], 100, 1, 128, 32),            # 28 rows of every tile that no head has
    ([33, 64, 1], [100, 64, 900], 40, 1, 128, 16),
    ([128, 127], [128, 400], 4, 4, 64, 32),          # the largest trees
    ([5, 6], [1000, 70], 48, 16, 128, 64),           # groups of 3: 42 tokens and 2 rows that no token has
    ([17] * 9, [40 + 61 * i for i in range(9)], 16, 2, 128, 16),
    ([2] * 3, [4000, 2, 2500], 16, 1, 128, 80),
]


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("ns,ctxs,H,Hkv,d,ps", TREE_CASES)
def test_tree_attn(ns, ctxs, H, Hkv, d, ps, kv8):
    rng = np.random.default_rng(sum(ctxs) + H)
    inp, vals = _tree_case(rng, ns, ctxs, H, Hkv, d, ps, kv8)
    sm = 1.0 / np.sqrt(d)
    ws = dsa.workspace(dsa.tree_attn_workspace_size(len(ns), sum(ns), H, Hkv, d), "cuda")
    out, lse = _run_tree(inp, sm=sm, ws=ws)
    assert dsa.dsa_stream_status(ws) == 0
    _check_tree(inp, vals, out, lse, sm)
    # looser bounds, a dirty workspace: the same bits
    ws.fill_(0xFF)
    out2, lse2 = _run_tree(inp, max_tree=128, max_context=ctxs[0] + 5000, sm=sm, ws=ws)
    if max(ctxs) <= ctxs[0] + 5000:
        assert dsa.dsa_stream_status(ws) == 0
        assert torch.equal(out2, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("kv8", [False, True])
def test_tree_attn_large_logits(kv8):
    """Logits of some hundreds, growing along the context: the running maximum moves, far weights vanish."""
    rng = np.random.default_rng(11)
    inp, vals = _tree_case(rng, [4, 3], [1500, 900], 16, 1, 128, 64, kv8, q_mul=40.0)
    _check_tree(inp, vals, *_run_tree(inp, sm=0.3), 0.3)


def test_tree_attn_equal_logits_and_zero_rows():
    """Zero queries: every allowed row weighs the same."""
    rng = np.random.default_rng(12)
    inp, vals = _tree_case(rng, [6, 2], [260, 2], 8, 2, 64, 16, False)
    inp["q"].zero_()
    out, lse = _run_tree(inp)
    _check_tree(inp, vals, out, lse, 0.125)
    depth = [len(a) for a in spec_ref.ancestors(inp["parents"][:6].numpy())]
    want = np.log(np.array([254 + n for n in depth]))[:, None].repeat(8, 1)
    assert np.all(np.abs(lse[:6].double().cpu().numpy() - want) <= 300 * F32_STEP + 8 * F32_STEP)


def test_tree_attn_padding_rows_and_bad_parents():
    rng = np.random.default_rng(13)
    for kv8 in (False, True):
        inp, vals = _tree_case(rng, [6, 5], [200, 5], 16, 2, 128, 32, kv8)
        p = inp["parents"]
        p[:6] = torch.tensor([-1, -2, 1, 0, -7, 3])          # 1 and 4 are padding, 2 stands under one
        p[6:] = torch.tensor([-1, 0, 1, -2, 3])
        out, lse = _run_tree(inp)
        _check_tree(inp, vals, out, lse, 128 ** -0.5)
        assert torch.all(out[[1, 2, 4, 9, 10]] == 0) and torch.all(torch.isneginf(lse[[1, 2, 4, 9, 10]]))
        p[3] = 5                                             # a parent behind its child
        ws = dsa.workspace(dsa.tree_attn_workspace_size(2, 11, 16, 2, 128), "cuda")
        out, lse = _run_tree(inp, ws=ws)
        assert dsa.dsa_stream_status(ws) == INVALID
        _check_tree(inp, vals, out, lse, 128 ** -0.5)


@pytest.mark.parametrize("kv8", [False, True])
def test_tree_attn_reports_and_skips_bad_sequences(kv8):
    rng = np.random.default_rng(14)
    ns, ctxs = [3, 4, 2, 5, 6], [200, 300, 250, 90, 400]
    inp, vals = _tree_case(rng, ns, ctxs, 16, 1, 128, 64, kv8)
    good, glse = _run_tree(inp)
    for change in (dict(at=1, ctx=3), dict(at=1, ctx=10 ** 6), dict(at=3, ctx=-1), dict(max_context=350, at=4),
                   dict(max_tree=5, at=4)):
        bad = {k: v.clone() for k, v in inp.items()}
        if "ctx" in change:
            bad["context_lens"][change["at"]] = change["ctx"]
        ws = dsa.workspace(dsa.tree_attn_workspace_size(5, 20, 16, 1, 128), "cuda")
        out, lse = torch.full_like(good, 7.0), torch.full_like(glse, 7.0)
        _run_tree(bad, max_tree=change.get("max_tree", 6), max_context=change.get("max_context", 400), out=out, lse=lse,
                  ws=ws)
        assert dsa.dsa_stream_status(ws) == INVALID
        r = slice(int(inp["token_start"][change["at"]]), int(inp["token_start"][change["at"] + 1]))
        keep = torch.ones(20, dtype=torch.bool)
        keep[r] = False
        assert torch.all(out[r] == 7.0) and torch.all(lse[r] == 7.0)
        _check_tree(inp, vals, out, lse, 128 ** -0.5, [b for b in range(5) if b != change["at"]])
    # token_start out of order and past N
    for ts in ([0, 3, 2, 9, 14, 20], [0, 3, 7, 9, 14, 21], [-2, 3, 7, 9, 14, 20]):
        bad = dict(inp, token_start=torch.tensor(ts, dtype=torch.int32))
        ws = dsa.workspace(dsa.tree_attn_workspace_size(5, 20, 16, 1, 128), "cuda")
        _run_tree(bad, max_tree=8, max_context=400, ws=ws)
        assert dsa.dsa_stream_status(ws) == INVALID


@pytest.mark.parametrize("kv8", [False, True])
def test_tree_attn_bad_pages_count_as_zero_rows(kv8):
    rng = np.random.default_rng(15)
    inp, vals = _tree_case(rng, [3, 2], [300, 129], 8, 1, 128, 32, kv8)
    P = inp["k_cache"].shape[0]
    for page in (-1, P, 2 ** 31 - 1, -2 ** 31):
        bad = {k: v.clone() for k, v in inp.items()}
        bad["block_table"][0, 2] = page
        ws = dsa.workspace(dsa.tree_attn_workspace_size(2, 5, 8, 1, 128), "cuda")
        out, lse = _run_tree(bad, ws=ws)
        assert dsa.dsa_stream_status(ws) == INVALID
        z = {x: v.copy() for x, v in vals.items()}
        for x in z:
            z[x][int(inp["block_table"][0, 2])] = 0
        _check_tree(inp, z, out, lse, 128 ** -0.5)


@pytest.mark.parametrize("ns,ctxs", [([4, 3], [100, 60]), ([4, 3], [3000, 2000]), ([40], [5000])])
def test_tree_attn_a_query_that_is_no_number_stays_in_its_row(ns, ctxs):
    rng = np.random.default_rng(24)
    for kv8 in (False, True):
        inp, vals = _tree_case(rng, ns, ctxs, 16, 1, 128, 64, kv8)
        want, want_lse = _run_tree(inp)
        inp["parents"][2] = -2                               # a padding row
        base, base_lse = _run_tree(inp)
        bad = dict(inp, q=inp["q"].clone())
        bad["q"][1, 3, 5], bad["q"][2], bad["q"][0, 0, 0] = float("nan"), float("nan"), float("inf")
        out, lse = _run_tree(bad)
        assert torch.isnan(out[1, 3]).all() and torch.isnan(lse[1, 3])
        assert torch.all(out[2] == 0) and torch.isneginf(lse[2]).all()
        keep = torch.ones(sum(ns), 16, dtype=torch.bool)
        keep[1, 3] = keep[0, 0] = False
        assert torch.equal(out[keep], base[keep]) and torch.equal(lse[keep], base_lse[keep])
        assert not torch.isnan(want).any() and not torch.isnan(want_lse).any()


def test_tree_attn_rows_behind_the_last_sequence_stay():
    rng = np.random.default_rng(16)
    inp, vals = _tree_case(rng, [3, 2], [130, 64], 16, 1, 128, 64, False)
    pad = 4
    more = dict(inp, q=torch.cat([inp["q"], torch.full((pad, 16, 128), float("nan"), dtype=torch.bfloat16)]),
                parents=torch.cat([inp["parents"], torch.full((pad,), 99, dtype=torch.int32)]))
    out = torch.full((5 + pad, 16, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((5 + pad, 16), 3.0, device="cuda")
    _run_tree(more, out=out, lse=lse)
    assert torch.all(out[5:] == 3.0) and torch.all(lse[5:] == 3.0)
    _check_tree(inp, vals, out, lse, 128 ** -0.5)


@pytest.mark.parametrize("B", [600, 1300])
def test_tree_attn_many_sequences(B):
    """More sequences than a CTA has threads, most of them without drafts in this step."""
    rng = np.random.default_rng(B)
    ns = [int(v) for v in rng.choice([0, 0, 0, 1, 2], B)]
    ctxs = [n + int(rng.integers(0, 90)) for n in ns]
    inp, vals = _tree_case(rng, ns, ctxs, 2, 1, 64, 16, False)
    out, lse = _run_tree(inp)
    _check_tree(inp, vals, out, lse, 0.125)


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_tree_attn_many_short_items(d, kv8):
    """Several items a CTA, single tiles and pairs in turn, some of one block: the sets' steps, the item ends
    and the statistics of one item must not be taken for another's."""
    rng = np.random.default_rng(19)
    ns = [int(v) for v in rng.choice([0, 1, 2, 3, 4, 5, 7], 700)]
    ctxs = [n + int(rng.choice([0, 3, 60, 130, 300], p=[0.3, 0.3, 0.2, 0.1, 0.1])) for n in ns]
    inp, vals = _tree_case(rng, ns, ctxs, 64, 1, d, 32, kv8)
    ws = dsa.workspace(dsa.tree_attn_workspace_size(700, sum(ns), 64, 1, d), "cuda")
    out, lse = torch.full((sum(ns), 64, d), 9.0, dtype=torch.bfloat16, device="cuda"), torch.full((sum(ns), 64), 9.0, device="cuda")
    for _ in range(5):
        _run_tree(inp, out=out, lse=lse, ws=ws)
        assert dsa.dsa_stream_status(ws) == 0
    _check_tree(inp, vals, out, lse, d ** -0.5, [b for b in range(700) if ns[b] and b % 7 == 0])
    again, lse2 = _run_tree(inp)
    assert torch.equal(again, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("kv8", [False, True])
def test_tree_attn_far_into_a_large_cache(kv8):
    """Pages whose elements lie past 2^31 of a cache."""
    rng = np.random.default_rng(17)
    d, ps, P = 128, 64, (2 ** 31 // (64 * 128)) + 5000
    small, vals = _tree_case(rng, [3], [300], 16, 1, d, ps, kv8)
    used = int((small["block_table"][0] >= 0).sum())
    far = torch.arange(P - used, P)
    big = {}
    for x in [k for k in small if "cache" in k]:
        shape = (P,) + tuple(small[x].shape[1:])
        c = torch.zeros(shape, dtype=small[x].dtype, device="cuda")
        c[far.cuda()] = small[x][small["block_table"][0, :used].long()].cuda()
        big[x] = c
    dev = {k: v.cuda() for k, v in small.items() if "cache" not in k}
    dev["block_table"][0, :used] = far.int().cuda()
    out, lse = dsa.dsa_tree_attn({**dev, **big}, 3, 300)
    _check_tree(small, vals, out, lse, d ** -0.5)


def test_tree_attn_single_tokens_match_the_decode():
    """A tree of one token is a decode step; with k >= the context the sparse decode selects every position."""
    import dsa_synth
    lens = (300, 64, 1, 1000)
    spec = dsa_synth.DecodeSpec("spec", context_lens=lens, H_I=64, d_I=128, k=1024, H_q=128, d=128, page_size=64,
                                needle_frac=0.01, needle_min_age=0, seed=3)
    inp = dsa_synth.make_decode(spec)
    dev = {k: v.cuda() for k, v in inp.items() if isinstance(v, torch.Tensor)}
    want, want_lse, _ = dsa.dsa_decode(dev, spec.k, max(lens))
    tree = dict(q=dev["q"], k_cache=dev["k_cache"], v_cache=dev["v_cache"], block_table=dev["block_table"],
                context_lens=dev["context_lens"], token_start=_dev(np.arange(5)), parents=_dev([-1] * 4))
    got, got_lse = dsa.dsa_tree_attn(tree, 1, max(lens))
    # two bf16 kernels of the same sums: weights rounded on both sides, and the outputs
    w = dev["v_cache"].float().abs().max()
    assert (got.float() - want.float()).abs().max() <= 4 * BF16_STEP * w
    assert (got_lse - want_lse).abs().max() <= 1e-4


def test_tree_attn_repeats_bit_for_bit_on_other_streams_and_in_graphs():
    rng = np.random.default_rng(18)
    inp, vals = _tree_case(rng, [9, 5, 1], [3000, 2100, 40], 32, 2, 128, 64, False)
    dev = {k: v.cuda() for k, v in inp.items()}
    want, want_lse = dsa.dsa_tree_attn(dev, 9, 3000)
    size = dsa.tree_attn_workspace_size(3, 15, 32, 2, 128)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(dsa.dsa_tree_attn(dev, 9, 3000, ws=dsa.workspace(size, "cuda")))
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want) and torch.equal(l, want_lse)
    ws, out, lse = dsa.workspace(size, "cuda"), torch.zeros_like(want), torch.zeros_like(want_lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.dsa_tree_attn(dev, 9, 3000, out=out, lse=lse, ws=ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    # other lengths in the same graph
    dev["context_lens"].copy_(_dev([1700, 2000, 7]))
    graph.replay()
    torch.cuda.synchronize()
    inp["context_lens"] = torch.tensor([1700, 2000, 7], dtype=torch.int32)
    _check_tree(inp, vals, out, lse, 128 ** -0.5)


# ------------------------------------------------------------------ verification

def _verify_case(rng, ns, V, point, chain=False, dup=False):
    N = sum(ns)
    P = rng.random((N, V)) ** 8
    P = (P / P.sum(-1, keepdims=True)).astype(np.float32)
    Q = rng.random((N, V)) ** 8
    Q = (Q / Q.sum(-1, keepdims=True)).astype(np.float32)
    tokens, parents = [], []
    for n in ns:
        for i in range(n):
            parents.append(i - 1 if chain or i == 0 else int(rng.integers(max(0, i - 4), i)))
            tokens.append(int(rng.integers(0, min(V, 3 if dup else V))))
    start = np.concatenate([[0], np.cumsum(ns)]).astype(int)
    for b, n in enumerate(ns):                               # tokens that the parent's target likes
        for i in range(1, n):
            t = start[b] + i
            if rng.random() < 0.7 and not dup:
                tokens[t] = int(np.argmax(P[start[b] + parents[t]] * rng.random(V)))
    return P, None if point else Q, np.array(tokens), np.array(parents), start, rng.random(N).astype(np.float32), \
        rng.random(len(ns)).astype(np.float32)


def _run_verify(P, Q, tokens, parents, start, ua, us, **kw):
    f = torch.float32
    return dsa.dsa_verify_tree(_dev(P, f), None if Q is None else _dev(Q, f), _dev(tokens), _dev(parents), _dev(start),
                               _dev(ua, f), _dev(us, f), **kw)


def _check_verify(case, max_path, got):
    P, Q, tokens, parents, start, ua, us = case
    path, acc, nxt = (x.cpu().numpy() for x in got)
    for b in range(len(us)):
        r = slice(int(start[b]), int(start[b + 1]))
        want, tok = spec_ref.verify(P[r], None if Q is None else Q[r], tokens[r], parents[r], ua[r], us[b], max_path)
        assert acc[b] == len(want) and list(path[b, :acc[b]]) == want and np.all(path[b, acc[b]:] == -1), b
        assert nxt[b] == tok, b


@pytest.mark.parametrize("point", [False, True])
@pytest.mark.parametrize("ns,V,chain", [([1], 1, True), ([1], 7, True), ([5], 1000, True), ([4, 0, 3], 129, False),
                                        ([16] * 5, 1023, False), ([64, 1, 33], 517, False), ([128], 64, False),
                                        ([9, 2], 32003, False), ([3] * 200, 50, False), ([2] * 700, 11, True)])
def test_verify(ns, V, chain, point):
    rng = np.random.default_rng(V + len(ns) + point)
    case = _verify_case(rng, ns, V, point, chain)
    st = _status()
    got = _run_verify(*case, status=st)
    _check_verify(case, 128, got)
    assert int(st.item()) == 0
    got2 = _run_verify(*case)
    assert all(torch.equal(a, b) for a, b in zip(got, got2))
    for m in (1, 2, 3):
        _check_verify(case, m, _run_verify(*case, max_path=m))


def test_verify_same_token_twice():
    """Siblings with the same token, and tokens that were already rejected."""
    rng = np.random.default_rng(21)
    for point in (False, True):
        case = _verify_case(rng, [20] * 40, 6, point, dup=True)
        _check_verify(case, 128, _run_verify(*case))


def test_verify_borders_are_exact():
    """Dyadic probabilities: sums and comparisons are exact, and a draw on a border takes the next token."""
    V = 4096
    P = np.zeros((1, V), np.float32)
    P[0, 1::4] = 4.0 / V                                     # 1024 tokens of 2^-10
    for k in (0, 1, 511, 512, 1023):
        for eps, want in ((0.0, k), (2.0 ** -12, k)):
            us = np.array([k / 1024 + eps], np.float32)
            _, acc, nxt = _run_verify(P, None, np.zeros(1, int), np.array([-1]), np.array([0, 1]), np.zeros(1, np.float32), us)
            assert int(acc) == 1 and int(nxt) == 1 + 4 * want
    # acceptance is strict: u Q = P is a rejection, and u = 0 accepts whatever has weight
    P = np.array([[0.25, 0.75, 0, 0], [0, 0, 1, 0]], np.float32)
    Q = np.array([[0.5, 0.25, 0.25, 0], [0.25] * 4], np.float32)
    for u, tok, want in ((0.5, 0, [0]), (0.499, 0, [0, 1]), (0.0, 0, [0, 1]), (0.0, 2, [0]), (0.0, 3, [0])):
        case = (P, Q, np.array([0, tok]), np.array([-1, 0]), np.array([0, 2]), np.array([0, u], np.float32),
                np.array([0.25], np.float32))
        got = _run_verify(*case)
        _check_verify(case, 128, got)
        assert list(got[0][0, :int(got[1])].tolist()) == want


def test_verify_reports():
    rng = np.random.default_rng(22)
    ns = [4, 3, 5]
    base = list(_verify_case(rng, ns, 100, False, chain=True))
    # tokens outside the vocabulary: rejected, nothing else changes
    case = list(base)
    case[2] = base[2].copy()
    case[2][[1, 5]] = [100, -1]
    st = _status()
    _check_verify(case, 128, _run_verify(*case, status=st))
    assert int(st.item()) == INVALID
    # rows without a positive finite sum
    for value in (0.0, np.nan, np.inf):
        case = list(base)
        case[0] = base[0].copy()
        case[0][4:7] = value
        case[3] = base[3]
        st = _status()
        path, acc, nxt = _run_verify(*case, status=st)
        assert int(nxt[1]) == -1 and int(st.item()) == INVALID
        if not np.isinf(value):
            _check_verify(case, 128, (path, acc, nxt))
    # token_start out of order, past N, and too many tokens
    for ts in ([0, 4, 2, 12], [0, 4, 7, 13], [-1, 4, 7, 12]):
        case = list(base)
        case[4] = np.array(ts)
        st = _status()
        path, acc, nxt = _run_verify(*case, status=st)
        assert int(st.item()) == INVALID
        for b in range(3):
            if ts[b] < 0 or ts[b + 1] < ts[b] or ts[b + 1] > 12:
                assert int(acc[b]) == 0 and int(nxt[b]) == -1 and torch.all(path[b] == -1)
    big = _verify_case(rng, [129, 2], 20, False)
    path, acc, nxt = _run_verify(*big, status=st)
    assert int(acc[0]) == 0 and int(nxt[0]) == -1 and int(acc[1]) > 0


def test_verify_without_tokens():
    f = torch.float32
    got = dsa.dsa_verify_tree(torch.empty((0, 10), device="cuda"), None, _dev([]), _dev([]), _dev([0, 0, 0]),
                              _dev([], f), _dev([0.5, 0.5], f))
    assert torch.all(got[0] == -1) and got[1].tolist() == [0, 0] and got[2].tolist() == [-1, -1]


# ------------------------------------------------------------------ compaction

def _compact_case(rng, ns, ctxs, ps, kv8, index, d=128, d_I=128):
    B = len(ns)
    pages = [-(-max(c, 1) // ps) for c in ctxs]
    P = sum(pages) + 2
    order = rng.permutation(P)
    bt = np.full((B, max(pages) + 1), -1)
    at = 0
    for b, p in enumerate(pages):
        bt[b, :p] = order[at:at + p]
        at += p
    caches = {}
    if index:
        caches["kidx_cache"] = rng.integers(0, 256, (P, ps, d_I)).astype(np.uint8)
        caches["kscale_cache"] = rng.random((P, ps)).astype(np.float32)
    for x in ("k", "v"):
        if kv8:
            caches[x + "_cache"] = rng.integers(0, 256, (P, ps, d)).astype(np.uint8)
            caches[x + "_cache_scale"] = rng.random((P, ps)).astype(np.float32)
        else:
            caches[x + "_cache"] = rng.integers(-2 ** 15, 2 ** 15, (P, ps, d)).astype(np.int16)
    width = max(max(ns), 1) + 2
    path, acc = np.full((B, width), -1), np.zeros(B, int)
    for b, n in enumerate(ns):
        p = np.nonzero(rng.random(n) < 0.5)[0]
        acc[b] = len(p)
        path[b, :len(p)] = p
    return caches, bt, np.array(ctxs), np.concatenate([[0], np.cumsum(ns)]), path, acc


def _run_compact(case, **kw):
    caches, bt, ctx, start, path, acc = case
    dev = {}
    for k, v in caches.items():
        t = torch.from_numpy(v.copy()).cuda()
        dev[k] = t.view(torch.bfloat16) if t.dtype == torch.int16 else t
    st = _status()
    keep = dsa.dsa_cache_compact(dev, _dev(bt), _dev(ctx), _dev(start), _dev(path), _dev(acc), status=st, **kw)
    dev = {k: (v.view(torch.int16) if v.dtype == torch.bfloat16 else v).cpu().numpy() for k, v in dev.items()}
    return dev, keep.cpu().numpy(), int(st.item())


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("ns,ctxs,ps,index,d,d_I", [
    ([1], [1], 16, True, 128, 128), ([5, 0, 7], [100, 33, 7], 16, True, 128, 128), ([128, 90], [128, 1000], 32, False, 64, 0),
    ([64] * 9, [70 + 31 * i for i in range(9)], 48, True, 128, 128), ([33, 20], [400, 20], 1, True, 8, 8),
    ([16] * 40, [300] * 40, 64, True, 256, 264)])
def test_compact(ns, ctxs, ps, index, d, d_I, kv8):
    case = _compact_case(np.random.default_rng(sum(ctxs) + kv8), ns, ctxs, ps, kv8, index, d, d_I or 8)
    dev, keep, st = _run_compact(case, N=sum(ns))
    caches, bt, ctx, start, path, acc = case
    want, err = spec_ref.compact(caches, bt, ctx, start, path, acc, sum(ns), len(caches["k_cache"]), ps)
    assert st == 0 and not err and np.array_equal(keep, want)
    for k, v in caches.items():
        assert np.array_equal(dev[k], v), k


def test_compact_leaves_bad_sequences_alone():
    ps = 16
    for kv8 in (False, True):
        case = list(_compact_case(np.random.default_rng(31), [8] * 9, [60] * 9, ps, kv8, True))
        caches, bt, ctx, start, path, acc = case
        acc[:] = 3
        path[:, :3] = [1, 4, 6]
        acc[0], acc[1] = 9, -1
        path[2, :3], path[3, :3], path[4, 2] = [1, 1, 5], [-1, 2, 3], 8
        ctx[5], ctx[6] = 7, 10 ** 6
        bt[7, 3] = len(caches["k_cache"])
        dev, keep, st = _run_compact(case)
        want, err = spec_ref.compact(caches, bt, ctx, start, path, acc, 72, len(caches["k_cache"]), ps)
        assert st == INVALID and err and np.array_equal(keep, want)
        assert list(keep[:8]) == list(ctx[:8]) and keep[8] == 55
        for k, v in caches.items():
            assert np.array_equal(dev[k], v), k


# ------------------------------------------------------------------ a step of speculative decoding

class _Step:
    """Buffers and calls of one step over a pool, as a serving loop keeps them."""

    def __init__(self, B, ps, width, P, n, H, V, kv8, d=128):
        i32 = dict(dtype=torch.int32, device="cuda")
        self.B, self.ps, self.P, self.n, self.H, self.V, self.kv8 = B, ps, P, n, H, V, kv8
        self.N = B * n
        self.max_context = width * ps
        self.pool = dict(block_table=torch.full((B, width), -1, **i32), context_lens=torch.zeros(B, **i32),
                         pages_held=torch.zeros(B, **i32), free_pages=torch.randperm(P, device="cuda").int(),
                         free_count=torch.full((1,), P, **i32))
        code = torch.uint8 if kv8 else torch.bfloat16
        self.caches = dict(kidx_cache=torch.zeros((P, ps, 128), dtype=torch.uint8, device="cuda"),
                           kscale_cache=torch.zeros((P, ps), device="cuda"))
        for x in ("k", "v"):
            self.caches[x + "_cache"] = torch.zeros((P, ps, d), dtype=code, device="cuda")
            if kv8:
                self.caches[x + "_cache_scale"] = torch.zeros((P, ps), device="cuda")
        self.append = dsa.dsa_cache_append_kv8 if kv8 else dsa.dsa_cache_append
        self.table = dsa.dsa_rope_freqs(64, scaling="yarn", factor=4.0)
        self.status = _status()
        self.new = torch.full((B,), n, **i32)
        self.plan = dict(token_start=torch.empty(B + 1, **i32), seq_ids=torch.empty(self.N, **i32),
                         positions=torch.empty(self.N, **i32),
                         slots=torch.empty(self.N, dtype=torch.int64, device="cuda"))
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.q, self.k, self.v = torch.empty((self.N, H, d), **bf), torch.empty((self.N, 1, d), **bf), torch.empty((self.N, d), **bf)
        self.kidx, self.depth = torch.empty((self.N, 128), **bf), torch.empty((self.N,), **i32)
        self.parents, self.tokens = torch.empty((self.N,), **i32), torch.empty((self.N,), **i32)
        self.target = torch.empty((self.N, V), device="cuda")
        self.draft = torch.empty((self.N, V), device="cuda")
        self.ua, self.us = torch.empty(self.N, device="cuda"), torch.empty(B, device="cuda")
        self.qr, self.kr = torch.empty_like(self.q), torch.empty_like(self.k)
        self.out, self.lse = torch.empty_like(self.q), torch.empty((self.N, H), device="cuda")
        self.ws = dsa.workspace(dsa.tree_attn_workspace_size(B, self.N, H, 1, d), "cuda")
        self.path = torch.empty((B, n), **i32)
        self.acc, self.next, self.keep = (torch.empty(B, **i32) for _ in range(3))

    def fill(self, seed):
        g = torch.Generator("cuda").manual_seed(seed)
        for x in (self.q, self.k, self.v, self.kidx):
            x.normal_(generator=g)
        rng = np.random.default_rng(seed)
        par = np.array([[-1] + [int(rng.integers(max(0, i - 3), i)) for i in range(1, self.n)] for _ in range(self.B)])
        depth = np.zeros_like(par)
        for i in range(1, self.n):
            depth[:, i] = depth[np.arange(self.B), par[:, i]] + 1
        self.depth.copy_(_dev(depth.reshape(-1)))
        self.parents.copy_(_dev(par.reshape(-1)))
        logits = torch.randn((self.N, self.V), generator=g, device="cuda")
        self.target.copy_(logits.softmax(-1))
        self.draft.copy_((logits + torch.randn((self.N, self.V), generator=g, device="cuda")).softmax(-1))
        self.tokens.copy_(torch.randint(0, self.V, (self.N,), generator=g, device="cuda"))
        self.ua.uniform_(generator=g)
        self.us.uniform_(generator=g)

    def run(self):
        start = self.plan["token_start"]
        dsa.dsa_blocks_extend(self.pool, self.new, self.ps, self.P, self.N, plan=self.plan, status=self.status)
        # a tree token's position for the rotation: the prefix plus its depth
        ctx = self.pool["context_lens"][self.plan["seq_ids"].long()] - self.n
        dsa.dsa_rope(self.q, (ctx + self.depth).int(), self.table, k=self.k, rot_begin=64, interleaved=True,
                     q_out=self.qr, k_out=self.kr)
        bt = self.pool["block_table"]
        self.append(self.caches, self.kidx, self.kr.view(self.N, -1), self.v, self.plan["seq_ids"],
                    self.plan["positions"], bt, status=self.status)
        inp = dict(q=self.qr, block_table=bt, context_lens=self.pool["context_lens"], token_start=start,
                   parents=self.parents, **{k: v for k, v in self.caches.items() if k[0] in "kv" and k[1] == "_"})
        dsa.dsa_tree_attn(inp, self.n, self.max_context, out=self.out, lse=self.lse, ws=self.ws)
        dsa.dsa_verify_tree(self.target, self.draft, self.tokens, self.parents, start, self.ua, self.us,
                            path=self.path, accept_len=self.acc, next_token=self.next, status=self.status)
        dsa.dsa_cache_compact(self.caches, bt, self.pool["context_lens"], start, self.path, self.acc, N=self.N,
                              keep_lens=self.keep, status=self.status)
        dsa.dsa_blocks_trim(self.pool, self.keep, self.ps, self.P, status=self.status)


@pytest.mark.parametrize("kv8", [False, True])
def test_steps_together(kv8):
    """Some steps, eagerly and replayed from a graph: the caches hold the accepted tokens' rows in order, the
    pool's pages stay whole, and the attention of the last step is the reference's over what was accepted."""
    B, ps, n, H, V = 5, 16, 7, 16, 300
    s = _Step(B, ps, 12, 70, n, H, V, kv8)
    s.fill(0)
    s.run()                                                  # the library loads its kernels before the capture
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    rows = [[] for _ in range(B)]                            # accepted (K, V) rows as they were appended

    def collect():
        torch.cuda.synchronize()
        acc, path = s.acc.cpu().numpy(), s.path.cpu().numpy()
        for b in range(B):
            assert acc[b] >= 1
            for i in range(acc[b]):
                t = b * n + int(path[b, i])
                rows[b].append((s.kr[t, 0].clone(), s.v[t].clone(), s.kidx[t].clone()))

    collect()
    with torch.cuda.graph(graph):
        s.run()
    for seed in range(1, 6):
        s.fill(seed)
        before = s.pool["context_lens"].cpu().numpy().copy()
        if seed % 2:
            graph.replay()
        else:
            s.run()
        torch.cuda.synchronize()
        assert dsa.dsa_stream_status(s.ws) == 0 and int(s.status.item()) == 0
        case = (s.target.cpu().numpy(), s.draft.cpu().numpy(), s.tokens.cpu().numpy(), s.parents.cpu().numpy(),
                np.arange(B + 1) * n, s.ua.cpu().numpy(), s.us.cpu().numpy())
        _check_verify(case, n, (s.path, s.acc, s.next))
        # attention: the accepted rows so far, then this step's drafts
        kr, v = s.kr[:, 0], s.v
        for b in range(B):
            t = slice(b * n, (b + 1) * n)
            K = torch.cat([torch.stack([r[0] for r in rows[b]]), kr[t]])
            Vv = torch.cat([torch.stack([r[1] for r in rows[b]]), v[t]])
            assert len(K) == before[b] + n
            if kv8:
                K, Vv = ((c.view(torch.float8_e4m3fn).double() * sc.double()[:, None]) for c, sc in
                         (dsa.dsa_quantize_e4m3(x.contiguous()) for x in (K, Vv)))
            ro, rl, to, tl = spec_ref.tree_attn(s.qr[t].double().cpu().numpy(), K.double().cpu().numpy()[:, None],
                                                Vv.double().cpu().numpy()[:, None], len(K), s.parents[t].cpu().numpy(), H,
                                                128 ** -0.5)
            assert np.all(np.abs(s.out[t].double().cpu().numpy() - ro) <= to)
            assert np.all(np.abs(s.lse[t].double().cpu().numpy() - rl) <= tl)
        collect()
        # the caches and the pool
        ctx, held, bt = (s.pool[k].cpu().numpy() for k in ("context_lens", "pages_held", "block_table"))
        count, free = int(s.pool["free_count"].item()), s.pool["free_pages"].cpu().numpy()
        assert np.array_equal(held, -(-ctx // ps))
        pages = np.concatenate([free[:count]] + [bt[b, :held[b]] for b in range(B)])
        assert np.array_equal(np.sort(pages), np.arange(70))
        for b in range(B):
            assert ctx[b] == len(rows[b])
            at = np.arange(ctx[b])
            slot = torch.from_numpy(bt[b, at // ps].astype(np.int64) * ps + at % ps).cuda()
            for j, x in enumerate(("k", "v", "kidx")):
                want = torch.stack([r[j] for r in rows[b]])
                got = s.caches[x + "_cache"].flatten(0, 1)[slot]
                if x == "kidx" or kv8:
                    codes, scale = dsa.dsa_quantize_e4m3(want)
                    assert torch.equal(got, codes)
                    name = "kscale_cache" if x == "kidx" else x + "_cache_scale"
                    assert torch.equal(s.caches[name].flatten()[slot], scale)
                else:
                    assert torch.equal(got, want)


def test_calls_on_tensors_of_a_stream():
    """The stream argument is the one that counts: work queued there before the call is seen by it."""
    side = torch.cuda.Stream()
    x = torch.zeros((4096, 16, 128), device="cuda")
    pos = torch.arange(4096, dtype=torch.int32, device="cuda")
    table = dsa.dsa_rope_freqs(128)
    y = torch.randn_like(x)
    out = torch.empty_like(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            x.add_(y)
    dsa.dsa_rope(x, pos, table, q_out=out, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, dsa.dsa_rope(x, pos, table)[0])


def test_memory_of_calls_on_another_stream():
    """With a stream argument, what the call allocates is that stream's: memory that the current stream takes
    right after the call is not the workspace or an output of the call, which has not begun yet."""
    rng = np.random.default_rng(24)
    inp, _ = _tree_case(rng, [9, 5, 1], [3000, 2100, 40], 32, 2, 128, 64, False)
    dev = {k: v.cuda() for k, v in inp.items()}
    P, tokens = torch.rand((3, 1000), device="cuda"), _dev([1, 2, 3])
    tree = (P, None, tokens, _dev([-1, 0, 1]), _dev([0, 3]), torch.rand(3, device="cuda"), torch.rand(1, device="cuda"))
    x, pos, table = torch.randn((500, 4, 64), device="cuda"), _dev(np.arange(500)), dsa.dsa_rope_freqs(64)

    pools = [dict(block_table=torch.full((2, 4), -1, dtype=torch.int32, device="cuda"), context_lens=_dev([0, 0]),
                  pages_held=_dev([0, 0]), free_pages=_dev(np.arange(8)), free_count=_dev([8])) for _ in range(2)]
    grow = _dev([20, 30])

    def calls(stream, blocks):
        return [*dsa.dsa_tree_attn(dev, 9, 3000, stream=stream), *dsa.dsa_verify_tree(*tree, max_path=3, stream=stream),
                *dsa.dsa_rope(x, pos, table, k=x, stream=stream),
                *dsa.dsa_blocks_extend(blocks, grow, 16, 8, 64, stream=stream).values()]

    want = calls(None, pools[0])
    torch.cuda.synchronize()
    held = torch.cuda.Stream()
    # freed blocks of every size in the current stream's pool, which a call must not take
    pool = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (*[512] * 16, *[1 << 18] * 8, *[1 << 25] * 4)]
    del pool
    torch.cuda.synchronize()
    with torch.cuda.stream(held):
        torch.cuda._sleep(50_000_000)
    got = calls(held, pools[1])
    sizes = (*[512] * 64, *[4096] * 16, *[1 << 18] * 16, *[1 << 25] * 4)
    taken = [torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)
    for t in taken:
        assert bool((t == 0x7f).all())


def test_binding_refusals():
    """What the binding checks before the library sees it: types, shapes, layouts and places of the tensors."""
    rng = np.random.default_rng(23)
    inp, _ = _tree_case(rng, [3, 2], [40, 20], 8, 2, 64, 16, False)
    dev = {k: v.cuda() for k, v in inp.items()}
    N = 5
    for change in (dict(q=dev["q"].half()), dict(q=dev["q"][:, ::2]), dict(q=inp["q"]), dict(q=dev["q"][0]),
                   dict(k_cache=dev["k_cache"][..., :32].contiguous()), dict(v_cache=dev["v_cache"][:-1].contiguous()),
                   dict(v_cache=dev["v_cache"].float()), dict(block_table=dev["block_table"].long()),
                   dict(context_lens=inp["context_lens"]), dict(token_start=dev["token_start"][:-1].contiguous()),
                   dict(parents=dev["parents"][1:].contiguous()), dict(k_cache_scale=torch.ones(3, device="cuda")),
                   dict(q=None)):
        with pytest.raises(ValueError):
            dsa.dsa_tree_attn({**dev, **change}, 3, 40)
    for kw in (dict(out=torch.empty_like(dev["q"])[:-1]), dict(out=torch.empty(N, 8, 64, device="cuda")),
               dict(lse=torch.empty(N, 7, device="cuda")), dict(ws=torch.empty(1 << 22, device="cuda"))):
        with pytest.raises(ValueError):
            dsa.dsa_tree_attn(dev, 3, 40, **kw)
    for kw in (dict(sm_scale=float("nan")), dict(ws=torch.empty(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(dsa.DSAError):
            dsa.dsa_tree_attn(dev, 3, 40, **kw)
    with pytest.raises(ValueError):
        dsa.dsa_tree_attn(dev, 2 ** 40, 40)                  # does not fit the C argument
    x, pos, table = torch.randn(4, 2, 64, device="cuda"), _dev(np.arange(4)), dsa.dsa_rope_freqs(64)
    for args, kw in (((x.double(), pos, table), {}), ((x, pos[:3], table), {}), ((x, pos.long(), table), {}),
                     ((x.transpose(0, 1), pos[:2], table), {}), ((x, pos, table), dict(k=x[:3])),
                     ((x, pos, table), dict(k=x.bfloat16())), ((x, pos, table), dict(q_out=x[:, :1])),
                     ((x, pos, table), dict(k=x, k_out=x.cpu()))):
        with pytest.raises(ValueError):
            dsa.dsa_rope(*args, **kw)
    P, i = torch.full((3, 10), 0.1, device="cuda"), _dev(np.zeros(3))
    good = [P, None, i, _dev([-1, 0, 1]), _dev([0, 3]), torch.rand(3, device="cuda"), torch.rand(1, device="cuda")]
    for at, bad in ((0, P.half()), (0, P[0]), (1, P[:, :9].contiguous()), (2, i[:2]), (3, i.long()), (4, i[:1]),
                    (5, P[0, :2].contiguous()), (6, P)):
        with pytest.raises(ValueError):
            dsa.dsa_verify_tree(*[bad if k == at else v for k, v in enumerate(good)])
    with pytest.raises(ValueError):
        dsa.dsa_verify_tree(*good, max_path=4, path=torch.empty((1, 5), dtype=torch.int32, device="cuda"))
    pool = dict(block_table=_dev(np.zeros((2, 4))), context_lens=_dev([0, 0]), pages_held=_dev([0, 0]),
                free_pages=_dev([1, 2]), free_count=_dev([2]))
    for change in (dict(block_table=_dev(np.zeros(8))), dict(context_lens=_dev([0])), dict(free_count=_dev([2, 2])),
                   dict(free_pages=torch.zeros(4, device="cuda"))):
        with pytest.raises(ValueError):
            dsa.dsa_blocks_trim({**pool, **change}, _dev([0, 0]), 16)
