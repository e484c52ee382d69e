"""Host-only checks of the speculative-decoding entry points: refusals before
anything is launched, and the rotary frequency table (host arithmetic)."""
import ctypes

import numpy as np
import pytest

import spec_ref
from long_context_fp8_b200 import build as dsa_build

OK, INVALID, UNSUP, WS = 0, 1, 2, 3
P = ctypes.c_void_p
FAKE = P(0x1000)             # never dereferenced: every call fails validation, or has nothing to do
ODD = P(0x1001)


@pytest.fixture(scope="module")
def lib():
    dsa_build.build()
    from long_context_fp8_b200 import dsa
    return dsa.load()


def _call(fn, args, **change):
    return fn(*[change.get(k, v) for k, v in args.items()])


@pytest.mark.parametrize("kw", [dict(rot_dim=64), dict(rot_dim=128, base=500000.0), dict(rot_dim=2),
                                dict(rot_dim=64, scaling="linear", factor=8.0),
                                dict(rot_dim=64, scaling="yarn", factor=40.0),
                                dict(rot_dim=256, scaling="yarn", factor=4.0, original_context=32768, base=1e6),
                                dict(rot_dim=128, scaling="yarn", factor=1.0, original_context=1)])
def test_rope_frequencies(lib, kw):
    from long_context_fp8_b200 import dsa
    got = np.array(list(dsa.dsa_rope_freqs(**kw)), dtype=np.float64) / 2.0 ** 64
    ref = spec_ref.rope_freqs(**kw) / (2 * np.pi)
    # 64-bit arithmetic on both sides: a few roundings of pow and log
    assert np.all(np.abs(got - ref) <= 1e-13 * ref + 2.0 ** -63)


def test_rope_frequency_refusals(lib):
    from long_context_fp8_b200 import dsa
    for kw in (dict(rot_dim=0), dict(rot_dim=63), dict(rot_dim=258), dict(rot_dim=64, base=1.0),
               dict(rot_dim=64, base=float("nan")), dict(rot_dim=64, scaling="linear", factor=0.5),
               dict(rot_dim=64, scaling="yarn", factor=2.0, original_context=0),
               dict(rot_dim=64, scaling="yarn", factor=2.0, beta_fast=1.0, beta_slow=1.0),
               dict(rot_dim=64, scaling="yarn", factor=2.0, beta_slow=0.0)):
        with pytest.raises(dsa.DSAError) as e:
            dsa.dsa_rope_freqs(**kw)
        assert e.value.status == INVALID
    assert lib.dsa_rope_freqs(64, 10000.0, 7, 1.0, 4096, 32.0, 1.0, FAKE) == INVALID
    assert lib.dsa_rope_freqs(64, 10000.0, 0, 1.0, 4096, 32.0, 1.0, None) == INVALID


def test_rope_refusals(lib):
    turns = (ctypes.c_uint64 * 32)()
    a = dict(q=FAKE, qs=16 * 128, hq=16, k=FAKE, ks=128, hk=1, pos=FAKE, rows=4, d=128, begin=0, dim=64, inter=0,
             turns=ctypes.addressof(turns), f=1.0, inv=0, qo=P(0x2000), qos=16 * 128, ko=P(0x3000), kos=128, dt=1,
             st=None)
    for bad in (dict(q=None), dict(q=ODD), dict(qo=None), dict(qo=ODD), dict(k=None), dict(ko=None), dict(k=ODD),
                dict(pos=None), dict(turns=None), dict(rows=-1), dict(d=0), dict(hq=0), dict(hk=-1), dict(dim=0),
                dict(begin=-8), dict(qs=16 * 128 - 8), dict(qs=16 * 128 + 4), dict(kos=64), dict(f=float("inf")),
                dict(hk=0), dict(qo=FAKE, qos=16 * 128 + 8)):
        assert _call(lib.dsa_rope, a, **bad) == INVALID, bad
    for bad in (dict(dt=2), dict(d=132, qs=16 * 132, qos=16 * 132, ks=136, kos=136), dict(begin=4), dict(dim=24),
                dict(begin=72), dict(dim=272, d=512, qs=16 * 512, qos=16 * 512, ks=512, kos=512),
                dict(d=2048, qs=16 * 2048, qos=16 * 2048, ks=2048, kos=2048), dict(rows=2 ** 31)):
        assert _call(lib.dsa_rope, a, **bad) == UNSUP, bad
    assert _call(lib.dsa_rope, a, rows=0) == OK
    assert _call(lib.dsa_rope, a, rows=0, q=None) == OK


def test_blocks_refusals(lib):
    a = dict(new=FAKE, ctx=FAKE, held=FAKE, bt=FAKE, free=FAKE, cap=10, count=FAKE, B=2, mp=4, P=20, ps=64, mt=8,
             ts=FAKE, seq=FAKE, pos=FAKE, slots=FAKE, status=None, st=None)
    for bad in (dict(new=None), dict(ctx=None), dict(held=None), dict(bt=None), dict(free=None), dict(count=None),
                dict(ts=None), dict(seq=None), dict(pos=None), dict(new=ODD), dict(slots=P(0x1008)), dict(B=-1),
                dict(cap=-1), dict(mt=-1), dict(mp=0), dict(P=0), dict(ps=0), dict(status=ODD)):
        assert _call(lib.dsa_blocks_extend, a, **bad) == INVALID, bad
    for bad in (dict(P=2 ** 31 // 64), dict(mp=2 ** 31 // 64), dict(cap=2 ** 31), dict(mt=2 ** 31)):
        assert _call(lib.dsa_blocks_extend, a, **bad) == UNSUP, bad
    assert _call(lib.dsa_blocks_extend, a, B=0, new=None) == OK
    t = {k: a[k] for k in ("new", "ctx", "held", "bt", "free", "cap", "count", "B", "mp", "P", "ps", "status", "st")}
    for bad in (dict(new=None), dict(ctx=None), dict(held=None), dict(bt=None), dict(free=None), dict(count=None),
                dict(new=ODD), dict(B=-1), dict(cap=-1), dict(mp=0), dict(P=0), dict(ps=-1), dict(status=ODD)):
        assert _call(lib.dsa_blocks_trim, t, **bad) == INVALID, bad
    assert _call(lib.dsa_blocks_trim, t, P=2 ** 31 // 64) == UNSUP
    assert _call(lib.dsa_blocks_trim, t, B=0, new=None) == OK


def test_tree_attn_refusals(lib):
    ws = lib.dsa_tree_attn_workspace_size(2, 10, 16, 1, 128)
    assert ws > 0 and ws % 256 == 0
    assert lib.dsa_tree_attn_workspace_size(0, 10, 16, 1, 128) == 0
    assert lib.dsa_tree_attn_workspace_size(2, 10, 16, 1, 96) == 0
    a = dict(q=FAKE, k=FAKE, ks=None, v=FAKE, vs=None, bt=FAKE, ctx=FAKE, ts=FAKE, par=FAKE, P=20, mp=4, ps=64, B=2,
             N=10, mt=8, mc=256, H=16, Hkv=1, d=128, sm=0.1, out=FAKE, lse=None, ws=FAKE, wsb=ws, st=None)
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(bt=None), dict(ctx=None), dict(ts=None), dict(par=None),
                dict(out=None), dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(out=ODD), dict(lse=ODD), dict(ks=FAKE),
                dict(vs=FAKE), dict(ks=ODD, vs=FAKE), dict(B=-1), dict(N=-1), dict(H=0), dict(Hkv=0), dict(d=0),
                dict(mt=0), dict(mc=0), dict(ps=0), dict(P=0), dict(mp=0), dict(sm=0.0), dict(sm=-0.1),
                dict(sm=float("nan")), dict(sm=float("inf")), dict(par=ODD)):
        assert _call(lib.dsa_tree_attn, a, **bad) == INVALID, bad
    for bad in (dict(d=96), dict(ps=24), dict(H=16, Hkv=3), dict(mt=129), dict(P=2 ** 31 // 64), dict(mp=2 ** 25),
                dict(B=65537), dict(N=2 ** 31)):
        assert _call(lib.dsa_tree_attn, a, **bad) == UNSUP, bad
    for bad in (dict(ws=None), dict(wsb=ws - 1), dict(ws=P(0x1080))):
        assert _call(lib.dsa_tree_attn, a, **bad) == WS, bad
    assert _call(lib.dsa_tree_attn, a, N=0, q=None) == OK
    assert _call(lib.dsa_tree_attn, a, B=0, q=None) == OK


def test_verify_refusals(lib):
    a = dict(p=FAKE, q=FAKE, tok=FAKE, par=FAKE, ts=FAKE, ua=FAKE, us=FAKE, B=2, N=10, V=100, mp=8, path=FAKE, acc=FAKE,
             nxt=FAKE, status=None, st=None)
    for bad in (dict(p=None), dict(tok=None), dict(par=None), dict(ts=None), dict(ua=None), dict(us=None),
                dict(path=None), dict(acc=None), dict(nxt=None), dict(p=P(0x1004)), dict(q=P(0x1008)), dict(tok=ODD),
                dict(B=-1), dict(N=-1), dict(V=0), dict(mp=0), dict(status=ODD)):
        assert _call(lib.dsa_verify_tree, a, **bad) == INVALID, bad
    for bad in (dict(V=2 ** 31), dict(N=2 ** 31), dict(B=2 ** 28)):
        assert _call(lib.dsa_verify_tree, a, **bad) == UNSUP, bad
    assert _call(lib.dsa_verify_tree, a, B=0, p=None) == OK


def test_compact_refusals(lib):
    a = dict(bt=FAKE, ctx=FAKE, ts=FAKE, path=FAKE, acc=FAKE, B=2, N=10, mp=8, pages=4, P=20, ps=64, dI=128, d=128,
             ki=FAKE, kis=FAKE, k=FAKE, ks=None, v=FAKE, vs=None, keep=None, status=None, st=None)
    for bad in (dict(bt=None), dict(ctx=None), dict(ts=None), dict(path=None), dict(acc=None), dict(k=None),
                dict(v=None), dict(ki=None), dict(kis=None), dict(ks=FAKE), dict(vs=FAKE), dict(k=P(0x1004)),
                dict(ki=P(0x1004)), dict(B=-1), dict(N=-1), dict(mp=0), dict(d=0), dict(dI=0), dict(pages=0),
                dict(P=0), dict(ps=0), dict(status=ODD), dict(keep=ODD)):
        assert _call(lib.dsa_cache_compact, a, **bad) == INVALID, bad
    for bad in (dict(dI=12), dict(d=6), dict(d=12, ks=FAKE, vs=FAKE), dict(P=2 ** 31 // 64)):
        assert _call(lib.dsa_cache_compact, a, **bad) == UNSUP, bad
    assert _call(lib.dsa_cache_compact, a, B=0, bt=None) == OK


def test_binding_refuses_host_tensors_and_wrong_types():
    import torch
    from long_context_fp8_b200 import dsa
    q = torch.zeros(2, 4, 64)
    with pytest.raises(ValueError):
        dsa.dsa_rope(q, torch.zeros(2, dtype=torch.int32), dsa.dsa_rope_freqs(64))
    with pytest.raises(ValueError):
        dsa.dsa_verify_tree(torch.zeros(2, 9), None, *[torch.zeros(2, dtype=torch.int32)] * 3, torch.zeros(2),
                            torch.zeros(1))


# ------------------------------------------------------------------ the references themselves

def test_reference_e4m3_matches_torch():
    import torch
    codes = torch.arange(256, dtype=torch.uint8)
    ref = codes.view(torch.float8_e4m3fn).double().numpy()
    got = spec_ref.e4m3_values(codes.numpy())
    assert np.array_equal(np.isnan(ref), np.isnan(got)) and np.array_equal(ref[~np.isnan(ref)], got[~np.isnan(got)])


def test_reference_trim_undoes_extend():
    rng = np.random.default_rng(0)
    for _ in range(20):
        B, ps, width = 6, 16, 12
        ctx = rng.integers(0, 100, B)
        held = -(-ctx // ps)
        order = rng.permutation(200)
        bt = np.full((B, width), -1)
        used = 0
        for b in range(B):
            bt[b, :held[b]] = order[used:used + held[b]]
            used += held[b]
        pool = dict(block_table=bt, context_lens=ctx.copy(), pages_held=held.copy(),
                    free_pages=np.append(order[used:], [-1] * 3), free_count=np.array([200 - used]))
        old = {k: v.copy() for k, v in pool.items()}
        plan, err = spec_ref.extend(pool, rng.integers(0, 60, B), ps, 200, 400)
        assert not err and np.unique(plan["slots"][plan["slots"] >= 0]).size == plan["token_start"][-1]
        assert not spec_ref.trim(pool, ctx, ps, 200)
        assert all(np.array_equal(pool[k], old[k]) for k in pool)


def test_reference_verification_follows_the_target():
    """Two children drawn from q, verified: the first emitted token's frequencies
    are the target's.  Exactly, by summing over a grid of the random numbers."""
    p, q = np.array([0.5, 0.3, 0.15, 0.05]), np.array([0.1, 0.2, 0.3, 0.4])
    target = np.stack([p] + [np.full(4, 0.25)] * 2).astype(np.float64)
    draft = np.stack([q] * 3).astype(np.float64)
    grid = (np.arange(25) + 0.5) / 25
    got = np.zeros(4)
    for x1 in range(4):
        for x2 in range(4):
            w = q[x1] * q[x2] / 25 ** 3
            for u1 in grid:
                for u2 in grid:
                    for us in grid:
                        path, nxt = spec_ref.verify(target, draft, [0, x1, x2], [-1, 0, 0], [0, u1, u2], us, 2)
                        got[[0, x1, x2][path[1]] if len(path) > 1 else nxt] += w
    # each of the three uniforms on 25 cells: a border inside a cell moves at most half of it
    assert np.all(np.abs(got - p) <= 3 * 0.5 / 25)
