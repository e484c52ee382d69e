"""Cases of the speculative-decoding operators over the paged caches: their
sizes, inputs, plain forms and 64-bit values.

One step of speculative decoding reserves cache slots for a tree of drafted
tokens ("blocks"), rotates the new queries and keys to their positions
("rope"), attends the tree over the cached context ("tree"), verifies the
drafts against the target's probabilities ("verify") and moves the accepted
tokens' cache rows together ("compact").
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a single short conversation, a small draft: latency alone counts
        dict(name="tree 1x700 h16", op="tree", batch=1, context=700, drafts=6, heads=16, kv_heads=1, dim=128, page=64,
             kv8=False),
        # the repository's decode workload (64K contexts, 128 heads on one K/V head) with 16 drafts a request
        dict(name="tree 16x64K h128", op="tree", batch=16, context=65536, drafts=16, heads=128, kv_heads=1, dim=128,
             page=64, kv8=False),
        # grouped heads, small pages, medium contexts, a batch of short drafts: the K/V bytes bound it
        dict(name="tree 32x8K h64/8", op="tree", batch=32, context=8191, drafts=8, heads=64, kv_heads=8, dim=128,
             page=16, kv8=False),
        # FP8 caches of the repository's decode workload at half the context, few drafts a request
        dict(name="tree kv8 64x32K h128", op="tree", batch=64, context=32768, drafts=3, heads=128, kv_heads=1, dim=128,
             page=64, kv8=True),
        # the drafted tokens of one decode step: 64 requests x 16 drafts, half of each head rotated
        dict(name="rope 1024x128 yarn", op="rope", rows=1024, heads=128, k_heads=1, dim=128, rot_begin=64, rot_dim=64,
             interleaved=True, scaling="yarn", dtype="bf16", inverse=False),
        # the index queries of a 16K prompt chunk in the gradient's direction, fp32
        dict(name="rope 16Kx64 inverse", op="rope", rows=16384, heads=64, k_heads=1, dim=128, rot_begin=0, rot_dim=64,
             interleaved=False, scaling="linear", dtype="f32", inverse=True),
        # a chain of four drafts of one request
        dict(name="verify 1x5 chain 32000", op="verify", batch=1, nodes=5, vocab=32000, chain=True, point=False),
        # a full batch of trees over a large vocabulary
        dict(name="verify 64x16 tree 128001", op="verify", batch=64, nodes=16, vocab=128001, chain=False, point=False),
        # every request of a decode step reserves 16 drafts and gives them back
        dict(name="blocks 64x16", op="blocks", batch=64, context=65536, new=16, page=64),
        # a batch of prompts enters and leaves
        dict(name="blocks 500x1000 prompts", op="blocks", batch=500, context=0, new=1000, page=16),
        # accepted paths of a full batch, FP8 K/V
        dict(name="compact 64x16 kv8", op="compact", batch=64, context=512, nodes=16, page=64, kv8=True),
        # accepted paths of the largest batch and trees, bf16 K/V
        dict(name="compact 256x64", op="compact", batch=256, context=300, nodes=64, page=32, kv8=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("tree", "tree", "tree", "rope", "rope", "verify", "verify", "blocks", "compact"))
    if op == "tree":
        heads, kv_heads = rng.choice(((16, 1), (128, 1), (64, 8), (32, 4), (24, 2), (8, 8), (256, 1), (40, 1)))
        dim, page, kv8 = rng.choice((64, 128, 128)), rng.choice((16, 32, 48, 64, 128)), rng.random() < 0.4
        drafts = rng.choice((1, 1, 2, 3, 5, 8, 13, 16, 24, 33, 48, 64))
        batch = _log(rng, 1, 64)
        most = min(65536, 2 ** 31 // (batch * drafts * heads), 2 ** 21 // (batch * kv_heads))
        context = _log(rng, drafts, max(drafts + 1, most))
        return dict(op=op, batch=batch, context=context, drafts=drafts, heads=heads, kv_heads=kv_heads, dim=dim,
                    page=page, kv8=kv8)
    if op == "rope":
        dim = rng.choice((64, 128, 192))
        rot_dim = rng.choice((32, 64, dim))
        heads = rng.choice((1, 4, 16, 64, 128))
        return dict(op=op, rows=_log(rng, 1, 2 ** 20 // heads), heads=heads, k_heads=rng.choice((0, 1, 2)), dim=dim,
                    rot_begin=rng.choice((0, dim - rot_dim)), rot_dim=rot_dim, interleaved=rng.random() < 0.5,
                    scaling=rng.choice(("none", "linear", "yarn")), dtype=rng.choice(("bf16", "f32")),
                    inverse=rng.random() < 0.3)
    if op == "verify":
        nodes = rng.choice((1, 2, 4, 7, 16, 31, 64))
        vocab = _log(rng, 1000, 160000)
        return dict(op=op, batch=_log(rng, 1, max(1, min(128, 2 ** 27 // (nodes * vocab)))), nodes=nodes, vocab=vocab,
                    chain=rng.random() < 0.4, point=rng.random() < 0.3)
    if op == "blocks":
        batch = _log(rng, 1, 1024)
        return dict(op=op, batch=batch, context=rng.choice((0, 1, 100, 4000, 65000)), new=_log(rng, 1, 500000 // batch),
                    page=rng.choice((16, 32, 48, 64, 128)))
    return dict(op=op, batch=_log(rng, 1, 256), context=_log(rng, 64, 512), nodes=rng.choice((1, 2, 5, 8, 16, 33, 64)),
                page=rng.choice((16, 32, 48, 64, 128)), kv8=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs

def _lengths(g, batch, most, least):
    """Ragged lengths in [least, most], the first of them the longest."""
    u = torch.rand(batch, generator=g)
    n = (least + (most - least) * (0.5 + 0.5 * u)).long().clamp(least, most)
    n[0] = most
    return n


def _table(g, pages, width):
    """Pages of each sequence, drawn without repeats from a pool a little larger than needed; -1 behind them."""
    total = int(pages.sum())
    num_pages = total + 3
    ids = torch.randperm(num_pages, generator=g)[:total].int()
    table = torch.full((pages.numel(), width), -1, dtype=torch.int32)
    held = torch.arange(width)[None, :] < pages[:, None]
    table[held] = ids
    return table, num_pages


def _tree(g, nodes, chain=False):
    """Parents of each row of drafts (`nodes`: drafts of each sequence): -1 for the first, then an earlier node,
    most often one of the last few."""
    width = int(nodes.max())
    i = torch.arange(width)[None, :].expand(nodes.numel(), width)
    back = 1 + (torch.rand(nodes.numel(), width, generator=g) ** 2 * i.clamp(max=6)).long()
    parents = i - 1 if chain else i - back.clamp(max=i.clamp(min=1))
    parents = torch.where(i == 0, torch.full_like(i, -1), parents)
    return parents[i < nodes[:, None]].int()


def _starts(n):
    return torch.cat([torch.zeros(1, dtype=torch.long), n.cumsum(0)]).int()


def _codes(rows, dim, g):
    """E4M3 codes and one scale a row of normal values."""
    x = torch.randn(rows + (dim,), generator=g, device=DEV)
    scale = x.abs().amax(-1) / 448.0
    return (x / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), scale


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(DEV).manual_seed(seed)
    # lengths, and with them the outputs' shapes, belong to the case; what lies in them, to the seed
    gs = torch.Generator().manual_seed(sum(v for v in case.values() if isinstance(v, int)))
    s = dict(case)
    return globals()["_prepare_" + case["op"]](s, gs, g, gd)


def _prepare_tree(s, gs, g, gd):
    B, n = s["batch"], s["drafts"]
    # the last sequence of a larger batch has no drafts in this step
    drafts = torch.randint((n + 1) // 2, n + 1, (B,), generator=gs)
    drafts[0] = n
    if B > 4:
        drafts[B - 1] = 0
    ctx = torch.maximum(_lengths(gs, B, s["context"], min(s["context"], n)), drafts.clamp(min=1))
    pages = (ctx + s["page"] - 1) // s["page"]
    table, num_pages = _table(g, pages, int(pages.max()) + 1)
    shape = (num_pages, s["page"], s["kv_heads"])
    N = int(drafts.sum())
    inp = dict(q=(1.5 * torch.randn((N, s["heads"], s["dim"]), generator=gd, device=DEV)).bfloat16(),
               block_table=table.to(DEV), context_lens=ctx.int().to(DEV), token_start=_starts(drafts).to(DEV),
               parents=_tree(g, drafts).to(DEV))
    for x in ("k", "v"):
        if s["kv8"]:
            inp[x + "_cache"], inp[x + "_cache_scale"] = _codes(shape, s["dim"], gd)
        else:
            inp[x + "_cache"] = torch.randn(shape + (s["dim"],), generator=gd, device=DEV).bfloat16()
    s["inp"], s["max_drafts"], s["max_context"] = inp, n, s["context"]
    s["out"], s["lse"] = torch.empty_like(inp["q"]), torch.empty((N, s["heads"]), device=DEV)
    if own:
        from long_context_fp8_b200 import dsa
        s["ws"] = dsa.workspace(dsa.tree_attn_workspace_size(B, N, s["heads"], s["kv_heads"], s["dim"]), DEV)
    return s


#: Long-context scaling of the rotary cases: factor, original context, and the ramp's turns; the yarn factor on q and k.
ROPE = dict(base=10000.0, factor=40.0, original_context=4096, beta_fast=32.0, beta_slow=1.0)


def _rope_kw(s):
    return dict(ROPE, scaling=s["scaling"]), (0.1 * math.log(ROPE["factor"]) + 1.0 if s["scaling"] == "yarn" else 1.0)


def _prepare_rope(s, gs, g, gd):
    t = torch.bfloat16 if s["dtype"] == "bf16" else torch.float32
    s["q"] = torch.randn((s["rows"], s["heads"], s["dim"]), generator=gd, device=DEV).to(t)
    s["k"] = torch.randn((s["rows"], s["k_heads"], s["dim"]), generator=gd, device=DEV).to(t) if s["k_heads"] else None
    s["positions"] = torch.randint(0, 1 << 20, (s["rows"],), generator=gd, device=DEV, dtype=torch.int32)
    s["q_out"] = torch.empty_like(s["q"])
    s["k_out"] = torch.empty_like(s["k"]) if s["k_heads"] else None
    kw, s["attn_factor"] = _rope_kw(s)
    s["freqs"] = _inv_freqs(s["rot_dim"], **kw).to(DEV)
    if own:
        from long_context_fp8_b200 import dsa
        s["table"] = dsa.dsa_rope_freqs(s["rot_dim"], **kw)
    return s


def _prepare_verify(s, gs, g, gd):
    B, n, V = s["batch"], s["nodes"], s["vocab"]
    nodes = torch.randint((n + 1) // 2, n + 1, (B,), generator=gs)
    nodes[0] = n
    parents, N = _tree(g, nodes, s["chain"]), int(nodes.sum())
    start = _starts(nodes)
    logits = 2.5 * torch.randn((N, V), generator=gd, device=DEV)
    s["target"] = logits.softmax(-1)
    logits += 0.7 * torch.randn((N, V), generator=gd, device=DEV)
    s["draft"] = logits.softmax(-1)
    # each drafted token is drawn from its parent's draft distribution
    row = parents.long() + start[:-1].long().repeat_interleave(nodes)
    row = torch.where(parents < 0, torch.arange(N), row).to(DEV)
    u = torch.rand((N, 1), generator=gd, device=DEV)
    s["tokens"] = torch.searchsorted(s["draft"].cumsum(-1)[row], u)[:, 0].clamp(max=V - 1).int()
    if s["point"]:
        s["draft"] = None
    s["parents"], s["start"] = parents.to(DEV), start.to(DEV)
    s["u_accept"] = torch.rand((N,), generator=gd, device=DEV)
    s["u_sample"] = torch.rand((B,), generator=gd, device=DEV)
    s["path"] = torch.empty((B, n), dtype=torch.int32, device=DEV)
    s["accepted"] = torch.empty((B,), dtype=torch.int32, device=DEV)
    s["next"] = torch.empty((B,), dtype=torch.int32, device=DEV)
    return s


def _prepare_blocks(s, gs, g, gd):
    B, ps = s["batch"], s["page"]
    ctx = _lengths(gs, B, s["context"], min(1, s["context"]))
    new = _lengths(gs, B, s["new"], 1)
    held = (ctx + ps - 1) // ps
    need = (ctx + new + ps - 1) // ps - held
    table, _ = _table(g, held, int((held + need).max()) + 2)
    spare = int(need.sum()) + 5
    s["num_pages"] = int(held.sum()) + spare
    order = torch.randperm(s["num_pages"], generator=g).int()
    table[table >= 0] = order[: int(held.sum())]
    free = torch.cat([order[int(held.sum()):], torch.full((7,), -1, dtype=torch.int32)])
    s["pool"] = dict(block_table=table.to(DEV), context_lens=ctx.int().to(DEV), pages_held=held.int().to(DEV),
                     free_pages=free.to(DEV), free_count=torch.tensor([spare], dtype=torch.int32, device=DEV))
    s["new_lens"], s["keep"] = new.int().to(DEV), ctx.int().to(DEV)
    s["max_tokens"] = int(new.sum()) + 3
    s["plan"] = dict(token_start=torch.empty(B + 1, dtype=torch.int32, device=DEV),
                     seq_ids=torch.empty(s["max_tokens"], dtype=torch.int32, device=DEV),
                     positions=torch.empty(s["max_tokens"], dtype=torch.int32, device=DEV),
                     slots=torch.empty(s["max_tokens"], dtype=torch.int64, device=DEV))
    return s


def _prepare_compact(s, gs, g, gd):
    B, n, ps = s["batch"], s["nodes"], s["page"]
    nodes = torch.randint((n + 1) // 2, n + 1, (B,), generator=gs)
    nodes[0] = n
    ctx = nodes + _lengths(gs, B, s["context"], 1)
    pages = (ctx + ps - 1) // ps
    table, num_pages = _table(g, pages, int(pages.max()) + 1)
    # an accepted path: the root, then later nodes in order
    take = (torch.rand((B, n), generator=g) < 0.4) & (torch.arange(n)[None, :] < nodes[:, None])
    take[:, 0] = True
    i = torch.arange(n)[None, :].expand(B, n)
    path = torch.where(take, i, torch.full_like(i, n)).sort(-1).values
    path = torch.where(path == n, torch.full_like(path, -1), path).int()
    caches = {}
    caches["kidx_cache"], caches["kscale_cache"] = _codes((num_pages, ps), 128, gd)
    for x in ("k", "v"):
        if s["kv8"]:
            caches[x + "_cache"], caches[x + "_cache_scale"] = _codes((num_pages, ps), 128, gd)
        else:
            caches[x + "_cache"] = torch.randn((num_pages, ps, 128), generator=gd, device=DEV).bfloat16()
    s["caches"], s["table"], s["context_lens"] = caches, table.to(DEV), ctx.int().to(DEV)
    s["start"], s["path"] = _starts(nodes).to(DEV), path.to(DEV)
    s["accepted"] = take.sum(-1).int().to(DEV)
    s["keep"] = torch.empty((B,), dtype=torch.int32, device=DEV)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        from long_context_fp8_b200 import dsa
        return _OWN[s["op"]](s, dsa)
    return _PLAIN[s["op"]](s)


def _own_tree(s, dsa):
    return dsa.dsa_tree_attn(s["inp"], s["max_drafts"], s["max_context"], out=s["out"], lse=s["lse"], ws=s["ws"])


def _own_rope(s, dsa):
    q, k = dsa.dsa_rope(s["q"], s["positions"], s["table"], k=s["k"], rot_begin=s["rot_begin"],
                        interleaved=s["interleaved"], attn_factor=s["attn_factor"], inverse=s["inverse"],
                        q_out=s["q_out"], k_out=s["k_out"])
    return [q, k]


def _own_verify(s, dsa):
    return dsa.dsa_verify_tree(s["target"], s["draft"], s["tokens"], s["parents"], s["start"], s["u_accept"],
                               s["u_sample"], path=s["path"], accept_len=s["accepted"], next_token=s["next"])


def _own_blocks(s, dsa):
    plan = dsa.dsa_blocks_extend(s["pool"], s["new_lens"], s["page"], s["num_pages"], s["max_tokens"], plan=s["plan"])
    dsa.dsa_blocks_trim(s["pool"], s["keep"], s["page"])
    return [plan, s["pool"]]


def _own_compact(s, dsa):
    dsa.dsa_cache_compact(s["caches"], s["table"], s["context_lens"], s["start"], s["path"], s["accepted"],
                          keep_lens=s["keep"])
    return [_values(s["caches"]), s["keep"]]


def _values(caches):
    return {k: v.view(torch.float8_e4m3fn) if v.dtype == torch.uint8 else v for k, v in caches.items()}


# ------------------------------------------------------------------ plain forms

def _padded(start, width):
    """[B, width] rows of packed tokens and which of them exist."""
    i = torch.arange(width, device=DEV)[None, :]
    n = (start[1:] - start[:-1]).long()[:, None]
    return torch.where(i < n, start[:-1].long()[:, None] + i, 0), i < n


def _ancestors(parents):
    """[B, n, n] truth values: node j is node i or one of its ancestors, from padded parents [B, n] (-1: none)."""
    n = parents.shape[1]
    reach = torch.eye(n, device=DEV)[None] + (parents[:, :, None] == torch.arange(n, device=DEV)).float()
    for _ in range(max(1, (n - 1).bit_length())):
        reach = ((reach @ reach) > 0).float()
    return reach > 0


def _plain_tree(s):
    p, H, hk, d = s["inp"], s["heads"], s["kv_heads"], s["dim"]
    rows, here = _padded(p["token_start"], s["max_drafts"])
    ctx, n = p["context_lens"].long(), (p["token_start"][1:] - p["token_start"][:-1]).long()
    pos = torch.arange(s["max_context"], device=DEV)
    page = p["block_table"].long()[:, (pos // s["page"]).clamp(max=p["block_table"].shape[1] - 1)].clamp(min=0)
    slot = page * s["page"] + pos % s["page"]
    alive = pos[None, :] < ctx[:, None]

    def rows_of(x):
        c = p[x + "_cache"].flatten(0, 1)[slot]
        if s["kv8"]:
            c = c.view(torch.float8_e4m3fn).float() * p[x + "_cache_scale"].flatten(0, 1)[slot][..., None]
        return torch.where(alive[:, :, None, None], c.float(), 0).permute(0, 2, 3, 1)    # [B, hk, d, S]

    B, w, g = rows.shape[0], rows.shape[1], H // hk
    q = p["q"][rows].float().view(B, w, hk, g, d).permute(0, 2, 1, 3, 4).reshape(B, hk, w * g, d)
    x = (q / math.sqrt(d)) @ rows_of("k")
    tree = _ancestors(torch.where(here, p["parents"].long()[rows], -1))
    j = pos[None, :] - (ctx - n)[:, None]
    seen = (j < 0)[:, None, :] | torch.gather(tree, 2, j.clamp(0, w - 1)[:, None, :].expand(B, w, -1))
    seen = (seen & alive[:, None, :])[:, None, :, None, :].expand(B, 1, w, g, -1).reshape(B, 1, w * g, -1)
    x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x @ rows_of("v").transpose(-1, -2)) / total
    lse = (top + total.log())[..., 0]
    o = o.view(B, hk, w, g, d).permute(0, 2, 1, 3, 4).reshape(B, w, H, d)[here]
    lse = lse.view(B, hk, w, g).permute(0, 2, 1, 3).reshape(B, w, H)[here]
    return [o.bfloat16(), lse]


def _inv_freqs(rot_dim, base, scaling, factor, original_context, beta_fast, beta_slow):
    """Radians a position turns each pair by, in 64 bits."""
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    f = base ** (-2.0 * i / rot_dim)
    if scaling == "linear":
        return f / factor
    if scaling == "yarn":
        def turns(beta):
            return rot_dim * math.log(original_context / (beta * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(turns(beta_fast)), 0), min(math.ceil(turns(beta_slow)), rot_dim - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        return f * (1 - ramp) + f / factor * ramp
    return f


def _plain_rope(s):
    angle = s["positions"].double()[:, None, None] * s["freqs"]
    sign = -1.0 if s["inverse"] else 1.0
    cos, sin = (angle.cos() * s["attn_factor"]).float(), (sign * angle.sin() * s["attn_factor"]).float()
    b, r = s["rot_begin"], s["rot_dim"]

    def turned(x):
        if x is None:
            return None
        y = x[..., b:b + r].float()
        if s["interleaved"]:
            a, c = y[..., 0::2], y[..., 1::2]
            z = torch.stack([a * cos - c * sin, c * cos + a * sin], -1).flatten(-2)
        else:
            a, c = y[..., : r // 2], y[..., r // 2:]
            z = torch.cat([a * cos - c * sin, c * cos + a * sin], -1)
        return torch.cat([x[..., :b], z.to(x.dtype), x[..., b + r:]], -1)

    return [turned(s["q"]), turned(s["k"])]


def _plain_verify(s):
    B, n, V = s["batch"], s["nodes"], s["vocab"]
    rows, here = _padded(s["start"], n)
    parents = torch.where(here, s["parents"][rows], -2)
    tokens, u = s["tokens"][rows].long(), s["u_accept"][rows].double()
    b = torch.arange(B, device=DEV)
    cur = torch.zeros(B, dtype=torch.long, device=DEV)
    path = torch.full((B, n), -1, dtype=torch.int32, device=DEV)
    path[:, 0] = 0
    count = torch.ones(B, dtype=torch.long, device=DEV)
    left, mass = s["target"][rows[:, 0]].double(), torch.ones(B, dtype=torch.float64, device=DEV)
    # children come after their parents and are tried in order: one pass over the nodes is the whole walk
    for i in range(1, n):
        tried = parents[:, i] == cur
        x, at = tokens[:, i], rows[b, cur]
        if s["draft"] is None:
            other = torch.zeros_like(left).scatter_(1, x[:, None], 1.0)
        else:
            other = s["draft"][at].double()
        ok = tried & (u[:, i] * other[b, x] * mass < left[b, x])
        less = (left / mass[:, None] - other).clamp(min=0)
        sum_less = less.sum(-1)
        no = tried & ~ok & (sum_less > 0)
        left = torch.where(no[:, None], less, torch.where(ok[:, None], s["target"][rows[:, i]].double(), left))
        mass = torch.where(no, sum_less, torch.where(ok, 1.0, mass))
        path[b, torch.where(ok, count, 0)] = torch.where(ok, i, 0).int()
        count, cur = count + ok, torch.where(ok, i, cur)
    run_sum = left.cumsum(-1)
    above = run_sum > (s["u_sample"].double() * run_sum[:, -1])[:, None]
    return [path, count.int(), above.int().argmax(-1).int()]


def _plain_blocks(s):
    pool, ps, B = s["pool"], s["page"], s["batch"]
    ctx, held, new = (x.long() for x in (pool["context_lens"], pool["pages_held"], s["new_lens"]))
    table, width = pool["block_table"].long(), pool["block_table"].shape[1]
    total = ctx + new
    need = torch.where(new > 0, ((total + ps - 1) // ps - held).clamp(min=0), 0)
    fits = (total <= width * ps) & (need.cumsum(0) <= pool["free_count"])
    new = torch.where(fits, new, 0)
    new = torch.where(new.cumsum(0) <= s["max_tokens"], new, 0)
    need = torch.where(new > 0, need, 0)
    first = need.cumsum(0) - need
    col = torch.arange(width, device=DEV)[None, :]
    fresh = (col >= held[:, None]) & (col < (held + need)[:, None])
    stack = (pool["free_count"].long() - 1 - first[:, None] - (col - held[:, None])).clamp(0, pool["free_pages"].numel() - 1)
    table = torch.where(fresh, pool["free_pages"].long()[stack], table)
    start = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), new.cumsum(0)])
    t = torch.arange(s["max_tokens"], device=DEV)
    seq = torch.searchsorted(start[1:], t, right=True)
    real = seq < B
    seq = seq.clamp(max=B - 1)
    position = ctx[seq] + t - start[seq]
    slot = table[seq, (position // ps).clamp(max=width - 1)] * ps + position % ps
    ctx, held, count = ctx + new, held + need, pool["free_count"].long() - need.sum()
    plan = dict(token_start=start.int(), seq_ids=torch.where(real, seq, -1).int(),
                positions=torch.where(real, position, -1).int(), slots=torch.where(real, slot, -1))
    # the tokens are given back: pages behind the kept length return to the stack, the first of them on top
    keep = s["keep"].long()
    stay = torch.minimum(held, (keep + ps - 1) // ps)
    gone = (col >= stay[:, None]) & (col < held[:, None])
    free, back = pool["free_pages"].clone(), table[gone].int()
    free[count + torch.arange(back.numel() - 1, -1, -1, device=DEV)] = back
    return [plan, dict(block_table=torch.where(gone, -1, table).int(), context_lens=keep.int(), pages_held=stay.int(),
                       free_pages=free, free_count=(count + back.numel()).int())]


def _plain_compact(s):
    ps, n = s["page"], s["start"][1:] - s["start"][:-1]
    first = (s["context_lens"] - n).long()[:, None]
    i = torch.arange(s["path"].shape[1], device=DEV)[None, :]
    real = i < s["accepted"][:, None]

    def slots(at):
        at = torch.where(real, at, 0)
        return (torch.gather(s["table"].long(), 1, at // ps) * ps + at % ps)[real]

    src, dst = slots(first + s["path"]), slots(first + i)
    for x in s["caches"].values():
        rows = x.flatten(0, 1)
        rows[dst] = rows[src]
    return [_values(s["caches"]), s["context_lens"] - n + s["accepted"]]


_OWN = dict(tree=_own_tree, rope=_own_rope, verify=_own_verify, blocks=_own_blocks, compact=_own_compact)
_PLAIN = dict(tree=_plain_tree, rope=_plain_rope, verify=_plain_verify, blocks=_plain_blocks, compact=_plain_compact)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "tree":
        n, B, H = 0.75 * case["drafts"], case["batch"], case["heads"]
        keys = 0.75 * case["context"] * B
        row = case["kv_heads"] * (case["dim"] + 4 if case["kv8"] else 2 * case["dim"])
        return dict(bytes=2 * keys * row + 4 * n * B * H * case["dim"], flops=4 * n * keys * H * case["dim"])
    if op == "rope":
        n = case["rows"] * (case["heads"] + case["k_heads"])
        return dict(bytes=2 * n * case["dim"] * (2 if case["dtype"] == "bf16" else 4) + 4 * case["rows"],
                    flops=3 * n * case["rot_dim"])
    if op == "verify":
        # one row of each distribution is summed for each sequence, the others are read at one token
        n = case["batch"] * case["vocab"]
        return dict(bytes=n * (4 if case["point"] else 8), flops=3 * n)
    if op == "blocks":
        return dict(bytes=case["batch"] * (0.75 * case["new"] * (16 + 8.0 / case["page"]) + 40), flops=0)
    row = 132 + (264 if case["kv8"] else 512)
    return dict(bytes=case["batch"] * 0.4 * 0.75 * case["nodes"] * 2 * row, flops=0)


# ------------------------------------------------------------------ the values in 64 bits

def exact(case, seed):
    if case["op"] == "tree":
        return _exact_tree(prepare(case, seed))
    if case["op"] == "rope":
        return _exact_rope(prepare(case, seed))
    if case["op"] == "compact":
        return _exact_compact(prepare(case, seed))
    return None     # whole numbers


def _exact_tree(s):
    """Sequence by sequence: softmax over the context before the drafts and each draft's ancestors."""
    p, g = s["inp"], s["heads"] // s["kv_heads"]
    start, ctx, table = p["token_start"].tolist(), p["context_lens"].tolist(), p["block_table"].long()
    parents = p["parents"].tolist()
    out = torch.zeros(p["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(out.shape[:2], dtype=torch.float64, device=DEV)
    for b, c in enumerate(ctx):
        t0, n = start[b], start[b + 1] - start[b]
        if n == 0:
            continue
        at = torch.arange(c, device=DEV)
        pg, off = table[b, at // s["page"]], at % s["page"]

        def rows_of(x):
            r = p[x + "_cache"][pg, off]
            if s["kv8"]:
                return r.view(torch.float8_e4m3fn).double() * p[x + "_cache_scale"][pg, off].double()[..., None]
            return r.double()

        hide = torch.zeros((n, c), dtype=torch.bool)
        hide[:, c - n:] = True
        for i in range(n):
            j = i
            while j >= 0:
                hide[i, c - n + j] = False
                j = parents[t0 + j]
        hide, K, V = hide.to(DEV), rows_of("k"), rows_of("v")
        for h in range(s["kv_heads"]):
            heads = slice(h * g, (h + 1) * g)
            x = torch.einsum("ngd,sd->ngs", p["q"][t0:t0 + n, heads].double(), K[:, h]) / math.sqrt(s["dim"])
            x.masked_fill_(hide[:, None, :], -math.inf)
            lse[t0:t0 + n, heads] = torch.logsumexp(x, -1)
            out[t0:t0 + n, heads] = torch.einsum("ngs,sd->ngd", torch.softmax(x, -1), V[:, h])
    return [out, lse]


def _exact_rope(s):
    """Each pair as a complex number times attn_factor * e^(+-i angle), the frequencies' formulas written out."""
    kw, f = _rope_kw(s)
    r, w = s["rot_dim"], []
    for i in range(r // 2):
        x = math.exp(-2.0 * i / r * math.log(kw["base"]))
        if kw["scaling"] == "linear":
            x /= kw["factor"]
        if kw["scaling"] == "yarn":
            at = [r / 2 * math.log(kw["original_context"] / (2 * math.pi * t)) / math.log(kw["base"])
                  for t in (kw["beta_fast"], kw["beta_slow"])]
            low, high = max(0, math.floor(at[0])), min(r - 1, math.ceil(at[1]))
            old = 1.0 - min(1.0, max(0.0, (i - low) / max(high - low, 0.001)))
            x = x * old + x / kw["factor"] * (1.0 - old)
        w.append(x)
    angle = s["positions"].double()[:, None] * torch.tensor(w, dtype=torch.float64, device=DEV)
    turn = torch.polar(torch.full_like(angle, f), -angle if s["inverse"] else angle)[:, None, :]

    def turned(x):
        if x is None:
            return None
        y = x.double()
        z = y[..., s["rot_begin"]:s["rot_begin"] + r]
        if s["interleaved"]:
            z.copy_(torch.view_as_real(torch.view_as_complex(z.unflatten(-1, (r // 2, 2)).contiguous()) * turn).flatten(-2))
        else:
            c = torch.complex(z[..., : r // 2].contiguous(), z[..., r // 2:].contiguous()) * turn
            z.copy_(torch.cat([c.real, c.imag], -1))
        return y

    return [turned(s["q"]), turned(s["k"])]


def _exact_compact(s):
    """Row by row, in the order of the path."""
    caches = {k: (v.view(torch.float8_e4m3fn) if v.dtype == torch.uint8 else v).double().cpu() for k, v in s["caches"].items()}
    table, ctx, start = s["table"].tolist(), s["context_lens"].tolist(), s["start"].tolist()
    ps = s["page"]
    for b, path in enumerate(s["path"].tolist()):
        first = ctx[b] - (start[b + 1] - start[b])
        for i, j in enumerate(path):
            if j >= 0:
                for x in caches.values():
                    x[table[b][(first + i) // ps], (first + i) % ps] = x[table[b][(first + j) // ps], (first + j) % ps]
    return [caches, None]
