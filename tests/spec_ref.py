"""Plain 64-bit references of the speculative-decoding operators (numpy, one
sequence, row or token at a time, from the operators' definitions)."""
import math

import numpy as np

BF16_HALF = 2.0 ** -8        # largest relative error of one rounding to bf16
F32_HALF = 2.0 ** -24


def e4m3_values(codes):
    """E4M3 (finite, no infinity) codes as float64."""
    c = codes.astype(np.int64)
    sign = np.where(c & 0x80, -1.0, 1.0)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    return sign * np.where((c & 0x7F) == 0x7F, np.nan, v)


# ------------------------------------------------------------------ rotary positions

def rope_freqs(rot_dim, base=10000.0, scaling="none", factor=1.0, original_context=4096, beta_fast=32.0, beta_slow=1.0):
    """Radians a position of each pair."""
    out = []
    for i in range(rot_dim // 2):
        f = base ** (-2.0 * i / rot_dim)
        if scaling == "linear":
            f /= factor
        elif scaling == "yarn":
            def t(beta):
                return rot_dim * math.log(original_context / (2 * math.pi * beta)) / (2 * math.log(base))
            low, high = max(math.floor(t(beta_fast)), 0), min(math.ceil(t(beta_slow)), rot_dim - 1)
            r = min(1.0, max(0.0, (i - low) / max(high - low, 0.001)))
            f = f * (1 - r) + f / factor * r
        out.append(f)
    return np.array(out)


def rope(x, positions, radians, begin, interleaved, factor=1.0, inverse=False):
    """x float64 [rows, H, d] -> (rotated, bound on the sum of the two products' magnitudes)."""
    half = len(radians)
    y, mag = x.copy(), np.abs(x)
    for i in range(half):
        a, c = (begin + 2 * i, begin + 2 * i + 1) if interleaved else (begin + i, begin + half + i)
        angle = positions.astype(np.float64) * radians[i] * (-1 if inverse else 1)
        co, si = np.cos(angle)[:, None], np.sin(angle)[:, None]
        y[:, :, a] = factor * (x[:, :, a] * co - x[:, :, c] * si)
        y[:, :, c] = factor * (x[:, :, c] * co + x[:, :, a] * si)
        mag[:, :, a] = mag[:, :, c] = abs(factor) * (np.abs(x[:, :, a]) + np.abs(x[:, :, c]))
    return y, mag


# ------------------------------------------------------------------ block tables

def extend(pool, new_lens, ps, num_pages, max_tokens):
    """The pool (dict of numpy arrays) grown in place -> (plan, error)."""
    bt, ctx, held = pool["block_table"], pool["context_lens"], pool["pages_held"]
    free, count = pool["free_pages"], int(pool["free_count"][0])
    seqs, pos, slots, start, err = [], [], [], [0], False
    asked = offered = taken = 0
    for b, grow in enumerate(int(v) for v in new_lens):
        c, h = int(ctx[b]), int(held[b])
        if grow != 0 and (grow < 0 or c < 0 or h < 0 or h > bt.shape[1] or h * ps < c or c + grow > bt.shape[1] * ps):
            err, grow = True, 0
        need = max(0, -(-(c + grow) // ps) - h) if grow else 0
        asked += need
        if need and asked > count:
            err, grow = True, 0
        offered += grow
        if grow and offered > max_tokens:
            err, grow = True, 0
        if grow:
            for j in range(need):
                page = int(free[count - 1 - taken])
                taken += 1
                bt[b, h + j] = page if 0 <= page < num_pages else -1
            ctx[b], held[b] = c + grow, h + need
            for p in range(c, c + grow):
                page = int(bt[b, p // ps])
                ok = 0 <= page < num_pages
                err |= not ok
                seqs.append(b)
                pos.append(p)
                slots.append(page * ps + p % ps if ok else -1)
        start.append(len(seqs))
    pool["free_count"][0] = count - taken
    pad = [-1] * (max_tokens - len(seqs))
    return dict(token_start=np.array(start), seq_ids=np.array(seqs + pad), positions=np.array(pos + pad),
                slots=np.array(slots + pad, dtype=np.int64)), err


def trim(pool, keep_lens, ps, num_pages):
    bt, ctx, held, free = (pool[k] for k in ("block_table", "context_lens", "pages_held", "free_pages"))
    count, err, asked, back = int(pool["free_count"][0]), False, 0, []
    for b, keep in enumerate(int(v) for v in keep_lens):
        h = int(held[b])
        if keep < 0 or keep > ctx[b] or h < 0 or h > bt.shape[1]:
            err = True
            continue
        stay = min(h, -(-keep // ps))
        asked += h - stay
        if h > stay and count + asked > len(free):
            err = True
            continue
        for j in range(stay, h):
            page = int(bt[b, j])
            ok = 0 <= page < num_pages
            err |= not ok
            back.append(page if ok else -1)
            bt[b, j] = -1
        ctx[b], held[b] = keep, stay
    for i, page in enumerate(back):
        free[count + len(back) - 1 - i] = page
    pool["free_count"][0] = count + len(back)
    return err


# ------------------------------------------------------------------ tree attention

def ancestors(parents):
    """Node sets; None for a padding row, a row under one, and a parent that is not below its child."""
    out = []
    for i, p in enumerate(int(v) for v in parents):
        if p < -1 or p >= i or (p >= 0 and out[p] is None):
            out.append(None)
        else:
            out.append((out[p] if p >= 0 else []) + [i])
    return out


def tree_attn(q, K, V, ctx, parents, group, sm):
    """One sequence: q [n, H, d], K and V [ctx, H_kv, d], float64 ->
    out, lse, and bounds on the errors of both for bf16 weights and fp32 sums."""
    n, H, d = q.shape
    out, lse = np.zeros((n, H, d)), np.full((n, H), -np.inf)
    tol_o, tol_l = np.zeros((n, H, d)), np.zeros((n, H))
    for i, nodes in enumerate(ancestors(parents)):
        if nodes is None:
            continue
        rows = list(range(ctx - n)) + [ctx - n + j for j in nodes]
        for h in range(H):
            k, v = K[rows, h // group], V[rows, h // group]
            s = sm * (k @ q[i, h])
            m = s.max()
            p = np.exp(s - m)
            l = p.sum()
            out[i, h] = (p @ v) / l
            lse[i, h] = m + math.log(l)
            # a logit is a sum of d fp32 products, then scaled (and, FP8, scaled twice): at most
            # (d + 4) roundings of the sum of magnitudes; the exponent's argument rounds twice more
            # at the size of the running maximum, and 2^x itself is good to 2^-22
            delta = (d + 4) * F32_HALF * (sm * (np.abs(k) @ np.abs(q[i, h]))).max() + 4 * F32_HALF * (
                abs(m) * 1.4427 + 16) + 2.0 ** -22
            sums = (len(rows) + 64) * F32_HALF
            weighed = (p @ np.abs(v)) / l
            # weights to bf16 (FP8: after V's scale); numerator and denominator both carry delta
            # fp32 ends at 2^-126: a weight, held relative to a maximum at most 2^8 below the largest, or
            # its product with V's scale (a code is at most 448 < 2^9 of them), is lost below 2^-126 of it
            floor = len(rows) * 2.0 ** (-126 + 8 + 9) * max(1.0, np.abs(v).max())
            tol_o[i, h] = weighed * (BF16_HALF * 1.01 + 2.1 * delta + 2 * sums) + np.abs(out[i, h]) * BF16_HALF * 1.01 + floor
            tol_l[i, h] = 1.1 * delta + sums + 4 * F32_HALF * (abs(lse[i, h]) + abs(m) + 1)
    return out, lse, tol_o, tol_l


# ------------------------------------------------------------------ verification

def verify(target, draft, tokens, parents, u_accept, u_sample, max_path):
    """One sequence's rows -> (path, next token or -1)."""
    n, V = len(tokens), target.shape[1]
    if n == 0:
        return [], -1
    path, cur, R, Z = [0], 0, target[0].astype(np.float64), 1.0
    i = 1
    while i < n and len(path) < max_path:
        if parents[i] == cur and 0 <= tokens[i] < V:
            x = int(tokens[i])
            Q = np.zeros(V) if draft is None else draft[cur].astype(np.float64)
            if draft is None:
                Q[x] = 1.0
            if float(u_accept[i]) * Q[x] * Z < R[x]:
                path.append(i)
                cur, R, Z = i, target[i].astype(np.float64), 1.0
            else:
                rest = np.maximum(R / Z - Q, 0.0)
                if rest.sum() > 0:
                    R, Z = rest, rest.sum()
        i += 1
    run = np.cumsum(R)
    if not (run[-1] > 0 and np.isfinite(run[-1])):
        return path, -1
    above = np.nonzero(run > float(u_sample) * run[-1])[0]
    return path, int(above[0]) if above.size else int(np.nonzero(R > 0)[0][-1])


# ------------------------------------------------------------------ compaction

def compact(caches, block_table, context_lens, token_start, path, accept_len, N, num_pages, ps):
    """Rows of the caches (dict of numpy arrays [pages, ps, ...]) moved in place -> (keep_lens, error)."""
    keep, err = [], False
    for b, ctx in enumerate(int(v) for v in context_lens):
        t0, t1, length = int(token_start[b]), int(token_start[b + 1]), int(accept_len[b])
        n, room = t1 - t0, block_table.shape[1] * ps
        ok = 0 <= t0 <= t1 <= N and n <= 128 and n <= ctx <= room and 0 <= length <= min(n, path.shape[1])
        steps = [int(v) for v in path[b, :length]] if ok else []
        ok = ok and all(p < n and p > q for p, q in zip(steps, [-1] + steps))
        moves = [(ctx - n + p, ctx - n + i) for i, p in enumerate(steps)] if ok else []
        ok = ok and all(0 <= block_table[b, at // ps] < num_pages for m in moves for at in m)
        if not ok:
            err = True
            keep.append(ctx)
            continue
        for src, dst in moves:
            s, t = ((int(block_table[b, at // ps]), at % ps) for at in (src, dst))
            for c in caches.values():
                c[t] = c[s]
        keep.append(ctx - n + length)
    return np.array(keep), err
