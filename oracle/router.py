"""Plain 64-bit statements of the router operators: the scored top-k gate, its gradient, the
block plan of a batch and the experts' token lists.

They restate the definitions of ``include/moeroute.h`` in numpy, row by row or request by
request where that is the plainest form, and share no code with the kernels.
"""
from __future__ import annotations

import numpy as np

NEG = -np.inf


def scores(x, score):
    """Scores of rows x [..., E] in 64 bits; masked experts (-inf, NaN) have 0, and so have
    sigmoids under the smallest normal fp32 number."""
    x = np.where(np.isnan(x), NEG, np.asarray(x, dtype=np.float64))
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            s = np.where(x == NEG, 0.0, 1.0 / (1.0 + np.exp(-x)))
        return np.where(s < 2.0 ** -126, 0.0, s)
    m = x.max(-1, keepdims=True)
    with np.errstate(invalid="ignore"):
        e = np.where(x == NEG, 0.0, np.where(x == m, 1.0, np.exp(x - m)))
    z = e.sum(-1, keepdims=True)
    return np.where(z > 0, e / np.where(z > 0, z, 1.0), 0.0)


def _order(c):
    """Indices by descending value, ties to the lower index, NaN last."""
    nan = np.isnan(c)
    v = np.where(nan, 0.0, -c)
    return np.lexsort((np.arange(len(c)), v, nan))


def choice_row(x, s, b, n_group, top_group, best):
    """What one row's experts are ordered by (nan: lowest; None where the group is dropped is
    nan below everything, given as the second result's False), and the margin by which the
    last kept group leads the first dropped one."""
    E = len(x)
    masked = np.isnan(x) | (x == NEG)
    by_score = np.where(np.isnan(x), np.nan, np.where(masked, NEG, s + (0.0 if b is None else b)))
    rank = by_score if b is not None else np.where(np.isnan(x), np.nan, x)
    kept = np.ones(E, dtype=bool)
    margin = np.inf
    if n_group > 1 and top_group < n_group:
        src = by_score if (b is not None or best == 2) else rank
        g = np.empty(n_group)
        for i, part in enumerate(np.split(src, n_group)):
            top = -np.sort(-np.where(np.isnan(part), NEG, part))[:best]
            v = top.sum() if not (np.isinf(top).any() and np.isnan(top.sum())) else NEG
            g[i] = v
        o = _order(g)
        kept[:] = False
        for i in o[:top_group]:
            kept[i * (E // n_group):(i + 1) * (E // n_group)] = True
        with np.errstate(invalid="ignore"):
            d = g[o[top_group - 1]] - g[o[top_group]]
        exact = b is None and best == 1
        margin = np.inf if exact or np.isnan(d) else d
    return rank, kept, margin


def score_topk(x, k, score="softmax", renorm=True, bias=None, n_group=1, top_group=1, best=1, scale=1.0):
    """x [L][T][E] -> ids [L][T][k], weights [L][T][k], score_sum [L][E], gap [L][T]: how far
    apart the closest two of the leading choices (and the groups) are; inf where the order is
    by the logits themselves, which has no rounding."""
    x = np.asarray(x, dtype=np.float64)
    L, T, E = x.shape
    s = scores(x, score)
    ids = np.zeros((L, T, k), dtype=np.int64)
    gap = np.full((L, T), np.inf)
    for l in range(L):
        b = None if bias is None else np.asarray(bias[l], dtype=np.float64)
        for t in range(T):
            rank, kept, margin = choice_row(x[l, t], s[l, t], b, n_group, top_group, best)
            o = _order(rank)
            o = o[kept[o]]
            ids[l, t] = o[:k]
            gap[l, t] = margin
            if b is not None:
                v = rank[o[:k + 1]]
                with np.errstate(invalid="ignore"):
                    d = np.abs(v[:-1] - v[1:])
                d = d[~np.isnan(d)]
                if len(d):
                    gap[l, t] = min(margin, d.min())
    if renorm and score == "softmax":
        w = scores(np.take_along_axis(x, ids, -1), "softmax")
    else:
        w = np.take_along_axis(s, ids, -1)
        if renorm:
            z = w.sum(-1, keepdims=True)
            w = np.where(z > 0, w / np.where(z > 0, z, 1.0), 0.0)
    return ids, w * scale, s.sum(1), gap


def score_topk_grad(x, ids, d_weights, d_score_sum=None, score="softmax", renorm=True, scale=1.0):
    """The gradient of sum(weights * d_weights) + sum(score_sum * d_score_sum) by x, with the ids
    fixed, and a bound on the terms that add up to each entry (for tolerances)."""
    x = np.asarray(x, dtype=np.float64)
    L, T, E = x.shape
    s = scores(x, score)
    a = np.zeros((L, 1, E)) if d_score_sum is None else np.asarray(d_score_sum, dtype=np.float64)[:, None, :]
    slope = s * (1.0 - s) if score == "sigmoid" else None
    dx, mag = np.zeros_like(x), np.zeros_like(x)
    g = np.asarray(d_weights, dtype=np.float64) * scale
    if score == "softmax":
        for sign in (0, 1):  # the value, then its terms' sizes
            aa, gg = (a, g) if sign == 0 else (np.abs(a), np.abs(g))
            pm = -1.0 if sign == 0 else 1.0
            out = s * (aa + pm * (aa * s).sum(-1, keepdims=True))
            if renorm:
                q = scores(np.take_along_axis(x, ids, -1), "softmax")
                part = q * (gg + pm * (gg * q).sum(-1, keepdims=True))
            else:
                p = np.take_along_axis(s, ids, -1)
                dot = (gg * p).sum(-1, keepdims=True)
                out = out + pm * s * dot
                part = gg * p
            for l in range(L):
                for t in range(T):
                    np.add.at(out[l, t], ids[l, t], part[l, t])
            (dx if sign == 0 else mag)[:] = out
        return dx, mag
    for sign in (0, 1):
        aa, gg = (a, g) if sign == 0 else (np.abs(a), np.abs(g))
        pm = -1.0 if sign == 0 else 1.0
        out = aa * slope
        part = gg
        if renorm:
            p = np.take_along_axis(s, ids, -1)
            z = p.sum(-1, keepdims=True)
            r = np.where(z > 0, 1.0 / np.where(z > 0, z, 1.0), 0.0)
            part = (gg + pm * (gg * p).sum(-1, keepdims=True) * r) * r
        part = part * np.take_along_axis(slope, ids, -1)
        for l in range(L):
            for t in range(T):
                np.add.at(out[l, t], ids[l, t], part[l, t])
        (dx if sign == 0 else mag)[:] = out
    return dx, mag


def block_plan(new_len, ctx_len, B, pages=None, free=None):
    """The plan of a batch, request by request; `pages` (int [R][width]) is filled in place."""
    tok0 = 0
    out = {k: [] for k in ("blk_tab", "insert_slot", "cache_idx", "slot_map", "tok_req", "tok_pos")}
    req, blk, cac = [0], [0], [0]
    taken = 0
    for r, (n, c) in enumerate(zip(new_len, ctx_len)):
        n, c = max(int(n), 0), max(int(c), 0)
        row = pages[r] if pages is not None else None
        if row is not None and free is not None:
            for i in range(-(-c // B), -(-(c + n) // B)):
                row[i] = free[taken]
                taken += 1
        else:
            taken += -(-(c + n) // B) - -(-c // B)
        for i in range(c // B):
            out["cache_idx"].append(row[i] if row is not None else -1)
        p = c
        while p < c + n:
            end = min(c + n, (p // B + 1) * B)
            page = int(row[p // B]) if row is not None else -1
            out["blk_tab"].append((tok0 + p - c, end - p))
            out["insert_slot"].append(page if end - p == B else -1)
            for q in range(p, end):
                out["slot_map"].append(page * B + q % B if page >= 0 else -1)
                out["tok_req"].append(r)
                out["tok_pos"].append(q)
            p = end
        tok0 += n
        req.append(tok0)
        blk.append(len(out["blk_tab"]))
        cac.append(len(out["cache_idx"]))
    res = {k: np.asarray(v, dtype=np.int64) for k, v in out.items()}
    res["blk_tab"] = res["blk_tab"].reshape(-1, 2)
    res.update(req_off=np.asarray(req), req_blk_off=np.asarray(blk), req_cache_off=np.asarray(cac),
               totals=np.asarray([tok0, blk[-1], cac[-1], taken]))
    return res


def expert_order(ids, E, align, ld):
    """Per layer the pairs of each expert in ascending order, segments padded to `align`; ids
    >= E belong to nobody."""
    L = ids.shape[0]
    flat = ids.reshape(L, -1)
    off = np.zeros((L, E + 1), dtype=np.int64)
    order = np.full((L, ld), -1, dtype=np.int64)
    inv = np.full(flat.shape, -1, dtype=np.int64)
    for l in range(L):
        at = 0
        for e in range(E):
            off[l, e] = at
            mine = np.flatnonzero(flat[l] == e)
            order[l, at:at + len(mine)] = mine
            inv[l, mine] = at + np.arange(len(mine))
            at += -(-len(mine) // align) * align
        off[l, E] = at
    return off, order, inv.reshape(ids.shape)
