"""What is measured of the router operators: scored top-k and its gradient, block plans and
expert orders.

A case is a dict of plain values.  ``prepare`` makes its inputs on the GPU, ``run`` makes one
pass: with ``own`` false in elementary torch operations in 32 bits, with ``own`` true through
the library's entry points.  ``exact`` gives the floating outputs from the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
MARGIN = 4e-6  # choice scores closer than this are drawn again: 32 bits do not order them


def _score(name, op, T, L, E, k, dtype, score, renorm, bias, groups, kept, best, sums, layout, scale=1.0):
    """A case of the scored top-k (op "score") or of its gradient (op "grad")."""
    return {"name": name, "op": op, "T": T, "L": L, "E": E, "k": k, "dtype": dtype, "score": score, "renorm": renorm,
            "bias": bias, "groups": groups, "kept": kept, "best": best, "sums": sums, "layout": layout, "scale": scale}


def listed():
    return [
        # one layer's router call while decoding a batch of 32 requests: latency
        _score("score_decode", "score", 32, 1, 128, 8, "f32", "softmax", True, False, 1, 1, 1, False, "layer"),
        # a prefill batch of 65,536 tokens over the 48 MoE layers of the 128-expert model
        _score("score_prefill", "score", 65536, 48, 128, 8, "f32", "softmax", True, False, 1, 1, 1, False, "layer"),
        # balance by bias: sigmoid scores, 8 groups of which 4 stay, scaled weights, 256 experts, an odd token count
        _score("score_groups", "score", 8209, 26, 256, 8, "bf16", "sigmoid", True, True, 8, 4, 2, False, "layer", 2.5),
        # training step of the 64-expert, k = 6 model: softmax weights as they are, token-major
        # logits, and the score sums that a balance loss takes
        _score("score_train", "score", 30011, 26, 64, 6, "bf16", "softmax", False, False, 1, 1, 1, True, "token"),
        # the gradient of a small fine-tuning batch at one layer
        _score("grad_layer", "grad", 1000, 1, 128, 8, "f32", "softmax", True, False, 1, 1, 1, False, "layer"),
        # the training step's backward pass: softmax weights and a balance loss, token-major
        _score("grad_train", "grad", 30011, 26, 64, 6, "bf16", "softmax", False, False, 1, 1, 1, True, "token"),
        # backward pass of renormalised sigmoid scores over 256 experts
        _score("grad_sigmoid", "grad", 16384, 48, 256, 8, "bf16", "sigmoid", True, False, 8, 4, 2, False, "layer", 2.5),
        # one decode step of 256 requests with long contexts: one new token each, a page where one begins
        {"name": "plan_decode", "op": "plan", "R": 256, "block": 16, "median": 1, "ctx": 8192, "reuse": 1.0, "cached": False},
        # the online stream: 14,000 requests, 30 % of them on a cached prefix
        {"name": "plan_stream", "op": "plan", "R": 14000, "block": 16, "median": 700, "ctx": 500, "reuse": 0.3, "cached": True},
        # a decode batch of 64 tokens at one layer, expert segments padded to tiles of 16 rows
        {"name": "order_decode", "op": "order", "T": 64, "L": 1, "E": 128, "k": 8, "align": 16, "skew": 1.0},
        # a prefill batch at every layer of the 128-expert model, tiles of 128 rows
        {"name": "order_prefill", "op": "order", "T": 65536, "L": 48, "E": 128, "k": 8, "align": 128, "skew": 1.0},
        # strongly skewed loads over 64 experts, k = 6, an odd token count, no padding
        {"name": "order_skewed", "op": "order", "T": 30011, "L": 26, "E": 64, "k": 6, "align": 1, "skew": 3.0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["score", "score", "grad", "grad", "plan", "order"])
    if op == "plan":
        return {"op": op, "R": _log_int(rng, 1, 14000), "block": rng.choice([8, 16, 32, 64]),
                "median": _log_int(rng, 1, 700), "ctx": _log_int(rng, 16, 8192 if rng.random() < 0.3 else 500),
                "reuse": rng.choice([0.0, 0.3, 1.0]), "cached": rng.random() < 0.5}
    E = rng.choice([16, 32, 60, 64, 64, 72, 96, 128, 128, 160, 192, 256, 256])
    k = rng.choice([1, 2, 4, 6, 8, 8, 8, 10])
    L = rng.choice([1, 1, 2, 16, 26, 48])
    if op == "order":
        T = _log_int(rng, 1, min(131072, 65536 * 48 * 8 // (L * k)))
        return {"op": op, "T": T, "L": L, "E": E, "k": k, "align": rng.choice([1, 1, 16, 64, 128]), "skew": rng.choice([0.0, 1.0, 3.0])}
    groups, kept, best = rng.choice([(1, 1, 1), (1, 1, 1), (4, 2, 1), (4, 2, 2), (8, 4, 2)])
    if E % groups or E // groups * kept < k or E // groups < best:
        groups, kept, best = 1, 1, 1
    score = rng.choice(["softmax", "sigmoid"])
    bias = op == "score" and score == "sigmoid" and rng.random() < 0.7
    most = 48_000_000 if bias or best == 2 or op == "grad" else 400_000_000
    T = _log_int(rng, 1, min(131072, most // (L * E)))
    c = _score("", op, T, L, E, k, rng.choice(["f32", "f32", "bf16", "bf16", "f16"]), score, k > 1 and rng.random() < 0.6, bias, groups, kept,
               best, rng.random() < 0.3, rng.choice(["layer", "layer", "token"]), rng.choice([1.0, 2.5]))
    del c["name"]
    return c


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _choice64(x, b, c):
    """Choice scores in 64 bits of rows x [n, E] with biases b [n, E] or None, those of dropped
    groups at -inf, and how near the last kept group is to the first dropped one."""
    s = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, -1)
    ch = s if b is None else s + b
    near = torch.full(x.shape[:1], math.inf, device=x.device, dtype=torch.float64)
    if c["groups"] > 1:
        by = ch.view(len(x), c["groups"], -1)
        g = by.sort(dim=-1, descending=True).values[..., :c["best"]].sum(-1)
        v, at = g.sort(dim=-1, descending=True, stable=True)
        near = (v[:, :-1] - v[:, 1:]).amin(-1)
        keep = torch.zeros_like(g, dtype=torch.bool).scatter_(1, at[:, :c["kept"]], True)
        ch = by.masked_fill(~keep[:, :, None], -math.inf).view(len(x), -1)
    return ch, near


def _unsettled(logits, bias, c, todo):
    """Those of the rows `todo` (layer * T + token) whose order 32 bits do not settle."""
    l, t = todo // logits.shape[1], todo % logits.shape[1]
    ch, near = _choice64(logits[l, t].double(), None if bias is None else bias[l].double(), c)
    if bias is not None:  # without a bias the logits themselves order a group's experts
        v = ch.sort(dim=-1, descending=True).values[:, :min(c["k"] + 1, ch.shape[1])]
        near = torch.minimum(near, (v[:, :-1] - v[:, 1:]).nan_to_num(math.inf, posinf=math.inf).amin(-1) if v.shape[1] > 1 else near)
    return todo[near < MARGIN]


def _make_logits(c, seed):
    """Router logits as [L, T, E] (a view where the layout is token-major): some experts are
    more popular than others at each layer."""
    gen = _gen(seed)
    T, L, E = c["T"], c["L"], c["E"]
    x = torch.randn((L, T, E) if c["layout"] == "layer" else (T, L, E), device="cuda", generator=gen).mul_(1.5)
    x = x if c["layout"] == "layer" else x.permute(1, 0, 2)
    x = x.add_(torch.randn((L, 1, E), device="cuda", generator=gen) * 0.5).to(DTYPES[c["dtype"]])
    bias = torch.randn((L, E), device="cuda", generator=gen) * 0.05 if c["bias"] else None
    return x, bias, gen


def _lengths(c, seed):
    """New and held tokens of each request: the same lengths for every seed, in another order."""
    R, rs = c["R"], np.random.RandomState(1)
    new = np.ones(R) if c["median"] == 1 else np.clip(np.rint(rs.lognormal(math.log(c["median"]), 0.75, R)), 1, 4096)
    ctx = np.where(rs.random_sample(R) < c["reuse"], rs.lognormal(math.log(c["ctx"]), 0.5, R), 0)
    ctx = np.minimum(ctx, 32768)
    if c["median"] > 1:  # a prefix is reused in whole blocks; a decode context ends anywhere
        ctx = ctx // c["block"] * c["block"]
    at = np.random.RandomState(seed & 0x7FFFFFFF).permutation(R)
    return new[at].astype(np.int32), ctx[at].astype(np.int32)


def prepare(case, seed):
    c = case
    if c["op"] == "plan":
        new, ctx = _lengths(c, seed)
        B, R = c["block"], c["R"]
        have = -(-ctx // B)
        need = -(-(ctx.astype(np.int64) + new) // B) - have
        width = int((have + need).max())
        pool = torch.randperm(int(have.sum() + need.sum()) + 64, device="cuda", generator=_gen(seed)).to(torch.int32)
        pages = torch.full((R, width), -1, dtype=torch.int32, device="cuda")
        held = torch.from_numpy(have.astype(np.int64)).cuda()
        pages[torch.arange(width, device="cuda")[None, :] < held[:, None]] = pool[:int(have.sum())]
        n = new.astype(np.int64)
        nblk = -(-((ctx % B) + n) // B)
        st = {"case": c, "new": torch.from_numpy(new).cuda(), "ctx": torch.from_numpy(ctx).cuda(), "pages": pages,
              "free": pool[int(have.sum()):].clone(), "T": int(n.sum()), "nblk": int(nblk.sum()),
              "ncached": int((ctx // B).sum()) if c["cached"] else 0, "need": int(need.sum())}
        return st
    if c["op"] == "order":
        gen = _gen(seed)
        T, L, E, k = c["T"], c["L"], c["E"], c["k"]
        ids = torch.empty((L, T, k), dtype=torch.uint8, device="cuda")
        pop = torch.randn((L, E), device="cuda", generator=gen) * c["skew"]
        for l in range(L):  # k distinct experts, by perturbed popularity
            z = pop[l] - torch.log(-torch.log(torch.rand((T, E), device="cuda", generator=gen).clamp_(1e-7, 1 - 1e-7)))
            ids[l] = z.topk(k, -1).indices.to(torch.uint8)
        return {"case": c, "ids": ids}
    x, bias, gen = _make_logits(c, seed)
    if c["op"] == "score" and (c["bias"] or c["best"] > 1):
        # rows whose order 32 bits do not settle are drawn again: either answer would be right there
        todo = torch.arange(c["L"] * c["T"], device="cuda")
        for _ in range(12):
            todo = _unsettled(x, bias, c, todo)
            if not len(todo):
                break
            x[todo // c["T"], todo % c["T"]] = (torch.randn((len(todo), c["E"]), device="cuda", generator=gen) * 1.5).to(x.dtype)
    st = {"case": c, "logits": x, "bias": bias}
    if c["op"] == "grad":
        st["ids"] = torch.empty((c["L"], c["T"], c["k"]), dtype=torch.uint8, device="cuda")
        for l in range(c["L"]):
            st["ids"][l] = x[l].float().topk(c["k"], -1).indices.to(torch.uint8)
        st["dw"] = torch.randn((c["L"], c["T"], c["k"]), device="cuda", generator=gen)
        st["da"] = torch.randn((c["L"], c["E"]), device="cuda", generator=gen) * 0.1 if c["sums"] else None
    return st


# ---------------------------------------------------------------- the plain forms
def _scores(x, c):
    if c["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    e = torch.exp(x - x.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _plain_score(st):
    c = st["case"]
    x = st["logits"].float()
    L, T, E = x.shape
    s = _scores(x, c)
    ch = x if st["bias"] is None else s + st["bias"][:, None, :]
    if c["groups"] > 1:
        by = (ch if c["best"] == 1 or st["bias"] is not None else s).view(L, T, c["groups"], -1)
        g = by.sort(dim=-1, descending=True).values[..., :c["best"]].sum(-1)
        keep = torch.zeros_like(g, dtype=torch.bool)
        keep.scatter_(-1, g.sort(dim=-1, descending=True, stable=True).indices[..., :c["kept"]], True)
        ch = torch.where(keep[..., None], ch.view(L, T, c["groups"], -1), -math.inf).view(L, T, E)
    ids = ch.sort(dim=-1, descending=True, stable=True).indices[..., :c["k"]]
    w = s.gather(-1, ids)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    out = {"ids": ids.to(torch.uint8), "weights": w * c["scale"]}
    if c["sums"]:
        out["score_sum"] = s.sum(1)
    return out


def _plain_grad(st):
    c = st["case"]
    x = st["logits"].float()
    s = _scores(x, c)
    ids = st["ids"].long()
    g = st["dw"] * c["scale"]
    if c["renorm"]:  # through w = s / sum of the chosen s
        sel = s.gather(-1, ids)
        total = sel.sum(-1, keepdim=True)
        g = (g - (g * sel).sum(-1, keepdim=True) / total) / total
    ds = torch.zeros_like(s) if st["da"] is None else st["da"][:, None, :].expand_as(s).clone()
    ds.scatter_add_(-1, ids, g)
    if c["score"] == "sigmoid":
        dx = ds * s * (1.0 - s)
    else:
        dx = s * (ds - (ds * s).sum(-1, keepdim=True))
    return dx.to(st["logits"].dtype)


def _plain_plan(st):
    c, B = st["case"], st["case"]["block"]
    new, ctx, pages = st["new"].long(), st["ctx"].long(), st["pages"]
    R, dev = c["R"], new.device
    zero = torch.zeros(1, dtype=torch.int64, device=dev)
    have = (ctx + B - 1) // B
    need = (ctx + new + B - 1) // B - have
    nb = torch.where(new > 0, (ctx % B + new + B - 1) // B, 0)
    rows = torch.arange(R, device=dev)
    off = torch.cat([zero, new.cumsum(0)])
    boff = torch.cat([zero, nb.cumsum(0)])
    noff = need.cumsum(0) - need
    # new pages of the block tables, in request order
    nr = torch.repeat_interleave(rows, need, output_size=st["need"])
    ni = torch.arange(st["need"], device=dev) - noff[nr]
    pages[nr, have[nr] + ni] = st["free"][:st["need"]]
    # token maps
    tr = torch.repeat_interleave(rows, new, output_size=st["T"])
    pos = ctx[tr] + torch.arange(st["T"], device=dev) - off[tr]
    slot = pages[tr, pos // B].long() * B + pos % B
    # blocks of the computed tokens
    br = torch.repeat_interleave(rows, nb, output_size=st["nblk"])
    first = ctx[br] // B + torch.arange(st["nblk"], device=dev) - boff[br]
    lo = torch.maximum(first * B, ctx[br])
    hi = torch.minimum(first * B + B, ctx[br] + new[br])
    tab = torch.stack([off[br] + lo - ctx[br], hi - lo], -1).to(torch.int32)
    out = {"req_off": off.to(torch.int32), "req_blk_off": boff.to(torch.int32), "blk_tab": tab, "pages": pages, "slot_map": slot,
           "insert_slot": torch.where(hi - lo == B, pages[br, first], -1), "tok_req": tr.to(torch.int32), "tok_pos": pos.to(torch.int32)}
    if c["cached"]:
        nc = ctx // B
        coff = torch.cat([zero, nc.cumsum(0)])
        cr = torch.repeat_interleave(rows, nc, output_size=st["ncached"])
        out["req_cache_off"] = coff.to(torch.int32)
        out["cache_idx"] = pages[cr, torch.arange(st["ncached"], device=dev) - coff[cr]]
    return out


def _order_rows(c):
    pairs, a = c["T"] * c["k"], c["align"]
    return pairs + min(c["E"], pairs) * (a - 1)


def _plain_order(st):
    c = st["case"]
    L, E, n, a = c["L"], c["E"], c["T"] * c["k"], c["align"]
    ids = st["ids"].view(L, n)
    sorted_ids, perm = ids.sort(dim=-1, stable=True)
    key = sorted_ids.long()
    cnt = torch.zeros((L, E), dtype=torch.int64, device=ids.device).scatter_add_(1, key, torch.ones_like(key))
    padded = (cnt + a - 1) // a * a
    off = torch.nn.functional.pad(padded.cumsum(1), (1, 0))
    first = cnt.cumsum(1) - cnt
    row = off.gather(1, key) + torch.arange(n, device=ids.device) - first.gather(1, key)
    order = torch.full((L, _order_rows(c)), -1, dtype=torch.int32, device=ids.device)
    order.scatter_(1, row, perm.to(torch.int32))
    inv = torch.empty((L, n), dtype=torch.int32, device=ids.device).scatter_(1, perm, row.to(torch.int32))
    return {"off": off.to(torch.int32), "order": order, "inv": inv.view(L, c["T"], c["k"])}


# ---------------------------------------------------------------- the library's calls
def _open(st):
    """What a program keeps between calls: shapes, options, outputs and a workspace."""
    from moe_expert_routing_top_gb300 import _native as nat
    c = st["case"]
    dev = "cuda"
    i32 = torch.int32
    h = {"nat": nat}
    if c["op"] == "plan":
        R, T, nb = c["R"], st["T"], st["nblk"]
        o = {"req_off": torch.empty(R + 1, dtype=i32, device=dev), "req_blk_off": torch.empty(R + 1, dtype=i32, device=dev),
             "blk_tab": torch.empty((nb, 2), dtype=i32, device=dev), "pages": st["pages"],
             "slot_map": torch.empty(T, dtype=torch.int64, device=dev), "insert_slot": torch.empty(nb, dtype=i32, device=dev),
             "tok_req": torch.empty(T, dtype=i32, device=dev), "tok_pos": torch.empty(T, dtype=i32, device=dev)}
        if c["cached"]:
            o["req_cache_off"] = torch.empty(R + 1, dtype=i32, device=dev)
            o["cache_idx"] = torch.empty(st["ncached"], dtype=i32, device=dev)
        h["out"] = o
        h["ws"] = torch.zeros(nat.moer_block_plan_workspace_bytes(R), dtype=torch.uint8, device=dev)
        h["plan"] = nat.make_block_plan(
            R=R, block=c["block"], T=T, nblk=nb, ncached=st["ncached"], ctx_len=st["ctx"], new_len=st["new"],
            free_pages=st["free"], n_free=len(st["free"]), ld_pages=st["pages"].shape[1], **o)
        return h
    h["dims"] = nat.make_dims(c["E"], c["k"], c["L"], [], 16)
    if c["op"] == "order":
        h["out"] = {"off": torch.empty((c["L"], c["E"] + 1), dtype=i32, device=dev),
                    "order": torch.empty((c["L"], _order_rows(c)), dtype=i32, device=dev),
                    "inv": torch.empty((c["L"], c["T"], c["k"]), dtype=i32, device=dev)}
        h["ws"] = torch.zeros(nat.moer_expert_order_workspace_bytes(h["dims"], c["T"]), dtype=torch.uint8, device=dev)
        return h
    h["opts"] = nat.make_score_opts(dtype=c["dtype"], score=c["score"], renorm=c["renorm"], n_group=c["groups"],
                                    top_group=c["kept"], group_best=c["best"], scale=c["scale"])
    h["ws"] = torch.zeros(nat.moer_score_workspace_bytes(h["dims"], c["T"]), dtype=torch.uint8, device=dev)
    if c["op"] == "grad":
        h["out"] = torch.empty_like(st["logits"])  # keeps the logits' layout
    else:
        h["out"] = {"ids": torch.empty((c["L"], c["T"], c["k"]), dtype=torch.uint8, device=dev),
                    "weights": torch.empty((c["L"], c["T"], c["k"]), dtype=torch.float32, device=dev)}
        if c["sums"]:
            h["out"]["score_sum"] = torch.empty((c["L"], c["E"]), dtype=torch.float32, device=dev)
    return h


def _own(st):
    h = st.get("handle")
    if h is None:
        h = st["handle"] = _open(st)
    c, nat, o, ws = st["case"], h["nat"], h["out"], h["ws"]
    if c["op"] == "plan":
        nat.moer_block_plan(h["plan"], ws, ws.numel())
    elif c["op"] == "order":
        nat.moer_expert_order(h["dims"], st["ids"], c["T"], c["align"], o["off"], o["order"], _order_rows(c), o["inv"], ws, ws.numel())
    elif c["op"] == "grad":
        x = st["logits"]
        nat.moer_score_topk_grad(h["dims"], h["opts"], x, c["T"], x.stride(1), x.stride(0), st["ids"], st["dw"], st["da"], o,
                                 o.stride(1), o.stride(0), ws, ws.numel())
    else:
        x = st["logits"]
        nat.moer_score_topk(h["dims"], h["opts"], x, c["T"], x.stride(1), x.stride(0), st["bias"], o["ids"], o["weights"],
                            o.get("score_sum"), ws, ws.numel())
    return o


def run(state):
    if own:
        return _own(state)
    return {"score": _plain_score, "grad": _plain_grad, "plan": _plain_plan, "order": _plain_order}[state["case"]["op"]](state)


def work(case):
    c = case
    if c["op"] == "plan":
        new, ctx = (a.astype(np.int64) for a in _lengths(c, 1))
        B = c["block"]
        T, nblk = int(new.sum()), int((-(-((ctx % B) + new) // B)).sum())
        nc = int((ctx // B).sum()) if c["cached"] else 0
        need = int((-(-(ctx + new) // B) - -(-ctx // B)).sum())
        return {"bytes": 16 * c["R"] + 16 * T + 12 * nblk + 4 * nblk + 8 * need + (8 * nc + 4 * c["R"] if c["cached"] else 0), "flops": 4 * T}
    rows = c["T"] * c["L"]
    if c["op"] == "order":
        return {"bytes": rows * c["k"] * 9 + 4 * c["L"] * (c["E"] + 1), "flops": 4 * rows * c["k"]}
    E, k, b = c["E"], c["k"], BYTES[c["dtype"]]
    if c["op"] == "grad":
        read = k * b if c["renorm"] and not c["sums"] else E * b  # only the chosen logits are needed there
        return {"bytes": rows * (read + E * b + 5 * k) + (4 * c["L"] * E if c["sums"] else 0), "flops": 8 * rows * E}
    return {"bytes": rows * (E * b + 5 * k) + 4 * c["L"] * E * (int(c["bias"]) + int(c["sums"])), "flops": 8 * rows * E}


# ---------------------------------------------------------------- from the definition, in 64 bits
def exact(case, seed):
    c = case
    if c["op"] in ("plan", "order"):
        return None
    st = prepare(c, seed)
    L, T, E, k = c["L"], c["T"], c["E"], c["k"]
    if c["op"] == "score":
        out = {"ids": None, "weights": torch.empty((L, T, k), dtype=torch.float64, device="cuda")}
        if c["sums"]:
            out["score_sum"] = torch.empty((L, E), dtype=torch.float64, device="cuda")
        for l in range(L):
            x = st["logits"][l].double()
            b = None if st["bias"] is None else st["bias"][l].double().expand(T, E)
            ch, _ = _choice64(x, b, c)
            rank = ch if b is not None else x.masked_fill(ch == -math.inf, -math.inf)
            ids = torch.argsort(rank, dim=-1, descending=True, stable=True)[:, :k]
            if c["renorm"] and c["score"] == "softmax":
                w = torch.softmax(x.gather(1, ids), -1)
            else:
                s = torch.special.expit(x) if c["score"] == "sigmoid" else torch.exp(torch.log_softmax(x, -1))
                w = s.gather(1, ids)
                w = w / w.sum(-1, keepdim=True) if c["renorm"] else w
                if c["sums"]:
                    out["score_sum"][l] = s.sum(0)
            if c["sums"] and c["renorm"] and c["score"] == "softmax":
                out["score_sum"][l] = torch.softmax(x, -1).sum(0)
            out["weights"][l] = w * c["scale"]
        return out
    d = torch.empty((L, T, E), dtype=torch.float64, device="cuda")
    for l in range(L):  # the chain rule, by automatic differentiation of the definition
        x = st["logits"][l].double().requires_grad_(True)
        s = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, -1)
        w = s.gather(1, st["ids"][l].long())
        w = w / w.sum(-1, keepdim=True) if c["renorm"] else w
        loss = (w * c["scale"] * st["dw"][l].double()).sum()
        if st["da"] is not None:
            loss = loss + (s.sum(0) * st["da"][l].double()).sum()
        d[l], = torch.autograd.grad(loss, x)
    return d
