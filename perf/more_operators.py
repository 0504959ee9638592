"""What is measured of the expert operators: the experts' matrix products (16-bit, and 8-bit with
scales) and their gradients, the norm before them, the activation between them and the combination
behind them.

A case is a dict of plain values.  ``prepare`` makes its inputs on the GPU, ``run`` makes one
pass: with ``own`` false in elementary torch operations in 32 bits, with ``own`` true through
the library's entry points.  ``exact`` gives the outputs from the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}
E4M3_MAX = 448.0
LEAST = 1e-30  # a block whose largest value is under it is scaled as if it were this
EPS = 1e-6


def _gemm(name, op, T, E, k, N, K, dtype, out, gather, align, skew):
    """A case of the experts' products: "forward" (x W^T), "grad_input" (dy W) or "grad_weight" (dy^T x)."""
    return {"name": name, "op": op, "T": T, "E": E, "k": k, "N": N, "K": K, "dtype": dtype, "out": out, "gather": gather,
            "align": align, "skew": skew}


def listed():
    return [
        # the experts' first product for a decode batch of 64 requests: nearly every expert, a few rows each
        _gemm("gemm_decode", "forward", 64, 128, 8, 1536, 2048, "bf16", "bf16", True, 16, 0.5),
        # the first product of a prefill batch at one layer of the 128-expert model, rows gathered by the experts' lists
        _gemm("gemm_prefill", "forward", 32768, 128, 8, 1536, 2048, "bf16", "bf16", True, 128, 0.5),
        # a training step of a 64-expert model with k = 6: the gradient by the rows, odd token count, no padding
        _gemm("gemm_grad_input", "grad_input", 16001, 64, 6, 2816, 2048, "bf16", "bf16", False, 1, 0.5),
        # the weights' gradient of the same step, summed in fp32 for the optimizer
        _gemm("gemm_grad_weight", "grad_weight", 16001, 64, 6, 2816, 2048, "bf16", "f32", True, 1, 0.5),
        # 8-bit decode: one new token each of 16 requests, 256 experts
        _gemm("fp8_decode", "forward", 16, 256, 8, 2048, 768, "e4m3", "bf16", False, 1, 0.5),
        # 8-bit prefill at one layer
        _gemm("fp8_prefill", "forward", 32768, 128, 8, 1536, 2048, "e4m3", "bf16", True, 128, 0.5),
        # the norm before a layer's router and experts: hidden states for the gate, 8-bit rows for the experts
        {"name": "norm_prefill", "op": "norm", "T": 65536, "H": 2048, "dtype": "bf16", "residual": True, "y": True, "quant": True},
        # its backward pass in a training step, with the gradient that comes along the residual
        {"name": "norm_grad", "op": "norm_grad", "T": 30011, "H": 2048, "dtype": "bf16", "residual": True},
        # between the two products of a prefill batch: gated activation, 8-bit rows for the second product
        {"name": "act_prefill", "op": "act", "rows": 278400, "used": 270208, "I": 768, "dtype": "bf16", "y": False, "quant": True},
        # its gradient in a training step
        {"name": "act_grad", "op": "act_grad", "rows": 96006, "used": 96006, "I": 1408, "dtype": "bf16"},
        # the experts' rows back to their tokens, weighted, on top of the residual
        {"name": "combine_prefill", "op": "combine", "T": 32768, "E": 128, "k": 8, "H": 2048, "dtype": "bf16", "add": True, "align": 128, "skew": 0.5},
        # the gradient by the experts' rows and by the weights
        {"name": "combine_grad", "op": "combine_grad", "T": 16001, "E": 64, "k": 6, "H": 2048, "dtype": "bf16", "add": False, "align": 1, "skew": 0.5},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "forward", "grad_input", "grad_weight", "e4m3", "e4m3", "norm", "norm_grad", "act", "act_grad",
                     "combine", "combine_grad"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f16"])
    if op in ("norm", "norm_grad"):
        T = _log_int(rng, 1, 65536)
        H = 8 * _log_int(rng, 8, min(1024, 65536 * 256 // T))
        c = {"op": op, "T": T, "H": H, "dtype": rng.choice([dtype, dtype, "f32"]), "residual": rng.random() < 0.6}
        if op == "norm":
            c["y"] = rng.random() < 0.7
            c["quant"] = not c["y"] or rng.random() < 0.5
        return c
    if op in ("act", "act_grad"):
        rows = _log_int(rng, 1, 250000)
        c = {"op": op, "rows": rows, "used": rng.randint(rows // 2, rows), "I": 8 * _log_int(rng, 8, min(512, 250000 * 96 // rows)), "dtype": dtype}
        if op == "act":
            c["y"] = rng.random() < 0.5
            c["quant"] = not c["y"] or rng.random() < 0.5
        return c
    E = rng.choice([8, 16, 60, 64, 64, 72, 128, 128, 160, 256])
    k = rng.choice([1, 2, 4, 6, 8, 8])
    align, skew = rng.choice([1, 1, 16, 64, 128]), rng.choice([0.0, 0.5, 0.5, 1.0])
    if op in ("combine", "combine_grad"):
        H = 8 * _log_int(rng, 8, 512)
        T = _log_int(rng, 1, max(1, min(65536, 16_000_000 * 8 // (H * k))))
        return {"op": op, "T": T, "E": E, "k": k, "H": H, "dtype": dtype, "add": op == "combine" and rng.random() < 0.5, "align": align, "skew": skew}
    unit = 16 if op == "e4m3" else 8
    N, K = (rng.choice([512, 768, 1024, 1408, 1536, 2048, 2816, 4096, unit * _log_int(rng, 4, 4096 // unit), unit * _log_int(rng, 4, 4096 // unit)])
            for _ in range(2))
    while E * N * K > 400_000_000 and E > 8:
        E //= 2
    E = max(4, E // 4 * 4)
    k = min(k, E)
    T = _log_int(rng, 1, max(1, min(32768, 100_000_000_000 // (N * K * k))))
    c = _gemm("", "forward" if op == "e4m3" else op, T, E, k, N, K, "e4m3" if op == "e4m3" else dtype,
              rng.choice(["f32", "16"]) if op != "e4m3" else "bf16", op != "grad_input" and rng.random() < 0.6, align, skew)
    c["out"] = dtype if c["out"] == "16" else c["out"]
    del c["name"]
    return c


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(c):
    pairs = c["T"] * c["k"]
    return pairs + min(c["E"], pairs) * (c["align"] - 1)


def _lists(c, gen):
    """The experts' token lists of one layer, as moer_expert_order gives them: offsets [E+1], the
    pair of each row [rows] (-1: padding) and each pair's row [T][k]."""
    T, E, k, a = c["T"], c["E"], c["k"], c["align"]
    pop = torch.randn(E, device="cuda", generator=gen) * c["skew"]
    z = pop - torch.log(-torch.log(torch.rand((T, E), device="cuda", generator=gen).clamp_(1e-7, 1 - 1e-7)))
    ids = z.topk(k, -1).indices.view(-1)
    n = T * k
    key, perm = ids.sort(stable=True)
    cnt = torch.zeros(E, dtype=torch.int64, device="cuda").scatter_add_(0, key, torch.ones_like(key))
    off = torch.nn.functional.pad(((cnt + a - 1) // a * a).cumsum(0), (1, 0))
    row = off[key] + torch.arange(n, device="cuda") - (cnt.cumsum(0) - cnt)[key]
    order = torch.full((_rows(c),), -1, dtype=torch.int32, device="cuda")
    order[row] = perm.to(torch.int32)
    inv = torch.empty(n, dtype=torch.int32, device="cuda")
    inv[perm] = row.to(torch.int32)
    return {"off": off.to(torch.int32), "order": order, "inv": inv.view(T, k), "most": int((off[1:] - off[:-1]).max())}


def _blocks(x, dim):
    """x with dimension `dim` as whole blocks of 128 (padded with zeros), and the padded tensor's blocked view."""
    pad = -x.shape[dim] % 128
    if pad:
        shape = list(x.shape)
        shape[dim] = pad
        x = torch.cat([x, x.new_zeros(shape)], dim)
    return x.unflatten(dim, (-1, 128))


def _quant(y):
    """Rows of fp32 values as e4m3 with a scale for each block of 128 of a row."""
    b = _blocks(y, 1)
    scale = b.abs().amax(-1).clamp_(min=LEAST) / E4M3_MAX
    q = (b / scale[:, :, None]).clamp_(-E4M3_MAX, E4M3_MAX).flatten(1)[:, :y.shape[1]]
    return q.to(torch.float8_e4m3fn).contiguous(), scale


def _normal(shape, gen, dtype, by=1.0):
    return torch.randn(shape, device="cuda", generator=gen).mul_(by).to(dtype)


def prepare(case, seed):
    c, gen = case, _gen(seed)
    op = c["op"]
    st = {"case": c}
    if op in ("norm", "norm_grad"):
        dt = DTYPES[c["dtype"]]
        st["x"] = _normal((c["T"], c["H"]), gen, dt)
        st["res"] = _normal((c["T"], c["H"]), gen, dt, 3.0) if c["residual"] else None
        st["g"] = (1.0 + 0.1 * torch.randn(c["H"], device="cuda", generator=gen)).to(dt)
        if op == "norm_grad":  # of the sum and the reciprocal norms that the forward call kept
            st["sum"] = st["x"] if st["res"] is None else (st["x"].float() + st["res"].float()).to(dt)
            st["rstd"] = torch.rsqrt(st["sum"].float().square().mean(-1) + EPS)
            st["dy"] = _normal((c["T"], c["H"]), gen, dt)
            st["dres"] = _normal((c["T"], c["H"]), gen, dt) if c["residual"] else None
        return st
    if op in ("act", "act_grad"):
        dt = DTYPES[c["dtype"]]
        st["h"] = _normal((c["rows"], 2 * c["I"]), gen, dt)
        st["used"] = torch.tensor([c["used"]], dtype=torch.int32, device="cuda")
        if op == "act_grad":
            st["dy"] = _normal((c["rows"], c["I"]), gen, dt)
        return st
    st.update(_lists(c, gen))
    if op in ("combine", "combine_grad"):
        dt = DTYPES[c["dtype"]]
        st["z"] = _normal((_rows(c), c["H"]), gen, dt)
        w = torch.rand((c["T"], c["k"]), device="cuda", generator=gen) + 0.05
        st["w"] = w / w.sum(-1, keepdim=True)
        st["add"] = _normal((c["T"], c["H"]), gen, dt) if c["add"] else None
        if op == "combine_grad":
            st["dy"] = _normal((c["T"], c["H"]), gen, dt)
        return st
    E, N, K = c["E"], c["N"], c["K"]
    wide = N if op == "grad_input" else K  # the columns of the rows' operand
    x = _normal((c["T"] if c["gather"] else _rows(c), wide), gen, torch.float32)
    if op == "grad_weight":
        st["dy"] = _normal((_rows(c), N), gen, DTYPES[c["dtype"]])
        pad = (st["order"] < 0)[:, None]
        st["dy"].masked_fill_(pad, 0.0)
        st["x"] = x.to(DTYPES[c["dtype"]])
        return st
    w = _normal((E, N, K), gen, torch.float32, 1.0 / math.sqrt(wide))
    if c["dtype"] != "e4m3":
        st["x"], st["w"] = x.to(DTYPES[c["dtype"]]), w.to(DTYPES[c["dtype"]])
        return st
    st["x"], st["sx"] = _quant(x)
    b = _blocks(_blocks(w, 1), 3)  # [E, N/128, 128, K/128, 128]
    st["sw"] = b.abs().amax((2, 4)) / E4M3_MAX
    q = (b / st["sw"][:, :, None, :, None].clamp(min=1e-30)).flatten(3, 4).flatten(1, 2)[:, :N, :K]
    st["w"] = q.to(torch.float8_e4m3fn).contiguous()
    return st


# ---------------------------------------------------------------- the plain forms
def _plain_gemm(st):
    """The ragged products as batched ones over every expert's rows, padded to the longest segment."""
    c, off, order, most = st["case"], st["off"].long(), st["order"].long(), st["most"]
    rows, E = _rows(c), c["E"]
    x, dev = st["x"].float(), st["x"].device
    if c["dtype"] == "e4m3":
        x = (_blocks(x, 1) * st["sx"][:, :, None]).flatten(1)[:, :c["K"]]
    at = off[:-1, None] + torch.arange(most, device=dev)          # [E, most] rows of each expert
    live = (at < off[1:, None]).flatten()
    at = at.clamp(max=rows - 1).flatten()
    src = at
    if c["gather"]:
        live &= order[at] >= 0
        src = order[at].clamp(min=0) // c["k"]
    xe = torch.where(live[:, None], x[src], 0.0).view(E, most, -1)
    if c["op"] == "grad_weight":
        dy = torch.where(live[:, None], st["dy"].float()[at], 0.0).view(E, most, -1)
        return torch.bmm(dy.transpose(1, 2), xe).to(DTYPES[c["out"]])
    w = st["w"].float()
    if c["dtype"] == "e4m3":
        w = (_blocks(_blocks(w, 1), 3) * st["sw"][:, :, None, :, None]).flatten(3, 4).flatten(1, 2)[:, :c["N"], :c["K"]]
    y = torch.bmm(xe, w if c["op"] == "grad_input" else w.transpose(1, 2)).flatten(0, 1)
    p = torch.arange(rows, device=dev)
    e = torch.searchsorted(off[1:], p, right=True).clamp(max=E - 1)
    return torch.where((p < off[-1])[:, None], y[e * most + (p - off[e]).clamp(max=most - 1)], 0.0).to(DTYPES[c["out"]])


def _plain_quant(y):
    b = _blocks(y, 1)
    scale = b.abs().amax(-1).clamp(min=LEAST) / E4M3_MAX
    q = (b / scale[:, :, None]).flatten(1)[:, :y.shape[1]]
    return q.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _plain_norm(st):
    c, x = st["case"], st["x"]
    s = x if st["res"] is None else (x.float() + st["res"].float()).to(x.dtype)
    f = s.float()
    rstd = torch.rsqrt((f * f).mean(-1) + EPS)
    y = f * rstd[:, None] * st["g"].float()
    out = {"rstd": rstd}
    if st["res"] is not None:
        out["res"] = s
    if c["y"]:
        out["y"] = y.to(x.dtype)
    if c["quant"]:
        out["q"], out["scale"] = _plain_quant(y)
    return out


def _plain_norm_grad(st):
    s, dy, rstd = st["sum"].float(), st["dy"].float(), st["rstd"][:, None]
    n = s * rstd
    gd = dy * st["g"].float()
    dx = rstd * (gd - n * (gd * n).mean(-1, keepdim=True))
    if st["dres"] is not None:
        dx = dx + st["dres"].float()
    return {"dx": dx.to(st["x"].dtype), "dg": (dy * n).sum(0)}


def _plain_act(st):
    c, h = st["case"], st["h"].float()
    a, b = h[:, :c["I"]], h[:, c["I"]:]
    y = a / (1.0 + torch.exp(-a)) * b
    live = (torch.arange(c["rows"], device=h.device) < st["used"])[:, None]
    out = {}
    if c["y"]:
        out["y"] = torch.where(live, y, 0.0).to(st["h"].dtype)
    if c["quant"]:
        q, scale = _plain_quant(y)
        out["q"], out["scale"] = torch.where(live, q.float(), 0.0).to(q.dtype), torch.where(live, scale, 0.0)
    return out


def _plain_act_grad(st):
    c, h, dy = st["case"], st["h"].float(), st["dy"].float()
    a, b = h[:, :c["I"]], h[:, c["I"]:]
    s = 1.0 / (1.0 + torch.exp(-a))
    d = torch.cat([dy * b * s * (1.0 + a * (1.0 - s)), dy * a * s], 1)
    return torch.where((torch.arange(c["rows"], device=h.device) < st["used"])[:, None], d, 0.0).to(st["h"].dtype)


def _plain_combine(st):
    z = st["z"].float()[st["inv"].long()]  # [T, k, H]
    y = (z * st["w"][:, :, None]).sum(1)
    if st["add"] is not None:
        y = y + st["add"].float()
    return y.to(st["z"].dtype)


def _plain_combine_grad(st):
    c, dy, order = st["case"], st["dy"].float(), st["order"].long()
    z = st["z"].float()[st["inv"].long()]
    dw = (z * dy[:, None, :]).sum(-1)
    pair = order.clamp(min=0)
    dz = dy[pair // c["k"]] * st["w"].flatten()[pair][:, None]
    return {"dz": torch.where((order >= 0)[:, None], dz, 0.0).to(st["z"].dtype), "dw": dw}


_PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "act": _plain_act, "act_grad": _plain_act_grad,
          "combine": _plain_combine, "combine_grad": _plain_combine_grad}


# ---------------------------------------------------------------- the library's calls
def _open(st):
    """What a program keeps between calls: arguments, outputs and a workspace."""
    from moe_expert_routing_top_gb300 import _native as nat
    c, op, dev = st["case"], st["case"]["op"], "cuda"

    def new(*shape, dtype=torch.float32):
        return torch.zeros(shape, dtype=dtype, device=dev)

    def quant(rows, cols):
        return {"q": new(rows, cols, dtype=torch.float8_e4m3fn), "scale": new(rows, (cols + 127) // 128)}
    if op in ("norm", "norm_grad"):
        T, H, dt = c["T"], c["H"], DTYPES[c["dtype"]]
        if op == "norm":
            o = {"rstd": new(T)}
            if c["residual"]:
                o["res"] = new(T, H, dtype=dt)
            if c["y"]:
                o["y"] = new(T, H, dtype=dt)
            if c["quant"]:
                o.update(quant(T, H))
            a = nat.make_norm(T=T, H=H, dtype=c["dtype"], eps=EPS, x=st["x"], residual=st["res"], weight=st["g"], sum=o.get("res"),
                              y=o.get("y"), q=o.get("q"), scale=o.get("scale"), rstd=o["rstd"])
            return nat.moer_rms_norm, a, o, new(nat.moer_rms_norm_workspace_bytes(T, H), dtype=torch.uint8)
        o = {"dx": new(T, H, dtype=dt), "dg": new(H)}
        a = nat.make_norm(T=T, H=H, dtype=c["dtype"], eps=EPS, sum=st["sum"], weight=st["g"], rstd=st["rstd"], d_y=st["dy"],
                          d_sum=st["dres"], d_x=o["dx"], d_weight=o["dg"])
        return nat.moer_rms_norm_grad, a, o, new(nat.moer_rms_norm_workspace_bytes(T, H), dtype=torch.uint8)
    if op in ("act", "act_grad"):
        rows, I, dt = c["rows"], c["I"], DTYPES[c["dtype"]]
        if op == "act":
            o = {"y": new(rows, I, dtype=dt)} if c["y"] else {}
            if c["quant"]:
                o.update(quant(rows, I))
            a = nat.make_expert_act(rows=rows, I=I, dtype=c["dtype"], h=st["h"], used=st["used"], y=o.get("y"), q=o.get("q"), scale=o.get("scale"))
            return nat.moer_expert_act, a, o, None
        o = new(rows, 2 * I, dtype=dt)
        a = nat.make_expert_act(rows=rows, I=I, dtype=c["dtype"], h=st["h"], used=st["used"], d_y=st["dy"], d_h=o)
        return nat.moer_expert_act_grad, a, o, None
    rows = _rows(c)
    if op in ("combine", "combine_grad"):
        dt = DTYPES[c["dtype"]]
        if op == "combine":
            o = new(c["T"], c["H"], dtype=dt)
            a = nat.make_expert_combine(T=c["T"], H=c["H"], k=c["k"], rows=rows, dtype=c["dtype"], z=st["z"], inv=st["inv"],
                                        weights=st["w"], add=st["add"], out=o)
            return nat.moer_expert_combine, a, o, new(256, dtype=torch.uint8)
        o = {"dz": new(rows, c["H"], dtype=dt), "dw": new(c["T"], c["k"])}
        a = nat.make_expert_combine(T=c["T"], H=c["H"], k=c["k"], rows=rows, dtype=c["dtype"], z=st["z"], inv=st["inv"],
                                    order=st["order"], weights=st["w"], d_out=st["dy"], d_z=o["dz"], d_weights=o["dw"])
        return nat.moer_expert_combine_grad, a, o, new(256, dtype=torch.uint8)
    E, N, K = c["E"], c["N"], c["K"]
    shape = {"forward": (rows, N), "grad_input": (rows, K), "grad_weight": (E, N, K)}[op]
    o = new(*shape, dtype=DTYPES[c["out"]])
    a = nat.make_expert_gemm(op=op, E=E, N=N, K=K, rows=rows, tokens=st["x"].shape[0], k=c["k"], dtype=c["dtype"], out_dtype=c["out"],
                             expert_off=st["off"], order=st["order"] if c["gather"] else None, x=st["x"], x_scale=st.get("sx"),
                             w=st.get("w"), w_scale=st.get("sw"), d_y=st.get("dy"), out=o)
    return nat.moer_expert_gemm, a, o, new(nat.moer_expert_gemm_workspace_bytes(a), dtype=torch.uint8)


def _own(st):
    h = st.get("handle")
    if h is None:
        h = st["handle"] = _open(st)
    call, a, o, ws = h
    if ws is None:
        call(a)
    else:
        call(a, ws, ws.numel())
    return o


def run(state):
    if own:
        return _own(state)
    return _PLAIN.get(state["case"]["op"], _plain_gemm)(state)


def work(case):
    c, op = case, case["op"]
    b = BYTES[c["dtype"]]
    if op in ("norm", "norm_grad"):
        n = c["T"] * c["H"]
        if op == "norm":
            per = b * (1 + 2 * c["residual"] + c["y"]) + (c["quant"] and 1 + 4 / 128)
            return {"bytes": n * per + 4 * c["T"] + b * c["H"], "flops": 6 * n}
        return {"bytes": n * b * (3 + c["residual"]) + 4 * c["T"] + (4 + b) * c["H"], "flops": 10 * n}
    if op in ("act", "act_grad"):
        n = c["used"] * c["I"]
        if op == "act":
            return {"bytes": n * (b * (2 + c["y"]) + (c["quant"] and 1 + 4 / 128)), "flops": 8 * n}
        return {"bytes": n * b * 5, "flops": 14 * n}
    pairs = c["T"] * c["k"]
    if op in ("combine", "combine_grad"):
        if op == "combine":
            return {"bytes": b * c["H"] * (pairs + c["T"] * (1 + c["add"])) + 8 * pairs, "flops": 2 * pairs * c["H"]}
        return {"bytes": b * c["H"] * (2 * pairs + c["T"]) + 16 * pairs, "flops": 3 * pairs * c["H"]}
    E, N, K = c["E"], c["N"], c["K"]
    active = E * (1.0 - (1.0 - c["k"] / E) ** c["T"])  # experts that some token chose
    ob = BYTES[c["out"]]
    xrows = c["T"] if c["gather"] else pairs
    flops = 2.0 * pairs * N * K
    if op == "grad_weight":
        return {"bytes": b * (xrows * K + pairs * N) + ob * E * N * K, "flops": flops}
    inner, outer = (N, K) if op == "grad_input" else (K, N)
    scales = 4.0 * (xrows * K / 128 + active * N * K / 16384) if c["dtype"] == "e4m3" else 0
    return {"bytes": b * (active * N * K + xrows * inner) + ob * pairs * outer + scales, "flops": flops}


# ---------------------------------------------------------------- from the definition, in 64 bits
def _exact_gemm(st):
    c, off, order = st["case"], st["off"].tolist(), st["order"].long()
    rows, E, k = _rows(c), c["E"], c["k"]
    shape = {"forward": (rows, c["N"]), "grad_input": (rows, c["K"]), "grad_weight": (E, c["N"], c["K"])}[c["op"]]
    out = torch.zeros(shape, dtype=torch.float64, device="cuda")
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if hi == lo:
            continue
        at = torch.arange(lo, hi, device="cuda")
        if c["gather"]:
            at = at[order[lo:hi] >= 0]
        src = order[at] // k if c["gather"] else at
        x = st["x"][src].double()
        if c["op"] == "grad_weight":
            out[e] = st["dy"][at].double().T @ x
            continue
        w = st["w"][e].double()
        if c["dtype"] == "e4m3":
            x = x * st["sx"][src].double().repeat_interleave(128, 1)[:, :c["K"]]
            w = w * st["sw"][e].double().repeat_interleave(128, 0)[:c["N"]].repeat_interleave(128, 1)[:, :c["K"]]
        out[at] = x @ (w if c["op"] == "grad_input" else w.T)
    return out


def _exact_quant(y):
    scale = torch.stack([p.abs().amax(1) for p in y.split(128, 1)], 1).clamp(min=LEAST) / E4M3_MAX
    return y / scale.repeat_interleave(128, 1)[:, :y.shape[1]], scale


def exact(case, seed):
    c = case
    st = prepare(c, seed)
    op = c["op"]
    if op == "norm":
        s = st["x"] if st["res"] is None else (st["x"].double() + st["res"].double()).to(st["x"].dtype)
        f = s.double()
        rstd = (f.pow(2).sum(-1) / c["H"] + EPS).pow(-0.5)
        y = f * rstd[:, None] * st["g"].double()
        out = {"rstd": rstd}
        if st["res"] is not None:
            out["res"] = f
        if c["y"]:
            out["y"] = y
        if c["quant"]:
            out["q"], out["scale"] = _exact_quant(y)
        return out
    if op == "norm_grad":  # the chain rule, by automatic differentiation of the definition
        s, g = st["sum"].double().requires_grad_(True), st["g"].double().requires_grad_(True)
        y = s / torch.sqrt(s.pow(2).mean(-1, keepdim=True) + EPS) * g
        dx, dg = torch.autograd.grad((y * st["dy"].double()).sum(), (s, g))
        return {"dx": dx if st["dres"] is None else dx + st["dres"].double(), "dg": dg}
    if op in ("act", "act_grad"):
        n = c["used"]
        h = st["h"][:n].double().requires_grad_(op == "act_grad")
        y = torch.special.expit(h[:, :c["I"]]) * h[:, :c["I"]] * h[:, c["I"]:]

        def whole(v):
            return torch.cat([v, v.new_zeros((c["rows"] - n, v.shape[1]))])
        if op == "act_grad":
            return whole(torch.autograd.grad((y * st["dy"][:n].double()).sum(), h)[0])
        out = {"y": whole(y)} if c["y"] else {}
        if c["quant"]:
            q, scale = _exact_quant(y)
            out["q"], out["scale"] = whole(q), whole(scale)
        return out
    if op in ("combine", "combine_grad"):
        w = st["w"].double()
        if op == "combine":
            y = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device="cuda") if st["add"] is None else st["add"].double()
            for j in range(c["k"]):
                y = y + w[:, j:j + 1] * st["z"][st["inv"][:, j].long()].double()
            return y
        dz = torch.zeros((_rows(c), c["H"]), dtype=torch.float64, device="cuda")
        dw = torch.empty_like(w)
        for j in range(c["k"]):
            at = st["inv"][:, j].long()
            dz[at] = w[:, j:j + 1] * st["dy"].double()
            dw[:, j] = (st["z"][at].double() * st["dy"].double()).sum(-1)
        return {"dz": dz, "dw": dw}
    return _exact_gemm(st)
