"""The expert operators on the GPU against their 64-bit statements (oracle/experts.py).

Tolerances.  Inputs are given in their own type, so their values are exact on both sides.
  - A sum of n terms in fp32, in any order, each addition off by at most 2^-23 of its result (a
    rounding is half that; matrix units may cut instead): n * 2^-23 * (sum of the terms'
    magnitudes).  Products of two 16-bit or 8-bit values are exact in fp32; where factors in fp32
    multiply a term, 2^-24 of it for each.
  - Rounding to a type: finfo(type).eps / 2 of the value, and half of the smallest subnormal.
  - e4m3: 2^-4 of the scaled value, 2^-10 under 2^-6; the scaled value itself is off by what the
    fp32 steps before it are.
"""
import numpy as np
import pytest

from oracle import experts as ex

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_routing_top_gb300 import _native as nat
    return torch, nat


def _types(torch):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _half_step(torch, dtype, v):
    """Largest error of rounding values near v to the type."""
    f = torch.finfo(_types(torch)[dtype])
    return f.eps / 2 * np.abs(v) * (1 + f.eps) + f.smallest_normal * f.eps / 2


def _np(t):
    return t.double().cpu().numpy()


def _rand(torch, shape, dtype, seed, by=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * by).to(_types(torch)[dtype]).cuda()


def _wide(torch, x, pad):
    """x with `pad` unused columns behind each row."""
    y = torch.full((*x.shape[:-1], x.shape[-1] + pad), float("nan"), dtype=torch.float32).to(x.dtype).cuda()
    y[..., :x.shape[-1]] = x
    return y[..., :x.shape[-1]]


def _ws(torch, n=256):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def _close(got, ref, tol, what=""):
    got = _np(got) if hasattr(got, "cpu") else got
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: {got[bad][0]} for {ref[bad][0]}"


def _check_quant(torch, q, scale, y, rel):
    """8-bit rows of y (known to a relative error `rel` of the block's values)."""
    s = _np(scale)
    ref = ex.block_scales(y)
    assert (np.abs(s - ref) <= (rel + 4 * U) * ref).all()
    v = y / ex.widen(s, y.shape[1])
    got = _np(q.float())
    assert (np.abs(got - v) <= np.maximum(np.abs(v) * 2.0 ** -4, 2.0 ** -10) * (1 + 1e-3) + (rel + 4 * U) * np.abs(v)).all()


# ------------------------------------------------------------------ norm
NORMS = [(1, 2048), (3, 64), (7, 8), (5, 1), (2, 129), (33, 1000), (9, 2049), (4, 4096), (3, 7168), (2, 16384), (3, 16383), (700, 256), (1, 520)]


@pytest.mark.parametrize("T,H", NORMS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("residual,pad", [(False, 0), (True, 0), (True, 3), (True, 8)])
def test_norm(env, T, H, dtype, residual, pad):
    torch, nat = env
    dt = _types(torch)[dtype]
    x = _wide(torch, _rand(torch, (T, H), dtype, 1), pad)
    r = _wide(torch, _rand(torch, (T, H), dtype, 2, 3.0), pad) if residual else None
    w = _rand(torch, (H,), dtype, 3)
    s = torch.empty((T, H + pad), dtype=dt, device="cuda")[:, :H]
    y = torch.empty((T, H + pad), dtype=dt, device="cuda")[:, :H]
    q = torch.zeros((T, H + pad), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)[:, :H]
    scale = torch.full((T, ex.blocks(H) + 1), -1.0, device="cuda")[:, :-1]
    rstd = torch.empty(T, device="cuda")
    a = nat.make_norm(T=T, H=H, dtype=dtype, eps=1e-6, x=x, residual=r, weight=w, sum=s, y=y, q=q, scale=scale, rstd=rstd)
    nat.moer_rms_norm(a)
    want = x if r is None else (x.float() + r.float()).to(dt)
    assert torch.equal(s, want)                      # an fp32 sum of two 16-bit values, rounded once
    yy, rr = ex.rms_norm(_np(want), _np(w), 1e-6)
    rel = (H + 16) * 2 * U / 2 + 4 * U               # half of the sum's relative error, root, reciprocal, division
    assert (np.abs(_np(rstd) - rr) <= rel * rr).all()
    _close(y, yy, (rel + 2 * U) * np.abs(yy) + _half_step(torch, dtype, yy), "y")
    _check_quant(torch, q, scale, yy, rel + 2 * U)


def test_norm_alone_outputs_and_in_place(env):
    torch, nat = env
    T, H = 37, 2048
    x, r, w = _rand(torch, (T, H), "bf16", 1), _rand(torch, (T, H), "bf16", 2), _rand(torch, (H,), "bf16", 3)
    want_s = (x.float() + r.float()).bfloat16()
    y = torch.empty_like(x)
    nat.moer_rms_norm(nat.make_norm(T=T, H=H, dtype="bf16", eps=1e-5, x=x, residual=r, weight=w, y=y))
    x2, r2 = x.clone(), r.clone()
    nat.moer_rms_norm(nat.make_norm(T=T, H=H, dtype="bf16", eps=1e-5, x=x2, residual=r2, weight=w, sum=r2, y=x2))
    assert torch.equal(r2, want_s) and torch.equal(x2, y)
    rstd = torch.empty(T, device="cuda")
    nat.moer_rms_norm(nat.make_norm(T=T, H=H, dtype="bf16", eps=1e-5, x=x, residual=r, weight=w, rstd=rstd))
    assert np.allclose(_np(rstd), ex.rms_norm(_np(want_s), _np(w), 1e-5)[1], rtol=1e-5)


def test_norm_extremes(env):
    """Rows of zeros, of NaN, of an infinity, of the type's lowest value, and blocks of zeros."""
    torch, nat = env
    H = 256
    x = torch.zeros(6, H)
    x[1, 5] = float("nan")
    x[2, 7], x[2, 200] = float("inf"), 1.0
    x[3] = -1e4
    x[4, :128] = 1.0
    x[5] = 1e-20
    x, w = x.bfloat16().cuda(), torch.ones(H).bfloat16().cuda()
    y, q = torch.empty_like(x), torch.zeros((6, H), dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty((6, 2), device="cuda")
    nat.moer_rms_norm(nat.make_norm(T=6, H=H, dtype="bf16", eps=1e-6, x=x, weight=w, y=y, q=q, scale=sc))
    yf, qf, sf = _np(y), _np(q.float()), _np(sc)
    assert (yf[0] == 0).all() and (qf[0] == 0).all() and np.isfinite(sf[0]).all()
    assert np.isnan(yf[1]).all() and np.isnan(qf[1]).all()
    assert np.isnan(yf[2, 7]) and yf[2, 200] == 0        # inf * (1 / inf)
    assert (yf[3] == -1).all() and (np.abs(qf[3] * ex.widen(sf, H)[3] + 1) < 1e-2).all()
    assert (qf[4, 128:] == 0).all() and np.isfinite(sf[4]).all()
    assert np.allclose(yf[5], 1e-20 / np.sqrt(1e-6), rtol=0.01)


@pytest.mark.parametrize("T,H", NORMS + [(5000, 72)])
@pytest.mark.parametrize("dtype,dsum,pad", [("bf16", True, 0), ("bf16", False, 3), ("f16", True, 8), ("f32", True, 0)])
def test_norm_grad(env, T, H, dtype, dsum, pad):
    torch, nat = env
    dt = _types(torch)[dtype]
    s, w = _wide(torch, _rand(torch, (T, H), dtype, 1, 2.0), pad), _rand(torch, (H,), dtype, 2)
    dy = _wide(torch, _rand(torch, (T, H), dtype, 3), pad)
    ds = _wide(torch, _rand(torch, (T, H), dtype, 4), pad) if dsum else None
    rstd = torch.from_numpy(ex.rms_norm(_np(s), _np(w), 1e-6)[1]).float().cuda()
    dx, dw = torch.empty((T, H + pad), dtype=dt, device="cuda")[:, :H], torch.empty(H, device="cuda")
    n = nat.moer_rms_norm_workspace_bytes(T, H)
    a = nat.make_norm(T=T, H=H, dtype=dtype, eps=1e-6, sum=s, weight=w, rstd=rstd, d_y=dy, d_sum=ds, d_x=dx, d_weight=dw)
    nat.moer_rms_norm_grad(a, _ws(torch, n), n)
    rx, mx, rw, mw = ex.rms_norm_grad(_np(s), _np(w), _np(rstd), _np(dy), None if ds is None else _np(ds))
    _close(dx, rx, (H + 24) * 2 * U * mx + _half_step(torch, dtype, rx), "d_x")
    _close(dw, rw, (T + 16) * 2 * U * mw + 1e-44, "d_weight")
    # in place of either gradient, and without the weight's
    for name in ("d_y", "d_sum"):
        if name == "d_sum" and not dsum:
            continue
        put = {"d_y": dy.clone(), "d_sum": None if ds is None else ds.clone()}
        nat.moer_rms_norm_grad(nat.make_norm(T=T, H=H, dtype=dtype, eps=1e-6, sum=s, weight=w, rstd=rstd, **put, d_x=put[name]), _ws(torch, n), n)
        assert torch.equal(put[name], dx)


def test_norm_grad_without_rows(env):
    torch, nat = env
    dw = torch.full((72,), 7.0, device="cuda")
    n = nat.moer_rms_norm_workspace_bytes(0, 72)
    nat.moer_rms_norm_grad(nat.make_norm(T=0, H=72, dtype="bf16", eps=0.0, d_weight=dw), _ws(torch, n), n)
    assert (dw == 0).all()


# ------------------------------------------------------------------ activation
ACTS = [(1, 768), (5, 8), (3, 1), (7, 130), (257, 128), (40, 1408), (1000, 72), (9, 136), (2, 4099)]


@pytest.mark.parametrize("rows,I", ACTS)
@pytest.mark.parametrize("dtype,pad", [("bf16", 0), ("f16", 8), ("f32", 0), ("bf16", 3)])
def test_act(env, rows, I, dtype, pad):
    torch, nat = env
    dt = _types(torch)[dtype]
    h = _wide(torch, _rand(torch, (rows, 2 * I), dtype, 1, 3.0), pad)
    y = torch.full((rows, I + pad), 5.0, dtype=dt, device="cuda")[:, :I]
    q = torch.full((rows, I + pad), 0x55, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)[:, :I]
    sc = torch.full((rows, ex.blocks(I)), 5.0, device="cuda")
    n = rows - rows // 3
    used = torch.tensor([n], dtype=torch.int32, device="cuda")
    nat.moer_expert_act(nat.make_expert_act(rows=rows, I=I, dtype=dtype, h=h, used=used, y=y, q=q, scale=sc))
    hv = _np(h)[:n]
    ref = ex.silu_gate(hv)
    # exp: 2 + 1.2 |a| steps, addition, division, two products
    rel = (24 + 2.4 * np.abs(hv[:, :I])) * U
    _close(y[:n], ref, rel * np.abs(ref) + _half_step(torch, dtype, ref) + 2.0 ** -120, "y")
    assert (y[n:] == 5).all() and (sc[n:] == 5).all() and (q.view(torch.uint8)[n:] == 0x55).all()
    _check_quant(torch, q[:n], sc[:n], ref, rel.max())


@pytest.mark.parametrize("rows,I", ACTS)
@pytest.mark.parametrize("dtype,pad", [("bf16", 0), ("f16", 8), ("f32", 0), ("bf16", 3)])
def test_act_grad(env, rows, I, dtype, pad):
    torch, nat = env
    dt = _types(torch)[dtype]
    h, dy = _wide(torch, _rand(torch, (rows, 2 * I), dtype, 1, 3.0), pad), _wide(torch, _rand(torch, (rows, I), dtype, 2), pad)
    dh = torch.full((rows, 2 * I + pad), 5.0, dtype=dt, device="cuda")[:, :2 * I]
    n = rows - rows // 3
    used = torch.tensor([n], dtype=torch.int32, device="cuda")
    nat.moer_expert_act_grad(nat.make_expert_act(rows=rows, I=I, dtype=dtype, h=h, used=used, d_y=dy, d_h=dh))
    hv, dv = _np(h)[:n], _np(dy)[:n]
    ref = ex.silu_gate_grad(hv, dv)
    a, b = hv[:, :I], hv[:, I:]
    s, big = ex.sigmoid(a), (32 + 4.8 * np.abs(a)) * U
    # s and 1 - s are off by `big` of 1 at most, and of themselves
    mag = np.concatenate([np.abs(dv * b) * s * (1 + 2 * np.abs(a)), np.abs(dv * a) * s], 1)
    _close(dh[:n], ref, np.concatenate([big, big], 1) * mag + _half_step(torch, dtype, ref) + 2.0 ** -120, "d_h")
    assert (dh[n:] == 5).all()
    inplace = h.clone()
    nat.moer_expert_act_grad(nat.make_expert_act(rows=rows, I=I, dtype=dtype, h=inplace, used=used, d_y=dy, d_h=inplace))
    assert torch.equal(inplace[:n], dh[:n]) and torch.equal(inplace[n:], h[n:])


@pytest.mark.parametrize("used", [-3, 0, 1, 12, 13, 99])
def test_act_used_rows(env, used):
    torch, nat = env
    h = _rand(torch, (12, 64), "bf16", 1)
    y = torch.full((12, 32), 5.0, dtype=torch.bfloat16, device="cuda")
    u = torch.tensor([used], dtype=torch.int32, device="cuda")
    nat.moer_expert_act(nat.make_expert_act(rows=12, I=32, dtype="bf16", h=h, used=u, y=y))
    n = min(max(used, 0), 12)
    assert (y[n:] == 5).all()
    assert np.allclose(_np(y[:n]), ex.silu_gate(_np(h[:n])), rtol=2.0 ** -7)


def test_act_large_arguments(env):
    torch, nat = env
    a = torch.tensor([-1e4, -200.0, -88.0, -30.0, 0.0, 30.0, 200.0, 3e4])
    h = torch.cat([a, torch.full((8,), 2.0)]).view(1, 16).float().cuda()
    y, dh = torch.empty((1, 8), device="cuda"), torch.empty((1, 16), device="cuda")
    nat.moer_expert_act(nat.make_expert_act(rows=1, I=8, dtype="f32", h=h, y=y))
    nat.moer_expert_act_grad(nat.make_expert_act(rows=1, I=8, dtype="f32", h=h, d_y=torch.ones((1, 8), device="cuda"), d_h=dh))
    assert np.allclose(_np(y), ex.silu_gate(_np(h)), rtol=3e-5, atol=1e-35)
    assert np.allclose(_np(dh), ex.silu_gate_grad(_np(h), np.ones((1, 8))), rtol=3e-5, atol=1e-35)


# ------------------------------------------------------------------ combination
def _lists(rs, counts, T, k, align):
    """Experts' lists with the given numbers of rows: any T * k = sum(counts) pairs, shuffled."""
    pairs = rs.permutation(T * k)
    off, order, at = [0], [], 0
    inv = np.full(T * k, -1)
    for c in counts:
        mine = np.sort(pairs[at:at + c])
        at += c
        inv[mine] = len(order) + np.arange(c)
        order += mine.tolist() + [-1] * (-c % align)
        off.append(len(order))
    return np.array(off, np.int32), np.array(order, np.int32), inv.reshape(T, k).astype(np.int32)


COMBS = [(1, 8, 2048, 1), (5, 2, 8, 4), (33, 6, 264, 16), (17, 9, 1, 1), (8, 32, 72, 1), (3, 1, 4100, 2), (40, 8, 513, 1), (300, 4, 96, 128)]


def _comb_case(T, k, align, extra=5):
    rs = np.random.RandomState(T + k)
    counts = np.bincount(rs.randint(0, 7, T * k), minlength=7)
    off, order, inv = _lists(rs, counts, T, k, align)
    order = np.concatenate([order, np.full(extra, -1, np.int32)])
    return off, order, inv


@pytest.mark.parametrize("T,k,H,align", COMBS)
@pytest.mark.parametrize("dtype,pad,add,weighted", [("bf16", 0, True, True), ("f16", 8, False, True), ("f32", 0, True, False), ("bf16", 3, True, True)])
def test_combine(env, T, k, H, align, dtype, pad, add, weighted):
    torch, nat = env
    dt = _types(torch)[dtype]
    _, order, inv = _comb_case(T, k, align)
    rows = len(order)
    inv.reshape(-1)[::7] = -1
    z = _wide(torch, _rand(torch, (rows, H), dtype, 1), pad)
    z[torch.from_numpy(order < 0).cuda()] = float("nan")       # padding is never read
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(2)).cuda() if weighted else None
    base = _wide(torch, _rand(torch, (T, H), dtype, 3), pad) if add else None
    out = torch.empty((T, H + pad), dtype=dt, device="cuda")[:, :H]
    ws, iv = _ws(torch), torch.from_numpy(inv).cuda()
    nat.moer_expert_combine(nat.make_expert_combine(T=T, H=H, k=k, rows=rows, dtype=dtype, z=z, inv=iv, weights=w, add=base, out=out), ws, 256)
    assert nat.moer_ws_status(ws) == 0
    ref, mag = ex.combine(_np(z), inv, None if w is None else _np(w), None if base is None else _np(base))
    _close(out, ref, (k + 2) * 2 * U * mag + _half_step(torch, dtype, ref))
    if add:
        nat.moer_expert_combine(nat.make_expert_combine(T=T, H=H, k=k, rows=rows, dtype=dtype, z=z, inv=iv, weights=w, add=base, out=base), ws, 256)
        assert torch.equal(base, out)


@pytest.mark.parametrize("T,k,H,align", COMBS)
@pytest.mark.parametrize("dtype,pad,weighted", [("bf16", 0, True), ("f16", 8, True), ("f32", 0, False), ("bf16", 3, True)])
def test_combine_grad(env, T, k, H, align, dtype, pad, weighted):
    torch, nat = env
    dt = _types(torch)[dtype]
    _, order, inv = _comb_case(T, k, align)
    rows = len(order)
    z = _wide(torch, _rand(torch, (rows, H), dtype, 1), pad)
    z[torch.from_numpy(order < 0).cuda()] = float("nan")
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(2)).cuda() if weighted else None
    do = _wide(torch, _rand(torch, (T, H), dtype, 3), pad)
    dz, dw = torch.full((rows, H + pad), 5.0, dtype=dt, device="cuda")[:, :H], torch.empty((T, k), device="cuda")
    ws, iv, od = _ws(torch), torch.from_numpy(inv).cuda(), torch.from_numpy(order).cuda()
    base = dict(T=T, H=H, k=k, rows=rows, dtype=dtype, inv=iv, order=od, weights=w, d_out=do)
    nat.moer_expert_combine_grad(nat.make_expert_combine(z=z, d_z=dz, d_weights=dw, **base), ws, 256)
    assert nat.moer_ws_status(ws) == 0
    rz, rw, mw = ex.combine_grad(_np(z), inv, None if w is None else _np(w), _np(do), rows)
    _close(dz, rz, U * np.abs(rz) + _half_step(torch, dtype, rz), "d_z")
    _close(dw, rw, (H + 2) * 2 * U * mw, "d_weights")
    dz2, dw2 = torch.full_like(dz, 5.0), torch.empty_like(dw)
    nat.moer_expert_combine_grad(nat.make_expert_combine(d_z=dz2, **base), ws, 256)
    nat.moer_expert_combine_grad(nat.make_expert_combine(z=z, d_weights=dw2, **base), ws, 256)
    assert torch.equal(dz2, dz) and torch.equal(dw2, dw) and nat.moer_ws_status(ws) == 0


def test_combine_bad_rows(env):
    """Rows past the buffer count as none; in the gradient a row goes to the pair that owns it."""
    torch, nat = env
    T, k, H, rows = 4, 2, 16, 8
    z, do = _rand(torch, (rows, H), "f32", 1), _rand(torch, (T, H), "f32", 2)
    inv = np.arange(8, dtype=np.int32).reshape(T, k)
    inv[1, 0], inv[3, 1] = 8, 2 ** 31 - 1
    ws, out = _ws(torch), torch.empty((T, H), device="cuda")
    nat.moer_expert_combine(nat.make_expert_combine(T=T, H=H, k=k, rows=rows, dtype="f32", z=z, inv=torch.from_numpy(inv).cuda(), out=out), ws, 256)
    assert nat.moer_ws_status(ws) == 6
    ok = np.where(inv >= rows, -1, inv)
    assert np.allclose(_np(out), ex.combine(_np(z), ok)[0], atol=1e-5)
    dup = np.arange(8, dtype=np.int32).reshape(T, k)
    dup[2, 1] = 0                                   # row 0 belongs to pair 0
    dz = torch.full((rows, H), 5.0, device="cuda")
    order = torch.arange(8, dtype=torch.int32, device="cuda")
    nat.moer_expert_combine_grad(nat.make_expert_combine(T=T, H=H, k=k, rows=rows, dtype="f32", inv=torch.from_numpy(dup).cuda(), order=order, d_out=do, d_z=dz), ws, 256)
    assert nat.moer_ws_status(ws) == 6
    assert torch.equal(dz[0], do[0]) and (dz[5] == 5).all() and torch.equal(dz[7], do[3])


# ------------------------------------------------------------------ products
#: rows of each expert, and the padding of segments
COUNTS = [([1], 1), ([0, 0, 5, 0], 1), ([3, 17, 0, 40], 16), ([257, 1, 64], 1), ([130, 300, 7], 128), ([0], 1), ([513], 1), ([64, 63, 65, 128], 8),
          ([2] * 33, 1)]


def _gemm_case(torch, counts, align, k, N, K, xcols, dtype, gather, seed=0, tail=6):
    n = sum(counts)
    T = -(-n // k)
    rs = np.random.RandomState(seed + n + N)
    counts = list(counts)
    counts[-1] += T * k - n                          # pairs have to fill the tokens
    off, order, inv = _lists(rs, counts, max(T, 0), k, align)
    order = np.concatenate([order, np.full(tail, -1, np.int32)])
    rows = len(order)
    x = _rand(torch, (T if gather else rows, xcols), dtype, seed + 1)
    return off, order, inv, rows, x


SHAPES = [(256, 256), (64, 64), (8, 8), (136, 72), (1, 8), (520, 264), (300, 1000)]


@pytest.mark.parametrize("counts,align", COUNTS)
@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("dtype,out,gather", [("bf16", "bf16", True), ("f16", "f32", False), ("bf16", "f32", False), ("f16", "f16", True)])
def test_gemm_forward(env, counts, align, N, K, dtype, out, gather):
    torch, nat = env
    k = 2
    off, order, _, rows, x = _gemm_case(torch, counts, align, k, N, K, K, dtype, gather)
    E = len(counts)
    w = _rand(torch, (E, N, K), dtype, 5)
    y = torch.full((rows, N), 7.0, dtype=_types(torch)[out], device="cuda")
    a = nat.make_expert_gemm(op="forward", E=E, N=N, K=K, k=k, dtype=dtype, out_dtype=out, rows=rows, tokens=len(x), x=x, w=w, out=y,
                             expert_off=torch.from_numpy(off).cuda(), order=torch.from_numpy(order).cuda() if gather else None)
    ws = _ws(torch, nat.moer_expert_gemm_workspace_bytes(a))
    nat.moer_expert_gemm(a, ws, ws.numel())
    assert nat.moer_ws_status(ws) == 0
    ref, mag = ex.gemm_rows(_np(x), _np(w), off, order if gather else None, k, out=np.full((rows, N), 7.0))
    _close(y, ref, K * 2 * U * mag + _half_step(torch, out, ref))


@pytest.mark.parametrize("counts,align", COUNTS)
@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("dtype,out,gather", [("bf16", "bf16", False), ("f16", "f32", True)])
def test_gemm_grad_input(env, counts, align, N, K, dtype, out, gather):
    torch, nat = env
    k, ldn = 2, -(-N // 8) * 8
    off, order, _, rows, dy = _gemm_case(torch, counts, align, k, N, K, ldn, dtype, gather)
    E = len(counts)
    w = _rand(torch, (E, N, K), dtype, 5)
    y = torch.full((rows, K), 7.0, dtype=_types(torch)[out], device="cuda")
    a = nat.make_expert_gemm(op="grad_input", E=E, N=N, K=K, k=k, dtype=dtype, out_dtype=out, rows=rows, tokens=len(dy), x=dy[:, :N], ld_x=ldn, w=w,
                             out=y, expert_off=torch.from_numpy(off).cuda(), order=torch.from_numpy(order).cuda() if gather else None)
    ws = _ws(torch, nat.moer_expert_gemm_workspace_bytes(a))
    nat.moer_expert_gemm(a, ws, ws.numel())
    assert nat.moer_ws_status(ws) == 0
    ref, mag = ex.gemm_rows(_np(dy)[:, :N], _np(w).transpose(0, 2, 1), off, order if gather else None, k, out=np.full((rows, K), 7.0))
    _close(y, ref, N * 2 * U * mag + _half_step(torch, out, ref))


@pytest.mark.parametrize("counts,align", COUNTS)
@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("dtype,out,gather", [("bf16", "f32", True), ("f16", "f16", False), ("bf16", "bf16", False)])
def test_gemm_grad_weight(env, counts, align, N, K, dtype, out, gather):
    torch, nat = env
    k, ldn = 2, -(-N // 8) * 8
    off, order, _, rows, x = _gemm_case(torch, counts, align, k, N, K, K, dtype, gather)
    E = len(counts)
    dy = _rand(torch, (rows, ldn), dtype, 6)
    pad = torch.from_numpy(order < 0).cuda()
    if gather:
        dy[pad] = float("nan")                       # nothing of a padding row enters
    else:
        x[int(off[-1]):] = float("nan")              # nor of rows behind the last segment
        dy[int(off[-1]):] = float("nan")
    g = torch.full((E, N, K), 7.0, dtype=_types(torch)[out], device="cuda")
    a = nat.make_expert_gemm(op="grad_weight", E=E, N=N, K=K, k=k, dtype=dtype, out_dtype=out, rows=rows, tokens=len(x), x=x, d_y=dy[:, :N], ld_d_y=ldn,
                             out=g, expert_off=torch.from_numpy(off).cuda(), order=torch.from_numpy(order).cuda() if gather else None)
    ws = _ws(torch, nat.moer_expert_gemm_workspace_bytes(a))
    nat.moer_expert_gemm(a, ws, ws.numel())
    assert nat.moer_ws_status(ws) == 0
    ref, mag = ex.gemm_weight_grad(_np(dy)[:, :N], _np(x), off, order if gather else None, k)
    _close(g, ref, (max(off[1:] - off[:-1]) + 1) * 2 * U * mag + _half_step(torch, out, ref))


def _to_8bit(v, bn):
    """Random-looking 8-bit rows: e4m3 codes' values and scales of blocks bn x 128."""
    import torch
    a = torch.from_numpy(v)
    s = np.stack([np.stack([np.abs(v[..., i * bn:(i + 1) * bn, j * 128:(j + 1) * 128]).max((-1, -2)) for j in range(ex.blocks(v.shape[-1]))], -1)
                  for i in range(-(-v.shape[-2] // bn))], -2).astype(np.float32) / np.float32(448)
    wide = np.repeat(np.repeat(s, bn, -2)[..., :v.shape[-2], :], 128, -1)[..., :v.shape[-1]]
    q = (a / torch.from_numpy(wide)).to(torch.float8_e4m3fn)
    return q, torch.from_numpy(s), wide.astype(np.float64)


@pytest.mark.parametrize("counts,align", COUNTS)
@pytest.mark.parametrize("N,K", [(256, 256), (64, 128), (8, 16), (136, 144), (1, 128), (520, 400), (300, 1040)])
@pytest.mark.parametrize("out,gather", [("bf16", True), ("f32", False)])
def test_gemm_8bit(env, counts, align, N, K, out, gather):
    torch, nat = env
    k = 2
    off, order, _, rows, x = _gemm_case(torch, counts, align, k, N, K, K, "f32", gather)
    E = len(counts)
    rs = np.random.RandomState(3)
    x = _np(x).astype(np.float32) * np.exp(rs.normal(size=(len(x), 1))).astype(np.float32)
    w = (rs.normal(size=(E, N, K)) * np.exp(rs.normal(size=(E, 1, 1)))).astype(np.float32)
    xq, xs, xw = _to_8bit(x, 1) if len(x) else (torch.zeros((0, K), dtype=torch.float8_e4m3fn), torch.zeros((0, ex.blocks(K))), np.zeros((0, K)))
    wq, wsc, ww = _to_8bit(w, 128)
    y = torch.full((rows, N), 7.0, dtype=_types(torch)[out], device="cuda")
    dev = [t.cuda() for t in (xq, xs, wq, wsc)]
    a = nat.make_expert_gemm(op="forward", E=E, N=N, K=K, k=k, dtype="e4m3", out_dtype=out, rows=rows, tokens=len(x), x=dev[0], x_scale=dev[1],
                             w=dev[2], w_scale=dev[3], out=y, expert_off=torch.from_numpy(off).cuda(),
                             order=torch.from_numpy(order).cuda() if gather else None)
    ws = _ws(torch, nat.moer_expert_gemm_workspace_bytes(a))
    nat.moer_expert_gemm(a, ws, ws.numel())
    assert nat.moer_ws_status(ws) == 0
    ref, mag = ex.gemm_rows(_np(xq.float()) * xw, _np(wq.float()) * ww, off, order if gather else None, k, out=np.full((rows, N), 7.0))
    _close(y, ref, (K + 4) * 2 * U * mag + _half_step(torch, out, ref))


@pytest.mark.parametrize("op", ["forward", "grad_input", "grad_weight"])
def test_gemm_strides(env, op):
    """Rows of x, weights and outputs that are slices of wider ones; experts that share their weights."""
    torch, nat = env
    counts, N, K, k = [70, 0, 33, 150], 136, 200, 1
    off, order, _, rows, _ = _gemm_case(torch, counts, 1, k, N, K, K, "bf16", True)
    E = len(counts)
    x = _wide(torch, _rand(torch, (rows, N if op == "grad_input" else K), "bf16", 1), 8)
    w = _wide(torch, _rand(torch, (E, N, K), "bf16", 2), 16)
    dy = _wide(torch, _rand(torch, (rows, N), "bf16", 3), 24)
    shape = {"forward": (rows, N), "grad_input": (rows, K), "grad_weight": (E, N, K)}[op]
    big = torch.full((*shape[:-1], shape[-1] + 3), 7.0, device="cuda")
    out = big[..., :-3]
    a = nat.make_expert_gemm(op=op, E=E, N=N, K=K, k=k, dtype="bf16", out_dtype="f32", rows=rows, tokens=len(x), x=x, w=w, d_y=dy, out=out,
                             expert_off=torch.from_numpy(off).cuda())
    ws = _ws(torch, nat.moer_expert_gemm_workspace_bytes(a))
    nat.moer_expert_gemm(a, ws, ws.numel())
    assert nat.moer_ws_status(ws) == 0 and (big[..., -3:] == 7).all()
    if op == "grad_weight":
        ref, mag = ex.gemm_weight_grad(_np(dy), _np(x), off)
    else:
        wv = _np(w) if op == "forward" else _np(w).transpose(0, 2, 1)
        ref, mag = ex.gemm_rows(_np(x), wv, off, out=np.full(shape, 7.0))
    _close(out, ref, 300 * 2 * U * mag + _half_step(torch, "f32", ref))
    if op == "forward":  # one expert's weights for all
        a = nat.make_expert_gemm(op=op, E=E, N=N, K=K, k=k, dtype="bf16", out_dtype="f32", rows=rows, tokens=len(x), x=x, w=w[:1], stride_w=0, out=out,
                                 expert_off=torch.from_numpy(off).cuda())
        nat.moer_expert_gemm(a, ws, ws.numel())
        ref, mag = ex.gemm_rows(_np(x), np.repeat(_np(w)[:1], E, 0), off, out=np.full(shape, 7.0))
        _close(out, ref, 300 * 2 * U * mag + _half_step(torch, "f32", ref))


@pytest.mark.parametrize("op", ["forward", "grad_weight"])
def test_gemm_bad_lists(env, op):
    """Offsets outside [0, rows] and falling ones are moved, order entries past the tokens are padding; both are said."""
    torch, nat = env
    E, N, K, rows, T = 4, 72, 64, 90, 30
    x, w, dy = _rand(torch, (T, K), "bf16", 1), _rand(torch, (E, N, K), "bf16", 2), _rand(torch, (rows, N), "bf16", 3)
    order = np.random.RandomState(0).permutation(90).astype(np.int32)
    order[[3, 40]] = [90, 2 ** 31 - 1]
    for off, good in (([0, 20, 20, 60, 200], [0, 20, 20, 60, 90]), ([-5, 20, 10, 60, 90], None), ([0, 20, 20, 60, 90], [0, 20, 20, 60, 90])):
        out = torch.full((rows, N) if op == "forward" else (E, N, K), 7.0, device="cuda")
        a = nat.make_expert_gemm(op=op, E=E, N=N, K=K, k=3, dtype="bf16", out_dtype="f32", rows=rows, tokens=T, x=x, w=w, d_y=dy, out=out,
                                 expert_off=torch.tensor(off, dtype=torch.int32, device="cuda"), order=torch.from_numpy(order).cuda())
        ws = _ws(torch, nat.moer_expert_gemm_workspace_bytes(a))
        nat.moer_expert_gemm(a, ws, ws.numel())
        assert nat.moer_ws_status(ws) == 6
        if good is None:
            continue
        if op == "forward":
            ref, mag = ex.gemm_rows(_np(x), _np(w), good, order, 3)
        else:
            ref, mag = ex.gemm_weight_grad(_np(dy), _np(x), good, order, 3)
        _close(out, ref, 100 * 2 * U * mag + _half_step(torch, "f32", ref))


def test_gemm_nan_and_infinity_stay_in_their_rows(env):
    torch, nat = env
    counts, N, K = [40, 70, 20], 72, 136
    off, order, _, rows, x = _gemm_case(torch, counts, 1, 1, N, K, K, "bf16", False, tail=0)
    w = _rand(torch, (3, N, K), "bf16", 2)
    x[39], x[40, 3], x[110, 7] = float("nan"), float("inf"), float("nan")
    y = torch.empty((rows, N), dtype=torch.bfloat16, device="cuda")
    a = nat.make_expert_gemm(op="forward", E=3, N=N, K=K, dtype="bf16", out_dtype="bf16", rows=rows, tokens=rows, x=x, w=w, out=y,
                             expert_off=torch.from_numpy(off).cuda())
    ws = _ws(torch, nat.moer_expert_gemm_workspace_bytes(a))
    nat.moer_expert_gemm(a, ws, ws.numel())
    bad = ~np.isfinite(_np(y)).all(1)
    assert np.flatnonzero(bad).tolist() == [39, 40, 110] and np.isnan(_np(y)[39]).all()
    # the weights' gradient: an expert's own rows alone
    g = torch.empty((3, N, K), dtype=torch.float32, device="cuda")
    x2 = _rand(torch, (rows, K), "bf16", 4)
    x2[40] = float("nan")
    a = nat.make_expert_gemm(op="grad_weight", E=3, N=N, K=K, dtype="bf16", out_dtype="f32", rows=rows, tokens=rows, x=x2, out=g,
                             d_y=_rand(torch, (rows, N), "bf16", 5), expert_off=torch.from_numpy(off).cuda())
    nat.moer_expert_gemm(a, ws, ws.numel())
    assert np.isfinite(_np(g)[0]).all() and np.isnan(_np(g)[1]).all() and np.isfinite(_np(g)[2]).all()


@pytest.mark.parametrize("op,dtype", [("forward", "bf16"), ("forward", "e4m3"), ("grad_input", "bf16"), ("grad_weight", "bf16")])
@pytest.mark.parametrize("gather,N", [(True, 768), (True, 512), (False, 768)])
def test_gemm_many_narrow_and_wide_tiles(env, op, dtype, gather, N):
    """Segments of few rows among long ones, over many tiles a block and many calls: threads that have
    nothing to bring for a tile must not lose their place in the stages (no wait expires), and every
    call gives the same bits."""
    torch, nat = env
    E, K, k = 96, 1536 if N == 768 else 512, 2
    rs = np.random.RandomState(0)
    counts = rs.choice([1, 2, 3, 9, 40, 130, 260], size=E)
    counts[-1] += counts.sum() % k
    off, order, _ = _lists(rs, counts, int(counts.sum()) // k, k, 1)
    rows, T = len(order), int(counts.sum()) // k
    n = T if gather else rows
    dev = dict(expert_off=torch.from_numpy(off).cuda(), order=torch.from_numpy(order).cuda() if gather else None)
    if dtype == "e4m3":
        q = torch.randint(0, 120, (n, K), dtype=torch.uint8, generator=torch.Generator().manual_seed(1)).cuda()
        w = torch.randint(0, 120, (E, N, K), dtype=torch.uint8, generator=torch.Generator().manual_seed(2)).cuda()
        dev.update(x=q, w=w, x_scale=torch.full((n, K // 128), 1e-3, device="cuda"), w_scale=torch.full((E, N // 128, K // 128), 1e-3, device="cuda"))
    else:
        dev.update(x=_rand(torch, (n, N if op == "grad_input" else K), dtype, 1), w=_rand(torch, (E, N, K), dtype, 2), d_y=_rand(torch, (rows, N), dtype, 3))
    out = torch.zeros({"forward": (rows, N), "grad_input": (rows, K), "grad_weight": (E, N, K)}[op], device="cuda")
    a = nat.make_expert_gemm(op=op, E=E, N=N, K=K, k=k, dtype=dtype, out_dtype="f32", rows=rows, tokens=n, out=out, **dev)
    ws = _ws(torch, nat.moer_expert_gemm_workspace_bytes(a))
    nat.moer_expert_gemm(a, ws, ws.numel())
    first = out.clone()
    for _ in range(150):
        nat.moer_expert_gemm(a, ws, ws.numel())
    assert nat.moer_ws_status(ws) == 0 and torch.equal(out, first) and torch.isfinite(out).all()


@pytest.mark.parametrize("E,stride", [(1024, 0), (5, 8), (5, 1024)])
def test_gemm_most_experts_and_odd_strides(env, E, stride):
    """As many experts as there may be, most without rows, and matrices that lie any multiple of eight
    elements apart."""
    torch, nat = env
    N, K = 72, 64
    rs = np.random.RandomState(E)
    counts = np.where(rs.rand(E) < 0.2, rs.randint(1, 40, E), 0)
    counts[0] = 300
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = int(off[-1])
    room = torch.zeros(E * (N * K + stride), dtype=torch.bfloat16, device="cuda")
    w = room.as_strided((E, N, K), (N * K + stride, K, 1))
    w.copy_(_rand(torch, (E, N, K), "bf16", 2))
    x = _rand(torch, (rows, K), "bf16", 1)
    y = torch.empty((rows, N), device="cuda")
    a = nat.make_expert_gemm(op="forward", E=E, N=N, K=K, dtype="bf16", out_dtype="f32", rows=rows, tokens=rows, x=x, w=w, out=y,
                             expert_off=torch.from_numpy(off).cuda())
    ws = _ws(torch)
    nat.moer_expert_gemm(a, ws, 256)
    assert nat.moer_ws_status(ws) == 0
    ref, mag = ex.gemm_rows(_np(x), _np(w), off)
    _close(y, ref, K * 2 * U * mag + _half_step(torch, "f32", ref))
    g = torch.empty((E, N, K), device="cuda")
    dy = _rand(torch, (rows, N), "bf16", 3)
    a = nat.make_expert_gemm(op="grad_weight", E=E, N=N, K=K, dtype="bf16", out_dtype="f32", rows=rows, tokens=rows, x=x, d_y=dy, out=g,
                             expert_off=torch.from_numpy(off).cuda())
    nat.moer_expert_gemm(a, ws, 256)
    assert nat.moer_ws_status(ws) == 0
    ref, mag = ex.gemm_weight_grad(_np(dy), _np(x), off)
    _close(g, ref, 301 * 2 * U * mag + _half_step(torch, "f32", ref))


def test_gemm_on_two_streams_at_once(env):
    """Calls that overlap, each with its own workspace, give what each gives alone."""
    torch, nat = env
    counts, N, K = [300, 17, 0, 520], 520, 264
    off, order, _, rows, x = _gemm_case(torch, counts, 1, 2, N, K, K, "bf16", True)
    w, dy = _rand(torch, (4, N, K), "bf16", 5), _rand(torch, (rows, N), "bf16", 6)
    lists = dict(expert_off=torch.from_numpy(off).cuda(), order=torch.from_numpy(order).cuda())

    def make(op, out):
        return nat.make_expert_gemm(op=op, E=4, N=N, K=K, k=2, dtype="bf16", out_dtype="f32", rows=rows, tokens=len(x), x=x, w=w, d_y=dy, out=out, **lists)
    outs = [[torch.zeros((rows, N), device="cuda"), torch.zeros((4, N, K), device="cuda")] for _ in range(2)]
    ws = [_ws(torch) for _ in range(2)]
    for op, o in zip(("forward", "grad_weight"), outs[0]):
        nat.moer_expert_gemm(make(op, o), ws[0], 256)
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(30):
        for op, o, s, v in zip(("forward", "grad_weight"), outs[1], sides, ws):
            nat.moer_expert_gemm(make(op, o), v, 256, s)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(*outs)) and all(nat.moer_ws_status(v) == 0 for v in ws)
