"""The expert operators on buffers of more than 2^31 elements: rows on both sides of that offset against the
same rows in a small buffer (bit by bit), or against the 64-bit statements."""
import numpy as np
import pytest

from oracle import experts as ex
from tests.test_gpu_experts import U, _close, _half_step, _np, _ws

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_routing_top_gb300 import _native as nat
    yield torch, nat
    torch.cuda.empty_cache()


def _big(torch, *shape, seed=1):
    return torch.randn(shape, device="cuda", dtype=torch.bfloat16, generator=torch.Generator(device="cuda").manual_seed(seed))


def test_norm(env):
    torch, nat = env
    T, H = 131072 + 3000, 16384
    at = torch.tensor([0, 1, 65535, 65536, 131071, 131072, 131073, T - 1], device="cuda")
    x, w = _big(torch, T, H), _big(torch, H, seed=2)

    def norm(x):
        o = dict(y=torch.empty_like(x), q=torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda"), scale=torch.empty((len(x), H // 128), device="cuda"),
                 rstd=torch.empty(len(x), device="cuda"))
        nat.moer_rms_norm(nat.make_norm(T=len(x), H=H, dtype="bf16", eps=1e-6, x=x, weight=w, **o))
        return o
    got, want = norm(x), norm(x[at])
    assert all(torch.equal(got[n].view(torch.uint8)[at] if n == "q" else got[n][at], want[n].view(torch.uint8) if n == "q" else want[n]) for n in want)
    y, rstd = got["y"], got["rstd"]
    del got

    def grad(x, dy, rstd):
        dx, n = torch.empty_like(x), nat.moer_rms_norm_workspace_bytes(len(x), H)
        nat.moer_rms_norm_grad(nat.make_norm(T=len(x), H=H, dtype="bf16", eps=1e-6, sum=x, weight=w, rstd=rstd, d_y=dy, d_x=dx), _ws(torch, n), n)
        return dx
    assert torch.equal(grad(x, y, rstd)[at], grad(x[at], y[at], rstd[at]))


def test_activation(env):
    torch, nat = env
    rows, I = 16384 + 500, 65536
    at = torch.tensor([0, 16383, 16384, 16385, rows - 1], device="cuda")
    h = _big(torch, rows, 2 * I)

    def act(h):
        o = dict(y=torch.empty((len(h), I), dtype=h.dtype, device="cuda"), q=torch.empty((len(h), I), dtype=torch.uint8, device="cuda"),
                 scale=torch.empty((len(h), I // 128), device="cuda"))
        nat.moer_expert_act(nat.make_expert_act(rows=len(h), I=I, dtype="bf16", h=h, **o))
        return o
    got, want = act(h), act(h[at])
    assert all(torch.equal(got[n][at], want[n]) for n in want)
    dy = got["y"]
    some = h[at]
    for part, d in ((some, dy[at]), (h, dy)):       # in place
        nat.moer_expert_act_grad(nat.make_expert_act(rows=len(part), I=I, dtype="bf16", h=part, d_y=d, d_h=part))
    assert torch.equal(h[at], some)


def test_combination(env):
    torch, nat = env
    rows, H, T, k = 32768 + 300, 65536, 40, 3
    rs = np.random.RandomState(0)
    at = np.concatenate([[0, 32767, 32768, 32769, rows - 1], rs.permutation(np.arange(1, 32767))[:T * k - 55], 32770 + rs.permutation(290)[:50]])
    inv = rs.permutation(at).reshape(T, k).astype(np.int32)
    order = np.full(rows, -1, np.int32)
    order[inv.reshape(-1)] = np.arange(T * k)
    z, do, w, ws = _big(torch, rows, H), _big(torch, T, H, seed=2), torch.rand((T, k), device="cuda"), _ws(torch)
    small = z[torch.from_numpy(inv.reshape(-1).astype(np.int64)).cuda()]
    outs = []
    for zz, iv, od in ((z, inv, order), (small, np.arange(T * k, dtype=np.int32).reshape(T, k), np.arange(T * k, dtype=np.int32))):
        out, dz, dw = torch.empty_like(do), torch.full_like(zz, 7.0), torch.empty_like(w)
        base = dict(T=T, H=H, k=k, rows=len(zz), dtype="bf16", z=zz, inv=torch.from_numpy(iv).cuda(), weights=w)
        nat.moer_expert_combine(nat.make_expert_combine(out=out, **base), ws, 256)
        nat.moer_expert_combine_grad(nat.make_expert_combine(order=torch.from_numpy(od).cuda(), d_out=do, d_z=dz, d_weights=dw, **base), ws, 256)
        assert nat.moer_ws_status(ws) == 0
        outs.append((out, dw, dz))
    (out, dw, dz), (out2, dw2, dz2) = outs
    assert torch.equal(out, out2) and torch.equal(dw, dw2)
    assert torch.equal(dz[torch.from_numpy(inv.reshape(-1).astype(np.int64)).cuda()], dz2)
    assert (dz[torch.from_numpy(order < 0).cuda()] == 0).all()


@pytest.mark.parametrize("what", ["out", "x", "x by a list", "x in 8 bits"])
def test_products_of_long_rows(env, what):
    torch, nat = env
    rows, wide, slim = 32768 + 300, 65536, 64
    N, K = (wide, slim) if what == "out" else (slim, wide)
    off = np.array([0, 5, 32760, 32770, rows], np.int32)
    order = np.random.RandomState(1).permutation(rows).astype(np.int32) if what == "x by a list" else None
    x, w = _big(torch, rows, K), _big(torch, 4, N, K, seed=2)
    more = dict(dtype="bf16")
    if what == "x in 8 bits":
        x, w = x.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn)
        more = dict(dtype="e4m3", x_scale=torch.ones((rows, K // 128), device="cuda"), w_scale=torch.ones((4, 1, K // 128), device="cuda"))
    y, ws = torch.empty((rows, N), dtype=torch.float32, device="cuda"), _ws(torch)
    a = nat.make_expert_gemm(op="forward", E=4, N=N, K=K, k=1, out_dtype="f32", rows=rows, tokens=rows, x=x, w=w, out=y, expert_off=torch.from_numpy(off).cuda(),
                             order=None if order is None else torch.from_numpy(order).cuda(), **more)
    nat.moer_expert_gemm(a, ws, 256)
    assert nat.moer_ws_status(ws) == 0
    wv = _np(w.float())
    for p in (0, 4, 5, 32759, 32767, 32768, 32769, 32770, rows - 1):
        xv, e = _np(x[p if order is None else int(order[p])].float()), int(np.searchsorted(off, p, "right")) - 1
        ref, mag = wv[e] @ xv, np.abs(wv[e]) @ np.abs(xv)
        _close(y[p], ref, K * 2 * U * mag + _half_step(torch, "f32", ref), str(p))


@pytest.mark.parametrize("op", ["forward", "grad_input", "grad_weight"])
def test_products_of_large_weights(env, op):
    """Weights, or their gradient, of more than 2^31 elements."""
    torch, nat = env
    E, N, K, each = 34, 8192, 8192, 3
    rows = E * each
    off = torch.arange(0, rows + 1, each, dtype=torch.int32, device="cuda")
    x, dy, ws = _big(torch, rows, N if op == "grad_input" else K), _big(torch, rows, N, seed=3), _ws(torch)
    w = None if op == "grad_weight" else _big(torch, E, N, K, seed=2)
    out = torch.empty({"forward": (rows, N), "grad_input": (rows, K), "grad_weight": (E, N, K)}[op], dtype=torch.float32, device="cuda")
    a = nat.make_expert_gemm(op=op, E=E, N=N, K=K, dtype="bf16", out_dtype="f32", rows=rows, tokens=rows, x=x, w=w, d_y=dy, out=out, expert_off=off)
    nat.moer_expert_gemm(a, ws, 256)
    assert nat.moer_ws_status(ws) == 0
    for e in (0, 31, 32, 33):
        xv = _np(x[e * each:(e + 1) * each])
        if op == "grad_weight":
            dv = _np(dy[e * each:(e + 1) * each])
            _close(out[e], dv.T @ xv, (each + 1) * 2 * U * (np.abs(dv).T @ np.abs(xv)) + _half_step(torch, "f32", dv.T @ xv), str(e))
            continue
        wv = _np(w[e]).T if op == "forward" else _np(w[e])
        _close(out[e * each:(e + 1) * each], xv @ wv, N * 2 * U * (np.abs(xv) @ np.abs(wv)) + _half_step(torch, "f32", xv @ wv), str(e))


def test_a_long_segment(env):
    """The weights' gradient over thousands of rows an expert, some of them padding, at the bounds of short ones."""
    torch, nat = env
    E, N, K, k = 3, 136, 72, 2
    rs = np.random.RandomState(0)
    off = np.array([0, 4001, 4001, 9003], np.int32)
    rows = 9010
    order = rs.permutation(rows).astype(np.int32)
    order[rs.rand(rows) < 0.05] = -1
    x, dy, ws = _big(torch, rows // k, K), _big(torch, rows, N, seed=2), _ws(torch)
    dy[torch.from_numpy(order < 0).cuda()] = float("nan")
    g = torch.empty((E, N, K), device="cuda")
    a = nat.make_expert_gemm(op="grad_weight", E=E, N=N, K=K, k=k, dtype="bf16", out_dtype="f32", rows=rows, tokens=len(x), x=x, d_y=dy, out=g,
                             expert_off=torch.from_numpy(off).cuda(), order=torch.from_numpy(order).cuda())
    nat.moer_expert_gemm(a, ws, 256)
    assert nat.moer_ws_status(ws) == 0
    ref, mag = ex.gemm_weight_grad(_np(dy), _np(x), off, order, k)
    _close(g, ref, (5002 + 1) * 2 * U * mag + _half_step(torch, "f32", ref))
