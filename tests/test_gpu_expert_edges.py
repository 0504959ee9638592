"""The expert operators at the edges of what the header allows, against the 64-bit statements
(oracle/experts.py), with the tolerances of test_gpu_experts.py."""
import os
import subprocess
import sys

import numpy as np
import pytest

from oracle import experts as ex
from tests.test_gpu_experts import U, _close, _half_step, _lists, _np, _rand, _types, _ws

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_routing_top_gb300 import _native as nat
    return torch, nat


# ------------------------------------------------------------------ norm
def norm_grad_of(H, dtype, T=5):
    import torch

    from moe_expert_routing_top_gb300 import _native as nat
    s, w, dy = (_rand(torch, n, dtype, i) for i, n in enumerate(((T, H), (H,), (T, H))))
    rstd = torch.from_numpy(ex.rms_norm(_np(s), _np(w), 1e-6)[1]).float().cuda()
    dx, dw = torch.empty_like(s), torch.empty(H, device="cuda")
    n = nat.moer_rms_norm_workspace_bytes(T, H)
    nat.moer_rms_norm_grad(nat.make_norm(T=T, H=H, dtype=dtype, eps=1e-6, sum=s, weight=w, rstd=rstd, d_y=dy, d_x=dx, d_weight=dw), _ws(torch, n), n)
    rx, mx, rw, mw = ex.rms_norm_grad(_np(s), _np(w), _np(rstd), _np(dy))
    _close(dx, rx, (H + 24) * 2 * U * mx + _half_step(torch, dtype, rx), f"d_x of {H}")
    _close(dw, rw, (T + 16) * 2 * U * mw + 1e-44, f"d_weight of {H}")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_norm_gradient_next_to_48_KB(env, dtype):
    """Rows whose weight's gradient takes 48 KB of shared memory or a little less: with the kernel's own
    64 bytes they need more than a launch has by default.  In a process of its own, smallest first: a call with
    a longer row raises the kernel's limit for good."""
    code = f"from tests.test_gpu_expert_edges import norm_grad_of\nfor H in (12272, 12273, 12280, 12281, 12288, 12289, 12296): norm_grad_of(H, {dtype!r})"
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


# ------------------------------------------------------------------ combination
@pytest.mark.parametrize("T,k,H,align", [(1, 1, 8, 4), (33, 6, 264, 16), (17, 9, 3, 1), (8, 32, 72, 1), (300, 4, 96, 128), (2000, 8, 40, 16)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_combine_grad_of_dropped_pairs(env, T, k, H, align, dtype):
    """A pair without a row adds nothing: the row that the lists still hold for it gets zeros, like
    one that is padding."""
    torch, nat = env
    rs = np.random.RandomState(T)
    off, order, inv = _lists(rs, np.bincount(rs.randint(0, 7, T * k), minlength=7), T, k, align)
    order = np.concatenate([order, np.full(3, -1, np.int32)])
    rows = len(order)
    inv.reshape(-1)[rs.rand(T * k) < 0.3] = -1
    inv[0, 0] = -5
    z, w, do = _rand(torch, (rows, H), dtype, 1), torch.rand((T, k), generator=torch.Generator().manual_seed(2)).cuda(), _rand(torch, (T, H), dtype, 3)
    dz, dw, ws = torch.full((rows, H), float("nan"), dtype=z.dtype, device="cuda"), torch.full((T, k), float("nan"), device="cuda"), _ws(torch)
    nat.moer_expert_combine_grad(nat.make_expert_combine(T=T, H=H, k=k, rows=rows, dtype=dtype, inv=torch.from_numpy(inv).cuda(), weights=w, z=z, d_out=do,
                                                         order=torch.from_numpy(order).cuda(), d_z=dz, d_weights=dw), ws, 256)
    assert nat.moer_ws_status(ws) == 0
    rz, rw, mw = ex.combine_grad(_np(z), inv, _np(w), _np(do), rows)
    _close(dz, rz, U * np.abs(rz) + _half_step(torch, dtype, rz), "d_z")
    _close(dw, rw, (H + 2) * 2 * U * mw, "d_weights")
    assert (dz[torch.from_numpy(rz == 0).cuda().all(1)] == 0).all()


def test_combine_grad_of_entries_that_name_no_pair(env):
    """An entry past the pairs is padding and is said; one whose pair has another row is said too, and its
    row is left."""
    torch, nat = env
    T, k, H, rows = 4, 2, 16, 12
    do, ws = _rand(torch, (T, H), "f32", 2), _ws(torch)
    order = np.concatenate([np.arange(8), [-1, -7, -1, -1]]).astype(np.int32)
    inv = torch.arange(8, dtype=torch.int32, device="cuda").view(T, k)

    def grad(order, inv, T=T):
        dz = torch.full((rows, H), 5.0, device="cuda")
        nat.moer_expert_combine_grad(nat.make_expert_combine(T=T, H=H, k=k, rows=rows, dtype="f32", inv=inv, order=torch.from_numpy(order).cuda(),
                                                             d_out=do[:T], d_z=dz), ws, 256)
        return dz, nat.moer_ws_status(ws)
    want, status = grad(order, inv)
    assert status == 0 and torch.equal(want[:8], do.repeat_interleave(k, 0)) and (want[8:] == 0).all()
    for bad in (8, 9, 2 ** 31 - 1):
        o = order.copy()
        o[[8, 11]] = bad
        dz, status = grad(o, inv)
        assert status == 6 and torch.equal(dz, want)
    o = order.copy()
    o[9] = 3                                        # whose row is 3
    dz, status = grad(o, inv)
    assert status == 6 and (dz[9] == 5).all()
    dz[9] = 0
    assert torch.equal(dz, want)
    past = inv.clone()
    past[1, 1] = rows                               # counts as none, and row 3 gets nothing
    dz, status = grad(order, past)
    assert status == 6 and (dz[3] == 0).all()
    dz, status = grad(order, None, 0)               # without tokens every entry is past the pairs
    assert status == 6 and (dz == 0).all()
    dz, status = grad(np.full(rows, -1, np.int32), None, 0)
    assert status == 0 and (dz == 0).all()


# ------------------------------------------------------------------ products without tokens
@pytest.mark.parametrize("op,dtype", [("forward", "bf16"), ("forward", "e4m3"), ("grad_input", "f16"), ("grad_weight", "bf16")])
@pytest.mark.parametrize("off,low,high,entry,status", [
    ([0, 16, 16, 40], 0, 40, -1, 0), ([8, 16, 24, 40], 8, 40, -1, 0), ([8, 8, 8, 8], 8, 8, -1, 0), ([8, 24, 16, 40], 8, 40, -1, 6),
    ([-4, 16, 16, 40], 0, 40, -1, 6), ([8, 16, 24, 99], 8, 50, -1, 6), ([8, 16, 24, 40], 8, 40, 0, 6)])
def test_products_without_tokens(env, op, dtype, off, low, high, entry, status):
    """Lists of padding alone: zeros in the rows of segments, those before the first and behind the last
    one left; offsets that fall or leave the rows are said, and so is an entry that names a token."""
    torch, nat = env
    E, N, K, rows = 3, 48, 32, 50
    order = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    order[10] = entry
    if low == 8 and high < 50:
        order[[0, 7, 49]] = 5                       # of no segment
    xc, dt = N if op == "grad_input" else K, torch.uint8 if dtype == "e4m3" else _types(torch)[dtype]
    shape = {"forward": (rows, N), "grad_input": (rows, K), "grad_weight": (E, N, K)}[op]
    out, ws = torch.full(shape, 7.0, device="cuda"), _ws(torch)
    more = dict(x_scale=torch.zeros((0, 1), device="cuda"), w_scale=torch.ones((E, 1, 1), device="cuda")) if dtype == "e4m3" else {}
    a = nat.make_expert_gemm(op=op, E=E, N=N, K=K, k=2, dtype=dtype, out_dtype="f32", rows=rows, tokens=0, x=torch.zeros((0, xc), dtype=dt, device="cuda"),
                             w=torch.zeros((E, N, K), dtype=dt, device="cuda"), d_y=torch.ones((rows, N), dtype=dt, device="cuda"), out=out,
                             expert_off=torch.tensor(off, dtype=torch.int32, device="cuda"), order=order, **more)
    nat.moer_expert_gemm(a, ws, 256)
    assert nat.moer_ws_status(ws) == status
    if op == "grad_weight":
        assert (out == 0).all()
    else:
        assert (out[low:high] == 0).all() and (out[:low] == 7).all() and (out[high:] == 7).all()


# ------------------------------------------------------------------ long calls
def test_a_product_of_more_than_two_seconds(env):
    """Waits are bounded to two seconds without progress, not calls: a weights' gradient over 120 million rows
    (d_y's elements pass 2^31) takes longer.  Whole numbers, few of them not zero, so that every sum is exact;
    NaN in rows of padding."""
    torch, nat = env
    N, K, rows, k = 24, 65536, 120_000_000, 1 << 20
    T = -(-rows // k)
    g = torch.Generator().manual_seed(0)
    x = torch.randint(-8, 9, (T, K), generator=g).bfloat16().cuda()
    at = torch.randperm(rows, generator=g, dtype=torch.int32)[:1024].long()
    at[:4] = torch.tensor([0, rows - 1, rows - 2, 64])
    at = torch.unique(at)
    pad, at = at[1::3], torch.cat([at[::3], at[2::3]])
    dy = torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda")
    order = torch.arange(rows, dtype=torch.int32, device="cuda")
    some = torch.randint(-4, 5, (len(at), N), generator=g).bfloat16()
    dy[at.cuda()] = some.cuda()
    dy[pad.cuda()] = float("nan")
    order[pad.cuda()] = -1
    out, ws = torch.empty((1, N, K), device="cuda"), _ws(torch)
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    a = nat.make_expert_gemm(op="grad_weight", E=1, N=N, K=K, k=k, dtype="bf16", out_dtype="f32", rows=rows, tokens=T, x=x, d_y=dy, out=out, expert_off=off,
                             order=order)
    nat.moer_expert_gemm(a, ws, 256)
    assert nat.moer_ws_status(ws) == 0
    want = some.double().T @ x.cpu().double()[at // k]
    assert torch.equal(out[0].cpu().double(), want)
