"""The last rounding of the expert operators: 8-bit rows are the e4m3 values nearest to their rows divided by
the block's scale, code by code, and rows in fp32 are as exact as fp32 arithmetic makes them."""
import numpy as np
import pytest

from oracle import experts as ex
from tests.test_gpu_experts import U, _np, _rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_routing_top_gb300 import _native as nat
    return torch, nat


def _same_codes(torch, y, q, scale):
    """y: the fp32 rows that q and scale stand for.  The fp32 quotient, rounded to e4m3 (ties to even)."""
    y, s = y.cpu(), scale.cpu()
    most = torch.stack([b.abs().amax(1) for b in y.split(128, 1)], 1)
    assert (np.abs(_np(s) - _np(most) / 448.0) <= 2 * U * _np(most) / 448.0).all()   # two roundings: of 1 / 448, and of the product
    want = (y / s.repeat_interleave(128, 1)[:, :y.shape[1]]).to(torch.float8_e4m3fn).view(torch.uint8)
    off = want != q.cpu().view(torch.uint8)
    assert not off.any(), f"{int(off.sum())} of {off.numel()} codes off"


def _borders(torch, cols, seed):
    """Values on the borders between e4m3 codes (and next to them), for blocks of many largest values."""
    v = ex.e4m3_values()[:127]
    mid = torch.from_numpy((v[1:] + v[:-1]) / 2)
    g = torch.Generator().manual_seed(seed)
    n = cols // 128
    most = torch.exp(torch.randn((n, 1), generator=g) * 3).float()
    s = (most * torch.tensor(1 / 448)).double()
    y = (mid[torch.randint(0, 126, (n, 128), generator=g)] * s).float()
    y = torch.nextafter(y, torch.where(torch.rand((n, 128), generator=g) < 0.5, 0.0, 1e30)) if seed % 2 else y
    y[:, 17:18] = most
    return torch.where(torch.rand((n, 128), generator=g) < 0.5, y, -y).view(cols)


@pytest.mark.parametrize("seed", range(6))
def test_norm_codes_on_borders(env, seed):
    """Rows of +-1 have a norm of exactly 1, so that the output is the weight."""
    torch, nat = env
    H, T = 16384, 3
    w = _borders(torch, H, seed).cuda()
    x = torch.ones((T, H), device="cuda")
    x[1] = -1
    x[2, ::2] = -1
    y, q, sc = torch.empty_like(x), torch.empty((T, H), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty((T, H // 128), device="cuda")
    nat.moer_rms_norm(nat.make_norm(T=T, H=H, dtype="f32", eps=0.0, x=x, weight=w, y=y, q=q, scale=sc))
    assert torch.equal(y, x * w)
    _same_codes(torch, y, q, sc)


@pytest.mark.parametrize("T,H", [(8192, 2048), (333, 1000), (7, 129), (1, 8)])
def test_norm_codes(env, T, H):
    torch, nat = env
    x, w = _rand(torch, (T, H), "f32", 1), _rand(torch, (H,), "f32", 2)
    y, q, sc = torch.empty_like(x), torch.empty((T, H), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty((T, ex.blocks(H)), device="cuda")
    nat.moer_rms_norm(nat.make_norm(T=T, H=H, dtype="f32", eps=1e-6, x=x, weight=w, y=y, q=q, scale=sc))
    _same_codes(torch, y, q, sc)


@pytest.mark.parametrize("rows,I", [(8192, 768), (333, 1000), (7, 129), (1, 8)])
def test_act_codes(env, rows, I):
    torch, nat = env
    h = _rand(torch, (rows, 2 * I), "f32", 1, 2.0)
    y, q, sc = torch.empty((rows, I), device="cuda"), torch.empty((rows, I), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty((rows, ex.blocks(I)), device="cuda")
    nat.moer_expert_act(nat.make_expert_act(rows=rows, I=I, dtype="f32", h=h, y=y, q=q, scale=sc))
    _same_codes(torch, y, q, sc)


def test_codes_of_extremes(env):
    """Blocks of NaN (what linspace makes of a range that fp32 does not hold), of the smallest scales, of zeros,
    with an infinity and with a NaN."""
    torch, nat = env
    w = torch.ones(768)
    w[:128] = torch.linspace(-3e38, 3e38, 128)
    w[128:256] = torch.linspace(-1e-30, 1e-30, 128)
    w[256:384] = 0.0
    w[384:512] = torch.linspace(1e-42, 1e-38, 128)
    w[520], w[650] = float("inf"), float("nan")
    x = torch.ones((1, 768), device="cuda")
    y, q, sc = torch.empty_like(x), torch.empty((1, 768), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty((1, 6), device="cuda")
    nat.moer_rms_norm(nat.make_norm(T=1, H=768, dtype="f32", eps=0.0, x=x, weight=w.cuda(), y=y, q=q, scale=sc))
    s = sc[0].cpu()
    least = torch.tensor(1e-30) * torch.tensor(1 / 448)
    assert s[2] == least and s[3] == least and s[4] == float("inf") and s[5] == torch.tensor(1 / 448)
    got, wide = q.cpu().float()[0], s.repeat_interleave(128)
    for at in (slice(0, 128), slice(128, 256), slice(256, 384), slice(384, 512)):
        want = (w / wide).to(torch.float8_e4m3fn).float()[at]
        assert torch.equal(got[at].isnan(), want.isnan()) and torch.equal(got[at].nan_to_num(), want.nan_to_num())
    stands = got * wide                                # an infinity: nothing of its block is a number
    assert stands[512:640].isnan().all() and got[650].isnan() and (got[640:650] == 448).all() and (got[651:] == 448).all()


def test_codes_of_the_largest_scales(env):
    torch, nat = env
    w = torch.cat([torch.linspace(-1, 1, 128) * 3e38, torch.linspace(0, 3.4028e38, 128), torch.linspace(-1, 1, 128) * 1e30])
    x, y = torch.ones((1, 384), device="cuda"), torch.empty((1, 384), device="cuda")
    q, sc = torch.empty((1, 384), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty((1, 3), device="cuda")
    nat.moer_rms_norm(nat.make_norm(T=1, H=384, dtype="f32", eps=0.0, x=x, weight=w.cuda(), y=y, q=q, scale=sc))
    assert torch.equal(y.cpu()[0], w) and w.isfinite().all()
    _same_codes(torch, y, q, sc)


def _arguments(torch):
    a = torch.cat([torch.linspace(-80, 80, 40001), torch.linspace(-2, 2, 8007)])
    return a.view(-1, 8).float().cuda()


def test_act_in_fp32(env):
    """Rows of fp32: the exponential (one step, 2 U), the sum, the division and two products, U each, are 6 U of
    the value; 8 U for terms of second order."""
    torch, nat = env
    a = _arguments(torch)
    b = _rand(torch, a.shape, "f32", 3)
    h, y = torch.cat([a, b], 1), torch.empty_like(a)
    nat.moer_expert_act(nat.make_expert_act(rows=len(a), I=8, dtype="f32", h=h, y=y))
    ref = ex.silu_gate(_np(h))
    bad = ~(np.abs(_np(y) - ref) <= 8 * U * np.abs(ref))
    assert not bad.any(), f"{bad.sum()} off, by {(np.abs(_np(y) - ref)[bad] / np.abs(ref)[bad]).max() / U} U"


def test_act_grad_in_fp32(env):
    """s is off by 4 U of itself, 1 - s by 4 U s + U, a (1 - s) by (4 s + 2) U |a|, 1 + a (1 - s) by that and U (1 + |a|),
    the products d b s and that by 4 U + 3 U: 14 U of d b s (1 + 2 |a|) holds them; d a s has 4 U + 2 U of itself."""
    torch, nat = env
    a = _arguments(torch)
    b, d = _rand(torch, a.shape, "f32", 3), _rand(torch, a.shape, "f32", 4)
    h = torch.cat([a, b], 1)
    dh = torch.empty_like(h)
    nat.moer_expert_act_grad(nat.make_expert_act(rows=len(a), I=8, dtype="f32", h=h, d_y=d, d_h=dh))
    ref = ex.silu_gate_grad(_np(h), _np(d))
    av, bv, dv = _np(a), _np(b), _np(d)
    s = ex.sigmoid(av)
    mag = np.concatenate([np.abs(dv * bv) * s * (1 + 2 * np.abs(av)) * 14, np.abs(dv * av) * s * 8], 1)
    bad = ~(np.abs(_np(dh) - ref) <= U * mag)
    assert not bad.any(), f"{bad.sum()} off, by {(np.abs(_np(dh) - ref)[bad] / (U * mag[bad])).max()} of the bound"
