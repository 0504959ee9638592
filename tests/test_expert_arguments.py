"""The expert entry points' refusals, on the CPU: every call here is rejected on the host."""
import pytest

nat = pytest.importorskip("moe_expert_routing_top_gb300._native")

BADPTR = 0x1001  # misaligned, never dereferenced


def _code(fn, *args):
    with pytest.raises(nat.MoerError) as ei:
        fn(*args)
    return ei.value.code


NORM = dict(T=10, H=64, dtype="bf16", eps=1e-6, x=64, residual=64, weight=64, sum=64, y=64, q=64, scale=64, rstd=64, d_y=64,
            d_sum=64, d_x=64, d_weight=64, ld_x=64, ld_residual=64, ld_sum=64, ld_y=64, ld_q=64, ld_scale=1, ld_d_y=64,
            ld_d_sum=64, ld_d_x=64)


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), 3), (dict(T=1 << 31), 3), (dict(H=0), 3), (dict(H=16385), 3), (dict(dtype=3), 1), (dict(dtype=-1), 1),
    (dict(eps=-1.0), 3), (dict(eps=float("nan")), 3), (dict(eps=float("inf")), 3), (dict(x=None), 1), (dict(x=BADPTR), 1),
    (dict(weight=None), 1), (dict(residual=BADPTR), 1), (dict(sum=BADPTR), 1), (dict(y=BADPTR), 1), (dict(scale=None), 1),
    (dict(scale=0x1002), 1), (dict(rstd=0x1002), 1), (dict(ld_x=63), 2), (dict(ld_residual=63), 2), (dict(ld_y=0), 2),
    (dict(ld_q=63), 2), (dict(ld_scale=0), 2), (dict(ld_x=1 << 40), 2)])
def test_norm(over, code):
    assert _code(nat.moer_rms_norm, nat.make_norm(**{**NORM, **over}), None, 0, 0) == code


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), 3), (dict(H=0), 3), (dict(dtype=3), 1), (dict(sum=None), 1), (dict(weight=None), 1), (dict(rstd=None), 1),
    (dict(d_y=None), 1), (dict(d_x=None), 1), (dict(d_y=BADPTR), 1), (dict(d_sum=BADPTR), 1), (dict(d_weight=0x1002), 1),
    (dict(ld_d_y=63), 2), (dict(ld_d_x=63), 2), (dict(ld_sum=1), 2), (dict(ld_d_sum=1), 2)])
def test_norm_grad(over, code):
    n = nat.moer_rms_norm_workspace_bytes(10, 64)
    assert _code(nat.moer_rms_norm_grad, nat.make_norm(**{**NORM, **over}), 64, n, 0) == code


def test_norm_workspace():
    n = nat.moer_rms_norm_workspace_bytes(10, 64)
    assert n <= nat.moer_rms_norm_workspace_bytes(1 << 20, 64) and nat.moer_rms_norm_workspace_bytes(1, 0) == 256
    a = nat.make_norm(**NORM)
    assert _code(nat.moer_rms_norm_grad, a, None, n, 0) == 1
    assert _code(nat.moer_rms_norm_grad, a, 0x1008, n, 0) == 1
    assert _code(nat.moer_rms_norm_grad, a, 64, n - 1, 0) == 5
    nat.moer_rms_norm(nat.make_norm(T=0, H=64, dtype="bf16", eps=0.0), None, 0, 0)   # no rows: nothing to do
    assert nat.LIB.moer_rms_norm(None, None, 0, None) == 1 and nat.LIB.moer_rms_norm_grad(None, None, 0, None) == 1


GEMM = dict(op="forward", E=8, N=64, K=32, k=2, dtype="bf16", out_dtype="bf16", rows=100, tokens=50, expert_off=64, order=64, x=64, w=64,
            d_y=64, out=64, ld_x=64, ld_d_y=64, ld_w=32, ld_out=64, stride_w=2048, stride_out=4096)
FP8 = dict(GEMM, dtype="e4m3", x_scale=64, w_scale=64, ld_x_scale=1)
GW = dict(GEMM, op="grad_weight")


@pytest.mark.parametrize("base,over,code", [
    (GEMM, dict(op=3), 1), (GEMM, dict(op=-1), 1), (GEMM, dict(dtype="f32"), 1), (GEMM, dict(dtype=4), 1), (GEMM, dict(out_dtype="e4m3"), 1),
    (GEMM, dict(E=0), 3), (GEMM, dict(E=1025), 3), (GEMM, dict(N=0), 3), (GEMM, dict(N=65537), 3), (GEMM, dict(K=0), 3), (GEMM, dict(K=65537), 3),
    (GEMM, dict(rows=-1), 3), (GEMM, dict(rows=1 << 31), 3), (GEMM, dict(tokens=-1), 3), (GEMM, dict(tokens=1 << 31), 3), (GEMM, dict(k=0), 3),
    (GEMM, dict(order=None), 2),                                     # 100 rows of 50
    (GEMM, dict(expert_off=None), 1), (GEMM, dict(expert_off=0x1002), 1), (GEMM, dict(order=0x1002), 1),
    (GEMM, dict(x=None), 1), (GEMM, dict(x=0x1008), 1), (GEMM, dict(w=None), 1), (GEMM, dict(w=0x1008), 1), (GEMM, dict(out=None), 1),
    (GEMM, dict(out=BADPTR), 1), (GEMM, dict(out=0x1002, out_dtype="f32"), 1), (GEMM, dict(ld_x=24), 2), (GEMM, dict(ld_x=36), 1),
    (GEMM, dict(ld_w=31), 2), (GEMM, dict(ld_w=36), 1), (GEMM, dict(ld_out=63), 2), (GEMM, dict(stride_w=-8), 2), (GEMM, dict(stride_w=2052), 1),
    (GEMM, dict(op="grad_input", ld_x=56), 2), (GEMM, dict(op="grad_input", ld_out=31), 2),
    (GW, dict(d_y=None), 1), (GW, dict(d_y=0x1008), 1), (GW, dict(ld_d_y=63), 2), (GW, dict(ld_d_y=68), 1), (GW, dict(stride_out=64 * 64 - 33), 2),
    (GW, dict(ld_out=31), 2),
    (FP8, dict(op="grad_input"), 1), (FP8, dict(op="grad_weight"), 1), (FP8, dict(x_scale=None), 1), (FP8, dict(w_scale=None), 1),
    (FP8, dict(x_scale=0x1002), 1), (FP8, dict(w_scale=0x1002), 1), (FP8, dict(ld_x_scale=0), 2), (FP8, dict(ld_x=40), 1), (FP8, dict(ld_w=40), 1),
    (FP8, dict(stride_w=2056), 1)])
def test_gemm(base, over, code):
    a = nat.make_expert_gemm(**{**base, **over})
    assert _code(nat.moer_expert_gemm, a, 64, 1 << 20, 0) == code


def test_gemm_workspace():
    a = nat.make_expert_gemm(**GEMM)
    n = nat.moer_expert_gemm_workspace_bytes(a)
    assert _code(nat.moer_expert_gemm, a, None, n, 0) == 1
    assert _code(nat.moer_expert_gemm, a, 0x1008, n, 0) == 1
    assert _code(nat.moer_expert_gemm, a, 64, n - 1, 0) == 5
    nat.moer_expert_gemm(nat.make_expert_gemm(**{**GEMM, "rows": 0}), None, 0, 0)   # no rows: nothing to do
    assert nat.LIB.moer_expert_gemm(None, 64, n, None) == 1


ACT = dict(rows=10, I=64, dtype="bf16", h=64, used=64, y=64, q=64, scale=64, d_y=64, d_h=64, ld_h=128, ld_y=64, ld_q=64, ld_scale=1,
           ld_d_y=64, ld_d_h=128)


@pytest.mark.parametrize("grad,over,code", [
    (False, dict(rows=-1), 3), (False, dict(rows=1 << 31), 3), (False, dict(I=0), 3), (False, dict(I=65537), 3), (False, dict(dtype=3), 1),
    (False, dict(h=None), 1), (False, dict(h=BADPTR), 1), (False, dict(used=0x1002), 1), (False, dict(y=BADPTR), 1), (False, dict(scale=None), 1),
    (False, dict(y=None, q=None), 1), (False, dict(ld_h=127), 2), (False, dict(ld_y=63), 2), (False, dict(ld_q=1), 2), (False, dict(ld_scale=0), 2),
    (True, dict(d_y=None), 1), (True, dict(d_h=None), 1), (True, dict(d_y=BADPTR), 1), (True, dict(ld_d_y=63), 2), (True, dict(ld_d_h=127), 2),
    (True, dict(h=None), 1), (True, dict(I=0), 3)])
def test_act(grad, over, code):
    f = nat.moer_expert_act_grad if grad else nat.moer_expert_act
    assert _code(f, nat.make_expert_act(**{**ACT, **over}), 0) == code
    f(nat.make_expert_act(**{**ACT, "rows": 0, "h": None}), 0)


COMB = dict(T=10, H=64, k=2, rows=20, dtype="bf16", ld_z=64, ld_add=64, ld_out=64, ld_d_out=64, ld_d_z=64, inv=64, order=64, weights=64,
            z=64, add=64, out=64, d_out=64, d_z=64, d_weights=64)


@pytest.mark.parametrize("grad,over,code", [
    (False, dict(T=-1), 3), (False, dict(T=1 << 31), 3), (False, dict(T=1 << 30, k=2), 3), (False, dict(rows=-1), 3), (False, dict(H=0), 3),
    (False, dict(H=65537), 3), (False, dict(k=0), 3), (False, dict(k=33), 3), (False, dict(dtype=3), 1), (False, dict(inv=None), 1),
    (False, dict(inv=0x1002), 1), (False, dict(weights=0x1002), 1), (False, dict(z=None), 1), (False, dict(z=BADPTR), 1), (False, dict(add=BADPTR), 1),
    (False, dict(out=None), 1), (False, dict(ld_z=63), 2), (False, dict(ld_add=1), 2), (False, dict(ld_out=63), 2),
    (True, dict(order=None), 1), (True, dict(d_out=None), 1), (True, dict(z=None), 1), (True, dict(d_z=BADPTR), 1), (True, dict(d_weights=0x1002), 1),
    (True, dict(ld_d_out=63), 2), (True, dict(ld_d_z=63), 2), (True, dict(k=33), 3)])
def test_combine(grad, over, code):
    f = nat.moer_expert_combine_grad if grad else nat.moer_expert_combine
    assert _code(f, nat.make_expert_combine(**{**COMB, **over}), 64, 256, 0) == code


def test_combine_workspace():
    a = nat.make_expert_combine(**COMB)
    for f in (nat.moer_expert_combine, nat.moer_expert_combine_grad):
        assert _code(f, a, None, 256, 0) == 1 and _code(f, a, 0x1008, 256, 0) == 1 and _code(f, a, 64, 255, 0) == 5
    nat.moer_expert_combine(nat.make_expert_combine(**{**COMB, "T": 0}), 64, 256, 0)


def test_arguments_from_tensors():
    torch = pytest.importorskip("torch")
    wide = torch.zeros(6, 80)
    a = nat.make_norm(T=6, H=64, x=wide[:, :64], weight=torch.ones(64))
    assert a.ld_x == 80 and a.x == wide.data_ptr()
    w = torch.zeros(3, 8, 32)
    g = nat.make_expert_gemm(op="grad_weight", dtype="f16", out_dtype="f32", out=w, w=w[1:2])
    assert (g.op, g.dtype, g.out_dtype, g.ld_out, g.stride_out, g.ld_w) == (2, 2, 0, 32, 256, 32)
    with pytest.raises(ValueError):
        nat.make_norm(T=6, H=6, x=torch.zeros(6, 6).t())
    with pytest.raises(ValueError):
        nat.make_norm(T=6, H=6, weight=torch.zeros(12)[::2])
    with pytest.raises(TypeError):
        nat.make_norm(T=6, H=6, no_such_field=1)
