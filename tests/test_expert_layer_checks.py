"""What ExpertLayer hands to the library, and what it refuses, on the CPU: the library's calls are
replaced by a recorder, so nothing is launched."""
import pytest

torch = pytest.importorskip("torch")
nat = pytest.importorskip("moe_expert_routing_top_gb300._native")
from moe_expert_routing_top_gb300 import pipeline  # noqa: E402

E, H, I, T, k = 4, 64, 32, 6, 2
BF, F8, F32, I32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.int32
CALLS = ("moer_rms_norm", "moer_rms_norm_grad", "moer_expert_gemm", "moer_expert_act", "moer_expert_act_grad", "moer_expert_combine",
         "moer_expert_combine_grad")


@pytest.fixture
def calls(monkeypatch):
    seen = []
    for name in CALLS:
        monkeypatch.setattr(nat, name, lambda *a, _n=name: seen.append((_n, a[0])))
    return seen


def _layer(dtype=BF, **more):
    w1, w2 = torch.zeros((E, 2 * I, H), dtype=dtype), torch.zeros((E, H, I), dtype=dtype)
    return pipeline.ExpertLayer(w1, w2, norm_weight=torch.ones(H, dtype=BF if dtype == F8 else dtype), **more)


def _scales():
    return torch.ones((E, 1, 1)), torch.ones((E, 1, 1))


def _lists(rows=20):
    return torch.zeros(E + 1, dtype=I32), torch.zeros(rows, dtype=I32), torch.zeros((T, k), dtype=I32), torch.zeros((T, k))


def test_forward_and_backward_calls(calls):
    layer = _layer()
    out, kept = layer.forward(torch.zeros((T, H), dtype=BF), *_lists(), add=torch.zeros((T, H), dtype=BF))
    assert [c[0] for c in calls] == ["moer_expert_gemm", "moer_expert_act", "moer_expert_gemm", "moer_expert_combine"]
    g1, act, g2, comb = (c[1] for c in calls)
    assert (g1.N, g1.K, g1.rows, g1.tokens, g1.k, g1.op) == (2 * I, H, 20, T, k, 0) and g1.order
    assert (g2.N, g2.K, g2.rows, g2.tokens) == (H, I, 20, 20) and not g2.order
    assert act.used == kept.off.data_ptr() + 4 * E and (act.ld_h, act.ld_y) == (2 * I, I)
    assert out.shape == (T, H) and comb.add and (comb.T, comb.k, comb.rows) == (T, k, 20)
    calls.clear()
    g = layer.backward(kept, torch.zeros((T, H), dtype=BF))
    assert [c[0] for c in calls] == ["moer_expert_combine_grad", "moer_expert_gemm", "moer_expert_gemm", "moer_expert_act_grad", "moer_expert_gemm",
                                     "moer_expert_gemm", "moer_expert_combine"]
    assert [c[1].op for c in calls if c[0] == "moer_expert_gemm"] == [1, 2, 2, 1]
    assert g["w1"].shape == (E, 2 * I, H) and g["w1"].dtype == F32 and g["weights"].shape == (T, k) and g["x"].dtype == BF


def test_eight_bit_calls(calls):
    layer = _layer(F8, scales=_scales())
    (q, s, y), total, rstd = layer.norm(torch.zeros((T, H), dtype=BF), torch.zeros((T, H), dtype=BF))
    assert (q.dtype, y.dtype, s.shape, total.shape, rstd.shape) == (F8, BF, (T, 1), (T, H), (T,))
    calls.clear()
    out, kept = layer.forward((q, s), *_lists())
    assert kept is None and out.dtype == BF
    assert all(c[1].dtype == nat.DTYPES["e4m3"] and c[1].x_scale and c[1].w_scale for c in calls if c[0] == "moer_expert_gemm")
    with pytest.raises(ValueError):
        layer.backward(kept, out)
    with pytest.raises(ValueError):
        layer.forward((torch.zeros((T, H), dtype=BF), s), *_lists())


@pytest.mark.parametrize("make", [
    lambda: pipeline.ExpertLayer(torch.zeros((E, 2 * I + 1, H), dtype=BF), torch.zeros((E, H, I), dtype=BF)),
    lambda: pipeline.ExpertLayer(torch.zeros((E, 2 * I, H), dtype=BF), torch.zeros((E, I, H), dtype=BF)),
    lambda: pipeline.ExpertLayer(torch.zeros((E, 2 * I, H)), torch.zeros((E, H, I))),
    lambda: pipeline.ExpertLayer(torch.zeros((E, 2 * I, H), dtype=BF), torch.zeros((E, H, I), dtype=torch.float16)),
    lambda: pipeline.ExpertLayer(torch.zeros((E, 2 * I, 2 * H), dtype=BF)[:, :, ::2], torch.zeros((E, H, I), dtype=BF)),
    lambda: pipeline.ExpertLayer(torch.zeros((E, 2 * 12, H), dtype=BF), torch.zeros((E, H, 12), dtype=BF)),
    lambda: pipeline.ExpertLayer(torch.zeros((E, 2 * 24, H), dtype=F8), torch.zeros((E, H, 24), dtype=F8), scales=_scales()),
    lambda: _layer(F8),
    lambda: _layer(BF, scales=_scales()),
    lambda: _layer(F8, scales=(torch.ones((E, 1, 2)), torch.ones((E, 1, 1)))),
    lambda: _layer(F8, scales=tuple(s.double() for s in _scales())),
    lambda: pipeline.ExpertLayer(torch.zeros((E, 2 * I, H), dtype=BF), torch.zeros((E, H, I), dtype=BF), norm_weight=torch.ones(H)),
    lambda: pipeline.ExpertLayer(torch.zeros((E, 2 * I, H), dtype=BF), torch.zeros((E, H, I), dtype=BF), norm_weight=torch.ones(H + 1, dtype=BF))])
def test_layers_that_do_not_fit(make):
    with pytest.raises(ValueError):
        make()


def _x(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("change", [
    dict(x=_x(T, H + 8)), dict(x=_x(T + 1, H)), dict(x=_x(T, H, dtype=torch.float16)), dict(x=_x(H, T).t()), dict(x=_x(1, T, H)), dict(x=_x(T, H).to("meta")),
    dict(off=_x(E, dtype=I32)), dict(off=_x(E + 1, dtype=torch.int64)), dict(off=_x(2, E + 1, dtype=I32)), dict(order=_x(2, 20, dtype=I32)),
    dict(order=_x(20, dtype=torch.int64)), dict(order=_x(40, dtype=I32)[::2]), dict(inv=_x(T * k, dtype=I32)), dict(inv=_x(T, k, dtype=torch.int64)),
    dict(inv=_x(k, T, dtype=I32).t()), dict(weights=_x(T, k)), dict(weights=_x(T, k + 1, dtype=F32)), dict(weights=_x(T, k, dtype=torch.float64)),
    dict(add=_x(T, H + 1)), dict(add=_x(T - 1, H)), dict(add=_x(T, H, dtype=F32))])
def test_arguments_that_do_not_fit(calls, change):
    off, order, inv, weights = _lists()
    a = dict(x=_x(T, H), off=off, order=order, inv=inv, weights=weights, add=None, **{})
    a.update(change)
    with pytest.raises(ValueError):
        _layer().forward(**a)
    assert not calls


def test_norm_arguments(calls):
    layer = _layer()
    for bad in ((_x(T, H + 1), None), (_x(T, H, dtype=F32), None), (_x(T, H), _x(T + 1, H)), (_x(T, H), _x(T, H, dtype=F32))):
        with pytest.raises(ValueError):
            layer.norm(*bad)
    s, rstd, dy = _x(T, H), _x(T, dtype=F32), _x(T, H)
    for bad in ((s, _x(T), dy), (s, _x(T + 1, dtype=F32), dy), (s, rstd, _x(T, H + 8)), (s, rstd, dy, _x(T - 1, H))):
        with pytest.raises(ValueError):
            layer.norm_grad(*bad)
    assert not calls
    layer.norm_grad(s, rstd, dy)
    assert calls[0][0] == "moer_rms_norm_grad"
    with pytest.raises(ValueError):
        pipeline.ExpertLayer(torch.zeros((E, 2 * I, H), dtype=BF), torch.zeros((E, H, I), dtype=BF)).norm(s)
    with pytest.raises(ValueError):
        layer.backward(pipeline.ExpertPass(s, s, s, s, *_lists()), _x(T, H + 1))


def test_8bit_blocks():
    w = torch.randn((3, 130, 200), generator=torch.Generator().manual_seed(0))
    q, s = pipeline.to_8bit_blocks(w)
    assert q.shape == w.shape and s.shape == (3, 2, 2)
    back = q.float() * s.repeat_interleave(128, 1)[:, :130].repeat_interleave(128, 2)[:, :, :200]
    # half a step of e4m3: 2^-4 of the value, and 2^-10 of a block's scale under the smallest normal
    assert ((back - w).abs() <= w.abs() * 2.0 ** -4 * 1.001 + 2.0 ** -10 * s.max()).all()
    assert (pipeline.to_8bit_blocks(torch.zeros((1, 16, 16)))[0].float() == 0).all()
