"""The expert operators together, as a layer behind the router: every step of a forward and a backward
pass against the 64-bit statements on the inputs that the step had (tolerances as in
test_gpu_experts.py), other streams, captured graphs, empty batches, the example."""
import importlib.util
import os

import numpy as np
import pytest

from oracle import experts as ex
from tests.test_gpu_experts import U, _check_quant, _close, _half_step, _np, _rand

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E, k, H, I = 16, 4, 256, 136


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_routing_top_gb300 import _native as nat
    from moe_expert_routing_top_gb300 import pipeline
    return torch, nat, pipeline


def _router(pipeline, nat, T, dev="cuda"):
    rs = pipeline.RoutingStats(E, k, 2, [0], 16, D=1, tau=0.1, centroids=np.zeros((1, E)), idf=np.ones((1, E)), loads=[0], live=False, G=1,
                               group_of=np.zeros((2, E)), max_T=T)
    rs.set_gate(nat.make_score_opts())
    return rs


def _lists(torch, nat, pipeline, T, align, seed=0):
    """One layer's lists and weights, by the router (experts of uneven popularity, one without rows)."""
    rs = _router(pipeline, nat, T)
    x = torch.randn((2, T, E), generator=torch.Generator().manual_seed(seed)) + torch.linspace(-2, 2, E)
    x[..., 3] = -float("inf")
    rs.score_topk(x.cuda())
    off, order, inv = rs.expert_order(T, align)
    assert rs.status() == 0
    return off[1], order[1], inv[1], rs.weights_for(T)[1].clone()


def _layer(torch, pipeline, dtype, **more):
    w1, w2 = _rand(torch, (E, 2 * I, H), dtype, 11, H ** -0.5), _rand(torch, (E, H, I), dtype, 12, I ** -0.5)
    return pipeline.ExpertLayer(w1, w2, norm_weight=_rand(torch, (H,), dtype, 13), **more)


class _Recorded:
    """A layer whose products are written down."""

    def __init__(self, layer):
        self.seen, inner = [], layer._gemm

        def gemm(op, out, **v):
            inner(op, out, **v)
            self.seen.append((op, v, out))
            return out
        layer._gemm = gemm


def _check_gemm(torch, dtype, op, v, out, used):
    off, order = v["expert_off"].cpu().numpy(), v.get("order")
    order = None if order is None else order.cpu().numpy()
    kk = v.get("k", 1)
    x = _np(v["x"])
    if op == "grad_weight":
        ref, mag = ex.gemm_weight_grad(_np(v["d_y"])[:used], x if order is not None else x[:used], off, None if order is None else order[:used], kk)
        _close(out, ref, (max(off[1:] - off[:-1]) + 1) * 2 * U * mag + _half_step(torch, "f32", ref), op)
        return
    w = _np(v["w"])
    if op == "grad_input":
        w = w.transpose(0, 2, 1)
    ref, mag = ex.gemm_rows(x if order is not None else x[:used], w, off, None if order is None else order[:used], kk)
    _close(out[:used], ref, w.shape[2] * 2 * U * mag + _half_step(torch, dtype, ref), op)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,align", [(150, 1), (33, 16), (1, 128), (700, 128)])
def test_forward_and_backward(env, dtype, T, align):
    torch, nat, pipeline = env
    off, order, inv, weights = _lists(torch, nat, pipeline, T, align)
    layer = _layer(torch, pipeline, dtype)
    rec = _Recorded(layer)
    hidden, x0 = _rand(torch, (T, H), dtype, 1, 2.0), _rand(torch, (T, H), dtype, 2)
    y, s, rstd = layer.norm(x0, hidden)
    assert torch.equal(s, (x0.float() + hidden.float()).to(x0.dtype))
    out, kept = layer.forward(y, off, order, inv, weights, add=s)
    used, iv, wv = int(off[-1]), inv.cpu().numpy(), _np(weights)
    for op, v, o in rec.seen:
        _check_gemm(torch, dtype, op, v, o, used)
    hv, av, zv = _np(kept.h[:used]), _np(kept.a[:used]), _np(kept.z[:used])
    ref = ex.silu_gate(hv)
    _close(av, ref, (24 + 2.4 * np.abs(hv[:, :I])) * U * np.abs(ref) + _half_step(torch, dtype, ref) + 2.0 ** -120, "activation")
    ref, mag = ex.combine(zv, iv, wv, _np(s))
    _close(out, ref, (k + 2) * 2 * U * mag + _half_step(torch, dtype, ref), "out")
    # backward
    rec.seen.clear()
    d_out = _rand(torch, (T, H), dtype, 3)
    g = layer.backward(kept, d_out)
    for op, v, o in rec.seen:
        _check_gemm(torch, dtype, op, v, o, used)
    (_, v2, d_a), (_, _, d_w2), (_, v1, d_w1), (_, _, d_rows) = rec.seen
    dz, dw, mw = ex.combine_grad(zv, iv, wv, _np(d_out), used)
    _close(v2["x"][:used], dz, U * np.abs(dz) + _half_step(torch, dtype, dz), "d_z")
    _close(g["weights"], dw, (H + 2) * 2 * U * mw, "d_weights")
    dav = _np(d_a[:used])
    ref = ex.silu_gate_grad(hv, dav)
    a, b = hv[:, :I], hv[:, I:]
    sg, big = ex.sigmoid(a), (32 + 4.8 * np.abs(a)) * U
    mag = np.concatenate([np.abs(dav * b) * sg * (1 + 2 * np.abs(a)), np.abs(dav * a) * sg], 1)
    _close(v1["d_y"][:used], ref, np.concatenate([big, big], 1) * mag + _half_step(torch, dtype, ref) + 2.0 ** -120, "d_h")
    assert g["w1"] is d_w1 and g["w2"] is d_w2
    ref, mag = ex.combine(_np(d_rows[:used]), iv)
    _close(g["x"], ref, (k + 2) * 2 * U * mag + _half_step(torch, dtype, ref), "d_x")
    d_x, d_g = layer.norm_grad(s, rstd, g["x"], d_out)
    rx, mx, rw, mw = ex.rms_norm_grad(_np(s), _np(layer.norm_weight), _np(rstd), _np(g["x"]), _np(d_out))
    _close(d_x, rx, (H + 24) * 2 * U * mx + _half_step(torch, dtype, rx), "norm d_x")
    _close(d_g, rw, (T + 16) * 2 * U * mw, "norm d_weight")
    assert layer.status() == 0


@pytest.mark.parametrize("T,align", [(150, 1), (40, 128)])
def test_8bit_layer(env, T, align):
    torch, nat, pipeline = env
    h8, i8 = 256, 144
    off, order, inv, weights = _lists(torch, nat, pipeline, T, align)
    w1, s1 = pipeline.to_8bit_blocks(_rand(torch, (E, 2 * i8, h8), "bf16", 11, h8 ** -0.5))
    w2, s2 = pipeline.to_8bit_blocks(_rand(torch, (E, h8, i8), "bf16", 12, i8 ** -0.5))
    layer = pipeline.ExpertLayer(w1, w2, scales=(s1, s2), norm_weight=_rand(torch, (h8,), "bf16", 13))
    rec = _Recorded(layer)
    (q, sc, y), s, rstd = layer.norm(_rand(torch, (T, h8), "bf16", 1))
    yy, _ = ex.rms_norm(_np(s), _np(layer.norm_weight), 1e-6)
    _close(y, yy, (h8 + 24) * U * np.abs(yy) + _half_step(torch, "bf16", yy), "y")
    _check_quant(torch, q, sc, yy, (h8 + 24) * U)
    out, kept = layer.forward((q, sc), off, order, inv, weights, add=s)
    assert kept is None and layer.status() == 0
    used, offn = int(off[-1]), off.cpu().numpy()

    def wide(w, s, n, kk):
        return _np(w.float()) * np.repeat(np.repeat(_np(s), 128, 1)[:, :n], 128, 2)[:, :, :kk]
    (_, v1, h), (_, v2, z) = rec.seen
    ref, mag = ex.gemm_rows(_np(q.float()) * ex.widen(_np(sc), h8), wide(w1, s1, 2 * i8, h8), offn, order.cpu().numpy()[:used], k)
    _close(h[:used], ref, (h8 + 4) * 2 * U * mag + _half_step(torch, "bf16", ref), "h")
    hv = _np(h[:used])
    ref = ex.silu_gate(hv)
    rel = ((24 + 2.4 * np.abs(hv[:, :i8])) * U).max()
    _check_quant(torch, v2["x"][:used], v2["x_scale"][:used], ref, rel)
    ref, mag = ex.gemm_rows(_np(v2["x"][:used].float()) * ex.widen(_np(v2["x_scale"][:used]), i8), wide(w2, s2, h8, i8), offn)
    _close(z[:used], ref, (i8 + 4) * 2 * U * mag + _half_step(torch, "bf16", ref), "z")
    ref, mag = ex.combine(_np(z[:used]), inv.cpu().numpy(), _np(weights), _np(s))
    _close(out, ref, (k + 2) * 2 * U * mag + _half_step(torch, "bf16", ref), "out")


def test_no_tokens(env):
    torch, nat, pipeline = env
    layer = _layer(torch, pipeline, "bf16")
    z = dict(device="cuda")
    out, kept = layer.forward(torch.empty((0, H), dtype=torch.bfloat16, **z), torch.zeros(E + 1, dtype=torch.int32, **z),
                              torch.empty(0, dtype=torch.int32, **z), torch.empty((0, k), dtype=torch.int32, **z), torch.empty((0, k), **z))
    g = layer.backward(kept, torch.empty((0, H), dtype=torch.bfloat16, **z))
    assert out.shape == (0, H) and (g["w1"] == 0).all() and (g["w2"] == 0).all() and g["x"].shape == (0, H) and layer.status() == 0


def test_another_stream(env):
    torch, nat, pipeline = env
    T = 300
    off, order, inv, weights = _lists(torch, nat, pipeline, T, 16)
    layer = _layer(torch, pipeline, "bf16")
    x, d = _rand(torch, (T, H), "bf16", 1), _rand(torch, (T, H), "bf16", 2)
    out, kept = layer.forward(x, off, order, inv, weights)
    g = layer.backward(kept, d)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = _layer(torch, pipeline, "bf16", stream=side)
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        out2, kept2 = other.forward(x, off, order, inv, weights)
        g2 = other.backward(kept2, d)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, out2) and all(torch.equal(g[n], g2[n]) for n in g)
        side.wait_stream(torch.cuda.current_stream())
    assert other.status() == 0


def test_captured(env):
    """A step with its gradients, captured once and replayed on other inputs, lists and weights."""
    torch, nat, pipeline = env
    T = 200
    side = torch.cuda.Stream()
    rows = T * k + E * 15
    b = [torch.empty_like(t) for t in _lists(torch, nat, pipeline, T, 16)]
    x, d = torch.empty((T, H), dtype=torch.bfloat16, device="cuda"), torch.empty((T, H), dtype=torch.bfloat16, device="cuda")

    def fill(seed):
        for t, v in zip(b, _lists(torch, nat, pipeline, T, 16, seed)):
            t.copy_(v)
        x.copy_(_rand(torch, (T, H), "bf16", seed))
        d.copy_(_rand(torch, (T, H), "bf16", seed + 1))
        torch.cuda.synchronize()
    fill(1)
    layer = _layer(torch, pipeline, "bf16", stream=side)
    graphs = []
    for _ in range(2):   # two graphs of one layer share its workspace
        layer.backward(layer.forward(x, *b)[1], d)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out, kept = layer.forward(x, *b)
            g = layer.backward(kept, d)
        graphs.append((graph, out, g))
    for seed in (5, 9):
        fill(seed)
        want, kept = layer.forward(x, *b)
        wg = layer.backward(kept, d)
        torch.cuda.synchronize()
        for graph, out, g in graphs:
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want) and all(torch.equal(g[n], wg[n]) for n in g)
    assert layer.status() == 0 and rows >= b[1].shape[0]


def test_example(env):
    torch, _, _ = env
    spec = importlib.util.spec_from_file_location("scored_router", os.path.join(ROOT, "examples", "scored_router.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    out = m.main(R=12)
    st, layer, kept = out["stats"], out["experts"], out["kept"]
    T = out["batch"].T
    assert layer.status() == 0 and torch.isfinite(out["out"]).all()
    ids, w = st.topk_for(T)[0].cpu().numpy(), _np(out["weights"])
    # each token's experts one by one, from the same rows
    x, w1, w2 = _np(kept.x), _np(layer.w1), _np(layer.w2)
    for t in (0, T // 2, T - 1):
        y = sum(w[t, j] * (w2[e] @ ex.silu_gate((w1[e] @ x[t])[None])[0]) for j, e in enumerate(ids[t]))
        got = _np(out["out"][t]) - _np(out["hidden"][t])
        # roundings of h, a, z and out to bf16: four half steps of 2^-8, twice that where terms cancel
        assert np.linalg.norm(got - y) <= 8 * 2.0 ** -8 * (np.linalg.norm(y) + np.linalg.norm(_np(out["hidden"][t])))
