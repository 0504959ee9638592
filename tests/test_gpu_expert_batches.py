"""ExpertLayer with more than one batch, stream or graph under way."""
import pytest

from tests.test_gpu_expert_layer import E, H, I, _layer, _lists, _router, k
from tests.test_gpu_experts import _rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_routing_top_gb300 import _native as nat
    from moe_expert_routing_top_gb300 import pipeline
    return torch, nat, pipeline


def test_two_batches_under_way(env):
    """The router's one buffer of weights, given as it is, takes the next batch's before the first one's
    backward pass."""
    torch, nat, pipeline = env
    T = 150
    rs, layer = _router(pipeline, nat, T), _layer(torch, pipeline, "bf16")
    x, d = _rand(torch, (T, H), "bf16", 1), _rand(torch, (T, H), "bf16", 2)

    def forward(seed):
        rs.score_topk(torch.randn((2, T, E), generator=torch.Generator().manual_seed(seed)).cuda())
        off, order, inv = rs.expert_order(T, 16)
        return layer.forward(x, off[1], order[1], inv[1], rs.weights_for(T)[1])[1]
    want = layer.backward(forward(1), d)
    first, second = forward(1), forward(2)
    other = layer.backward(second, d)
    got = layer.backward(first, d)
    assert layer.status() == 0 and rs.status() == 0
    assert all(torch.equal(got[n], want[n]) for n in want) and not torch.equal(other["w1"], want["w1"])


def test_backward_of_dropped_pairs(env):
    """Pairs without a row, by the lists' inverse, have the gradients of pairs of weight 0, whatever lay in
    the memory that the pass takes."""
    torch, nat, pipeline = env
    T = 150
    off, order, inv, weights = _lists(torch, nat, pipeline, T, 16)
    layer = _layer(torch, pipeline, "bf16")
    x, d = _rand(torch, (T, H), "bf16", 1), _rand(torch, (T, H), "bf16", 2)
    drop = torch.rand((T, k), generator=torch.Generator().manual_seed(3)).cuda() < 0.25
    out, kept = layer.forward(x, off, order, inv, torch.where(drop, 0.0, weights))
    want = layer.backward(kept, d)
    out2, kept2 = layer.forward(x, off, order, torch.where(drop, -1, inv), weights)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    n = order.shape[0]
    stale = [torch.full(s, float("nan"), dtype=torch.bfloat16, device="cuda") for s in ((n, H), (n, I), (n, 2 * I), (n, H)) for _ in range(2)]
    torch.cuda.synchronize()
    del stale
    got = layer.backward(kept2, d)
    assert layer.status() == 0 and torch.equal(out, out2)
    for name in ("x", "w1", "w2"):
        assert torch.equal(got[name], want[name]), name
    assert (got["weights"][drop] == 0).all() and torch.equal(got["weights"][~drop], want["weights"][~drop])


@pytest.mark.parametrize("eight", [False, True])
def test_weights_dropped_while_launches_wait(env, eight):
    """A layer on a stream of its own may go, and its weights with it, as soon as its calls are made: the
    memory is not given out again before they ran."""
    torch, nat, pipeline = env
    T, h8, i8 = 300, 256, 144
    off, order, inv, weights = _lists(torch, nat, pipeline, T, 16)
    x = _rand(torch, (T, h8), "bf16", 1)

    def layer(stream=None):
        w1, w2 = _rand(torch, (E, 2 * i8, h8), "bf16", 11, h8 ** -0.5), _rand(torch, (E, h8, i8), "bf16", 12, i8 ** -0.5)
        more = {}
        if eight:
            (w1, s1), (w2, s2) = pipeline.to_8bit_blocks(w1), pipeline.to_8bit_blocks(w2)
            more = {"scales": (s1, s2)}
        return pipeline.ExpertLayer(w1, w2, norm_weight=_rand(torch, (h8,), "bf16", 13), stream=stream, **more)

    def run(layer):
        y = layer.norm(x)[0]
        return layer.forward(y[:2] if eight else y, off, order, inv, weights)[0]
    want = run(layer())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = layer(side)
    run(other)
    shapes = [(t.shape, t.dtype) for t in (other.w1, other.w2, other.norm_weight, *(other.scales or ()))]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(500_000_000)                # a quarter of a second: the launches wait behind it
    out = run(other)
    assert not side.query()
    del other
    junk = [torch.full(s, 3.0, dtype=torch.float32, device="cuda").to(t) for s, t in shapes for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(out, want) and len(junk) == 4 * len(shapes)


def test_captured_norm_gradients_at_the_same_time(env):
    """Two graphs of one layer's norm and its gradient, on other inputs, replayed on two streams at once."""
    torch, nat, pipeline = env
    T, side = 3001, torch.cuda.Stream()
    layer = _layer(torch, pipeline, "bf16", stream=side)
    x, d = ([_rand(torch, (T, H), "bf16", s + i) for i in range(2)] for s in (1, 3))
    torch.cuda.synchronize()

    def step(i):
        y, s, rstd = layer.norm(x[i], d[i])
        return (y, s, *layer.norm_grad(s, rstd, d[i], x[i]))
    want, graphs = [], []
    for i in range(2):
        out = step(i)
        torch.cuda.synchronize()
        want.append([t.clone() for t in out])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step(i)
        graphs.append((graph, out))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(100):
        for (graph, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for (_, out), w in zip(graphs, want):
        assert all(torch.equal(a, b) for a, b in zip(out, w))
    assert layer.status() == 0


def test_norm_on_another_stream(env):
    torch, nat, pipeline = env
    T = 300
    x, r, d = (_rand(torch, (T, H), "bf16", i) for i in range(3))
    layer, side = _layer(torch, pipeline, "bf16"), torch.cuda.Stream()
    y, s, rstd = layer.norm(x, r)
    want = [y, s, rstd, *layer.norm_grad(s, rstd, d, r)]
    torch.cuda.synchronize()
    other = _layer(torch, pipeline, "bf16", stream=side)
    torch.cuda.synchronize()
    for _ in range(5):
        side.wait_stream(torch.cuda.current_stream())
        y, s, rstd = other.norm(x.clone(), r.clone())
        side.wait_stream(torch.cuda.current_stream())
        got = [y, s, rstd, *other.norm_grad(s, rstd, d, r)]
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
