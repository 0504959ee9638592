"""ExpertLayer with more than one batch, stream or graph under way."""
import pytest

from tests.test_gpu_expert_layer import E, H, _layer, _router
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
