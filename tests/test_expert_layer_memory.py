"""Whose memory ExpertLayer's calls use and keep, on the CPU: the library's calls are replaced by a
recorder, so nothing is launched."""
import pytest

torch = pytest.importorskip("torch")
nat = pytest.importorskip("moe_expert_routing_top_gb300._native")
from tests.test_expert_layer_checks import BF, CALLS, H, T, _layer, _lists  # noqa: E402


@pytest.fixture
def calls(monkeypatch):
    seen = []
    for name in CALLS:
        monkeypatch.setattr(nat, name, lambda *a, _n=name: seen.append((_n, *a)))
    return seen


def test_a_pass_keeps_its_own_weights(calls):
    layer = _layer()
    off, order, inv, weights = _lists()
    weights.copy_(torch.rand(weights.shape))
    want = weights.clone()
    kept = layer.forward(torch.zeros((T, H), dtype=BF), off, order, inv, weights)[1]
    weights.fill_(-1)                                 # the next batch's
    assert torch.equal(kept.weights, want)
    calls.clear()
    layer.backward(kept, torch.zeros((T, H), dtype=BF))
    assert calls[0][0] == "moer_expert_combine_grad" and calls[0][1].weights == kept.weights.data_ptr()
    assert layer.forward(torch.zeros((T, H), dtype=BF), off, order, inv)[1].weights is None


def test_partial_sums_are_the_calls_own(calls):
    """Two gradients of a norm share no workspace, be they captured or not."""
    layer = _layer()
    s, rstd, dy = torch.zeros((T, H), dtype=BF), torch.zeros(T), torch.zeros((T, H), dtype=BF)
    for _ in range(2):
        layer.norm_grad(s, rstd, dy)
    (_, _, first, n, _), (_, _, second, m, _) = calls
    need = nat.moer_rms_norm_workspace_bytes(T, H)
    assert n == m == first.numel() == second.numel() == need
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel()) for t in (first, second, layer.ws))
    assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))
