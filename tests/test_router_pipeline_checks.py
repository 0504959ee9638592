"""What RoutingStats' scored calls hand to the library, and what they refuse, on the CPU: the
library's calls are replaced by a recorder, so nothing is launched."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
nat = pytest.importorskip("moe_expert_routing_top_gb300._native")
from moe_expert_routing_top_gb300 import pipeline  # noqa: E402

L, E, k, B = 2, 64, 6, 16


@pytest.fixture
def calls(monkeypatch):
    seen = []
    for name in ("moer_score_topk", "moer_score_topk_grad", "moer_expert_order", "moer_ids_signature", "moer_block_stitch",
                 "moer_affinity_load", "moer_route"):
        monkeypatch.setattr(nat, name, lambda *a, _n=name: seen.append((_n, a)))
    return seen


def _stats(max_T=0, gate=True, **opts):
    rs = pipeline.RoutingStats(E, k, L, [0], B, D=1, tau=0.1, centroids=np.zeros((1, E)), idf=np.ones((1, E)), loads=[0], live=False,
                               G=1, group_of=np.zeros((L, E)), max_T=max_T, max_nblk=max_T, max_R=4, device="cpu", stream=0)
    if gate:
        rs.set_gate(nat.make_score_opts(**opts))
    return rs


def _ids(T):
    return torch.zeros((L, T, k), dtype=torch.uint8)


BAD_LOGITS = [("f32", torch.zeros((L, 8, E), dtype=torch.bfloat16)), ("bf16", torch.zeros((L, 8, E))), ("f16", torch.zeros((L, 8, E), dtype=torch.bfloat16)),
              ("f32", torch.zeros((L, 8, E), dtype=torch.float64)), ("f32", torch.zeros((8, E))), ("f32", torch.zeros((L + 1, 8, E))),
              ("f32", torch.zeros((L - 1, 8, E))), ("f32", torch.zeros((L, 8, E - 4))), ("f32", torch.zeros((L, E, 8)).transpose(1, 2)),
              ("f32", torch.zeros((L, 8, 2 * E))[:, :, ::2]), ("f32", torch.zeros((L, 8, E), device="meta"))]


@pytest.mark.parametrize("dtype,logits", BAD_LOGITS)
def test_logits_that_do_not_fit_the_gate(calls, dtype, logits):
    rs = _stats(8, dtype=dtype)
    with pytest.raises(ValueError):
        rs.score_topk(logits)
    with pytest.raises(ValueError):
        rs.score_grad(logits, torch.zeros((L, 8, k)))
    assert not calls


@pytest.mark.parametrize("dtype,of", [("f32", torch.float32), ("bf16", torch.bfloat16), ("f16", torch.float16)])
def test_logits_that_fit(calls, dtype, of):
    rs = _stats(8, dtype=dtype)
    for x in (torch.zeros((L, 8, E), dtype=of), torch.zeros((8, L, E), dtype=of).permute(1, 0, 2), torch.zeros((L, 8, E + 8), dtype=of)[:, :, 4:E + 4]):
        rs.score_topk(x)
        name, a = calls.pop()
        assert name == "moer_score_topk" and a[2] is x and a[3:6] == (8, x.stride(1), x.stride(0))


def test_no_gate(calls):
    with pytest.raises(ValueError):
        _stats(8, gate=False).score_topk(torch.zeros((L, 8, E)))
    assert not calls


@pytest.mark.parametrize("sums", [torch.zeros((L, E), dtype=torch.float64), torch.zeros((L, E + 4)), torch.zeros((E, L)).t(), torch.zeros(E)])
def test_score_sums_that_do_not_fit(calls, sums):
    with pytest.raises(ValueError):
        _stats(8).score_topk(torch.zeros((L, 8, E)), sums)
    assert not calls


@pytest.mark.parametrize("out", [torch.zeros((L, 8, E), dtype=torch.bfloat16), torch.zeros((L, 7, E)), torch.zeros((L, E, 8)).transpose(1, 2)])
def test_gradient_buffers_that_do_not_fit(calls, out):
    with pytest.raises(ValueError):
        _stats(8).score_grad(torch.zeros((L, 8, E)), torch.zeros((L, 8, k)), out=out)
    assert not calls


def _batch(T):
    z = torch.zeros(T + 1, dtype=torch.int32)
    return pipeline.BatchDev(T=T, R=1, nblk=1, blk_tab=z, req_blk_off=z, cache_idx=None, req_cache_off=None, insert_slot=None)


def test_buffers_grow_with_the_logits(calls):
    """A batch larger than what the buffers were made for, given to score_topk itself."""
    rs = _stats(8)
    rs.score_topk(torch.zeros((L, 100, E)))
    name, a = calls.pop()
    ids, w, ws, n = a[7], a[8], a[10], a[11]
    assert ids.numel() >= L * 100 * k and w.numel() >= L * 100 * k and n >= nat.moer_score_workspace_bytes(rs.dims, 100) and ws.numel() >= n
    rs.expert_order(100)
    assert calls.pop()[1][-1 - 1] >= nat.moer_expert_order_workspace_bytes(rs.dims, 100)


def test_step_takes_the_batchs_tokens_of_padded_logits(calls):
    rs = _stats(8)
    x = torch.zeros((L, 128, E))
    rs.score_step(x, _batch(100))
    a = dict(calls)["moer_score_topk"]
    assert a[2].data_ptr() == x.data_ptr() and a[3:6] == (100, E, 128 * E)
    assert dict(calls)["moer_ids_signature"][2] == 100 and dict(calls)["moer_expert_order"][2] == 100
    calls.clear()
    with pytest.raises(ValueError):
        rs.score_step(torch.zeros((L, 99, E)), _batch(100))
    assert not calls


def test_lists_and_gradient_of_the_last_batch_only(calls):
    rs = _stats(8)
    rs.score_topk(torch.zeros((L, 8, E)))
    calls.clear()
    with pytest.raises(ValueError):
        rs.expert_order(9)      # more ids than there are
    for T in (9, 7):            # another batch's layout
        with pytest.raises(ValueError):
            rs.score_grad(torch.zeros((L, T, E)), torch.zeros((L, T, k)))
    rs.score_grad(torch.zeros((L, 8, E)), torch.zeros((L, 8, k)))
    assert calls.pop()[0] == "moer_score_topk_grad"
    rs.ensure(16, 1, 1)         # the ids went with the smaller buffer
    with pytest.raises(ValueError):
        rs.score_grad(torch.zeros((L, 8, E)), torch.zeros((L, 8, k)))
    assert not calls


GRADS = [torch.ones(()).expand(L, 8, k), torch.randn((8, L, k)).transpose(0, 1), torch.randn((L, 8, k)).to(torch.bfloat16),
         torch.randn((L, 8, k), dtype=torch.float64), torch.randn((L, 8, 2 * k))[..., ::2]]


@pytest.mark.parametrize("dw", GRADS)
def test_gradients_of_any_layout_are_laid_out(calls, dw):
    """An expanded gradient (of a sum), a transposed one, another type: the library reads fp32 rows."""
    rs = _stats(8)
    rs.score_topk(torch.zeros((L, 8, E)))
    rs.score_grad(torch.zeros((L, 8, E)), dw, torch.ones(()).expand(L, E))
    a = calls.pop()[1]
    assert a[7].dtype == torch.float32 and a[7].is_contiguous() and torch.equal(a[7], dw.float())
    assert a[8].dtype == torch.float32 and a[8].is_contiguous() and torch.equal(a[8], torch.ones((L, E)))


def test_gradients_that_fit_are_not_copied(calls):
    rs = _stats(8)
    rs.score_topk(torch.zeros((L, 8, E)))
    dw, da = torch.zeros((L, 8, k)), torch.zeros((L, E))
    rs.score_grad(torch.zeros((L, 8, E)), dw, da)
    assert calls[-1][1][7] is dw and calls[-1][1][8] is da


@pytest.mark.parametrize("dw,da", [(torch.zeros((L, 7, k)), None), (torch.zeros((L, 8, k + 1)), None), (torch.zeros((L, 8, k)), torch.zeros(E)),
                                   (torch.zeros((L, 8, k)), torch.zeros((L, E + 4))), (torch.zeros((L, 8, k), dtype=torch.int32), None),
                                   (torch.zeros((L, 8, k), device="meta"), None)])
def test_gradients_of_other_shapes(calls, dw, da):
    rs = _stats(8)
    rs.score_topk(torch.zeros((L, 8, E)))
    calls.clear()
    with pytest.raises(ValueError):
        rs.score_grad(torch.zeros((L, 8, E)), dw, da)
    assert not calls


def test_gradient_of_an_earlier_batch_by_its_ids(calls):
    rs = _stats(64)
    rs.score_topk(torch.zeros((L, 8, E)))
    ids = torch.arange(L * 8 * k, dtype=torch.uint8).view(L, 8, k)
    rs.score_topk(torch.zeros((L, 33, E)))
    rs.score_grad(torch.zeros((L, 8, E)), torch.zeros((L, 8, k)), topk=ids)
    assert calls[-1][1][6] is ids
    with pytest.raises(ValueError):
        rs.score_grad(torch.zeros((L, 8, E)), torch.zeros((L, 8, k)))
    calls.clear()
    for bad in (ids[:, :7], ids.long(), ids.expand(L, 8, k).transpose(0, 1), torch.zeros((L, 8, 2 * k), dtype=torch.uint8)[..., ::2], ids.to("meta")):
        with pytest.raises(ValueError):
            rs.score_grad(torch.zeros((L, 8, E)), torch.zeros((L, 8, k)), topk=bad)
    assert not calls


def test_bias_in_use(calls):
    """The gate's bias is the tensor `bias`: the given one where the library can take it as it is."""
    own = torch.zeros((L, E))
    rs = _stats(8)
    rs.set_gate(nat.make_score_opts(), own)
    assert rs.bias is own
    for given in (torch.arange(L * E, dtype=torch.float64).view(L, E), torch.arange(L * E).view(E, L).t(), np.ones((L, E))):
        rs.set_gate(nat.make_score_opts(), given)
        assert rs.bias.dtype == torch.float32 and rs.bias.is_contiguous() and torch.equal(rs.bias, torch.as_tensor(given, dtype=torch.float32))
        rs.bias += 1
        rs.score_topk(torch.zeros((L, 8, E)))
        assert calls[-1][1][6] is rs.bias
    for bad in (torch.zeros(E), torch.zeros((L, E + 1)), torch.zeros((E, L)), torch.zeros((L + 1, E))):
        with pytest.raises(ValueError):
            rs.set_gate(nat.make_score_opts(), bad)
