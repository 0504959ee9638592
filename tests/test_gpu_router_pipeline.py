"""The pipeline's scored path over several batches, streams and layouts."""
import numpy as np
import pytest

from oracle import router

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_routing_top_gb300 import _native as nat
    from moe_expert_routing_top_gb300 import pipeline
    return torch, nat, pipeline


def _stats(pipeline, nat, L, E, k, max_T=0, stream=None, **gate):
    rs = pipeline.RoutingStats(E, k, L, [0], 16, D=1, tau=0.1, centroids=np.zeros((1, E)), idf=np.ones((1, E)), loads=[0], live=False,
                               G=1, group_of=np.zeros((L, E)), max_T=max_T, max_nblk=max_T, max_R=8, stream=stream)
    rs.set_gate(nat.make_score_opts(**gate))
    return rs


def _check(rs, x, T, k, **o):
    ids, w, _, _ = router.score_topk(x, k, **o)
    assert np.array_equal(rs.topk_for(T).cpu().numpy(), ids)
    assert np.allclose(rs.weights_for(T).cpu().numpy(), w, rtol=4e-6, atol=0)


@pytest.mark.parametrize("L,E,k,most,then", [(48, 128, 8, 1000, (1000, 809, 1000, 17)), (26, 256, 8, 1500, (1497, 1496, 900))])
def test_smaller_batches_after_a_large_one(env, L, E, k, most, then):
    torch, nat, pipeline = env
    rs = _stats(pipeline, nat, L, E, k, max_T=most)
    for T in then:
        x = torch.randn((L, T, E), device="cuda")
        sums = torch.empty((L, E), device="cuda")
        rs.score_topk(x, sums)
        assert rs.status() == 0
        p = torch.softmax(x.double(), -1).sum(1)
        assert ((sums - p).abs() <= 6e-6 * p).all()
