"""The router operators at the ends of their inputs' ranges, against oracle/router.py.

Tolerances and comparisons are those of test_gpu_router.py, whose header derives them.
"""
import numpy as np
import pytest

from tests.test_gpu_router import _check_forward, _forward, _logits, env  # noqa: F401

pytestmark = pytest.mark.gpu


# Choice scores past the keys' range of [-1, 3) in groups ranked by their two best: the few
# rows' kernel and the throughput kernel, with whole, split and shared groups
@pytest.mark.parametrize("E,k,n", [(64, 6, 8), (128, 8, 4), (256, 8, 8), (160, 6, 8), (72, 6, 4), (128, 16, 4)])
@pytest.mark.parametrize("T", [40, 1060])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_group_sums_of_large_biases(env, E, k, n, T, score, dtype):
    torch, _ = env
    rs = np.random.RandomState(E + T)
    dev, x = _logits(torch, rs, 3, T, E, dtype)
    gs = E // n
    bias = rs.normal(0, 0.3, size=(3, E))
    for l, (at, top) in enumerate(((0, 10.0), (n - 1, np.inf), (1, 3.5))):
        bias[l, at * gs:(at + 1) * gs] -= 0.5  # one expert far above a low group's others
        bias[l, at * gs + 2] = top
        other = (at + 1) % n                   # a group that is high as a whole
        bias[l, other * gs:(other + 1) * gs] += 2.0
    o = dict(score=score, renorm=True, n_group=n, top_group=1, best=2)
    _check_forward(_forward(env, dev, E, k, dtype, bias=bias, **o), x, k, bias=bias, **o)
