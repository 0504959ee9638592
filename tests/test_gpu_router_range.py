"""The router operators at the ends of their inputs' ranges, against oracle/router.py.

Tolerances and comparisons are those of test_gpu_router.py, whose header derives them.
"""
import numpy as np
import pytest

from tests.test_gpu_router import DT, _backward, _check_forward, _check_grad, _forward, _ids, _logits, env  # noqa: F401

pytestmark = pytest.mark.gpu


def _device(torch, x, dtype, layout="layer"):
    """Logits x on the GPU in `dtype` (rows on odd elements with layout "odd"), and their values."""
    t = torch.from_numpy(x).to(getattr(torch, DT[dtype]))
    if layout == "layer":
        return t.cuda(), t.double().numpy()
    L, T, E = x.shape
    buf = torch.full((L, T, E + 3), 7.0, dtype=t.dtype, device="cuda")
    buf[:, :, 1:E + 1] = t.cuda()
    return buf[:, :, 1:E + 1], t.double().numpy()


def _small(rs, L, T, E):
    """Logits whose sigmoids are near the smallest normal number (at -87.3365) and under it, but
    not so near that fp32 and 64 bits may see them on different sides."""
    x = rs.uniform(-104.0, -80.0, size=(L, T, E))
    x[:, 1::3][rs.random_sample(x[:, 1::3].shape) < 0.1] = -30.0   # beside larger scores,
    x[:, 2::3][rs.random_sample(x[:, 2::3].shape) < 0.5] = -np.inf  # masks,
    x[:, 4] = -95.0                                                 # and where no score is left
    x[:, 5] = -87.0
    x[np.abs(x + 87.3365) < 0.02] = -87.0
    return x


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


@pytest.mark.parametrize("E,k", [(64, 6), (100, 12), (128, 8), (256, 20)])
@pytest.mark.parametrize("layout", ["layer", "odd"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradient_of_small_scores(env, E, k, layout, renorm, dtype):
    torch, _ = env
    rs = np.random.RandomState(E)
    dev, x = _device(torch, _small(rs, 2, 70, E), dtype, layout)
    ids, dw, da = _ids(rs, 2, 70, E, k), rs.normal(size=(2, 70, k)), rs.normal(size=(2, E))
    dw[:, :3] = 0.0  # nothing comes from these rows, so nothing may go back to them
    for a in (None, da):
        got, status = _backward(env, dev, ids, dw, a, E, k, dtype, score="sigmoid", renorm=renorm, scale=8.0)
        assert status == 0
        _check_grad(got, x, ids, dw, a, dtype, score="sigmoid", renorm=renorm, scale=8.0)
        assert a is not None or (got[:, :3] == 0).all()


# A softmax does not change with a common offset: rows far from 0, or filled with one large number
@pytest.mark.parametrize("E,k", [(64, 6), (100, 12), (128, 8), (256, 8)])
@pytest.mark.parametrize("offset", [100.0, -100.0, 1e3, 1e4, 1e5, -1e9, 1e30, -3e38])
@pytest.mark.parametrize("layout", ["layer", "odd"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_of_large_logits(env, E, k, offset, layout, renorm):
    torch, _ = env
    rs = np.random.RandomState(E + 2)
    dev, x = _device(torch, rs.normal(offset, 2.0, size=(2, 70, E)).astype(np.float32), "f32", layout)
    ids, dw, da = _ids(rs, 2, 70, E, k), rs.normal(size=(2, 70, k)), rs.normal(size=(2, E))
    for a in (None, da):
        got, _ = _backward(env, dev, ids, dw, a, E, k, "f32", score="softmax", renorm=renorm)
        _check_grad(got, x, ids, dw, a, "f32", score="softmax", renorm=renorm)


# Weights at throughput sizes: the plain softmax's, whose sum over the row is formed apart from the
# chosen exponentials, and the others beside them
@pytest.mark.parametrize("E,k,n", [(64, 6, 1), (128, 8, 1), (256, 8, 8), (128, 12, 1), (160, 6, 8)])
@pytest.mark.parametrize("offset", [-100.0, 60.0, 100.0])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_weights_of_large_logits(env, E, k, n, offset, biased, dtype):
    torch, _ = env
    rs = np.random.RandomState(E + 3)
    dev, x = _device(torch, rs.normal(offset, 2.0, size=(2, 1060, E)).astype(np.float32), dtype)
    bias = rs.normal(0, 0.05, size=(2, E)) if biased else None
    for renorm in (True, False):
        for sums in (True, False):
            o = dict(score="softmax", renorm=renorm, n_group=n, top_group=max(1, n // 2), best=1)
            _check_forward(_forward(env, dev, E, k, dtype, bias=bias, sums=sums, **o), x, k, bias=bias, **o)


# Renormalised weights of scores near the smallest normal number and under it: a large scale must
# not meet 1 / sum first
@pytest.mark.parametrize("E,k", [(64, 6), (128, 8), (256, 8), (128, 12), (256, 20)])
@pytest.mark.parametrize("T", [70, 1060])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_weights_of_small_scores(env, E, k, T, biased, dtype):
    torch, _ = env
    rs = np.random.RandomState(E + 1)
    dev, x = _device(torch, _small(rs, 2, T, E), dtype)
    bias = rs.normal(0, 0.3, size=(2, E)) if biased else None
    for renorm in (True, False):
        o = dict(score="sigmoid", renorm=renorm, scale=1000.0)
        _check_forward(_forward(env, dev, E, k, dtype, bias=bias, **o), x, k, bias=bias, **o)
