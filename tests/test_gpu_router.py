"""The router operators on the GPU against their 64-bit statements (oracle/router.py).

Tolerances.  A score in fp32: exp's argument x - m carries |x - m| 2^-24, so the exponential
is off by |x - m| 6e-8 relative (2e-6 at 32), plus a few units in the last place for exp, sum
and division (5e-7): 4e-6 relative.  Sums of positive scores keep that bound, and adding
fp32 terms in a tree of depth d adds d 6e-8.  A gradient adds a few such products, so it is held to
1e-5 of the sum of its terms' sizes, which the oracle gives beside it; a value stored in 16 bits
has to lie between the two ends of that range rounded to its type.  Ids are equal, except where the 64-bit choice
scores are closer than 1e-5 of the fp32 ones' size: there the chosen scores must agree to it.
"""
import numpy as np
import pytest

from oracle import router

pytestmark = pytest.mark.gpu

DT = {"f32": "float32", "bf16": "bfloat16", "f16": "float16"}


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_routing_top_gb300 import _native as nat
    return torch, nat


def _logits(torch, rs, L, T, E, dtype, layout="layer", std=2.0, special=None):
    x = rs.normal(0.0, std, size=(L, T, E))
    if special == "masks":
        x[rs.random_sample(x.shape) < 0.3] = -np.inf
        x[rs.random_sample(x.shape) < 0.05] = np.nan
        if T > 2:
            x[:, 1] = -np.inf            # a row that the mask leaves empty
            x[:, 2, 1:] = -np.inf        # and one with a single expert
    elif special == "ties":
        x = np.round(x)
        x[rs.random_sample(x.shape) < 0.1] = -0.0
    elif special == "inf":
        x[rs.random_sample(x.shape) < 0.05] = np.inf
    elif special == "lowest":
        x[rs.random_sample(x.shape) < 0.4] = {"f32": -3.4028235e38, "bf16": -3.3895314e38, "f16": -65504.0}[dtype]
    t = torch.from_numpy(x).to(getattr(torch, DT[dtype]))
    pad = 0
    if layout == "token":
        dev = t.permute(1, 0, 2).contiguous().cuda().permute(1, 0, 2)
    elif layout == "odd":                # rows that start on odd elements
        pad = 3
        buf = torch.full((L, T, E + pad), 7.0, dtype=t.dtype, device="cuda")
        buf[:, :, 1:E + 1] = t.cuda()
        dev = buf[:, :, 1:E + 1]
    else:
        dev = t.contiguous().cuda()
    return dev, t.double().numpy()


def _forward(env, dev, E, k, dtype, bias=None, sums=True, weights=True, stream=None, **o):
    torch, nat = env
    L, T = dev.shape[:2]
    d = nat.make_dims(E, k, L, [], 16)
    names = {"score": "score", "renorm": "renorm", "n_group": "n_group", "top_group": "top_group", "best": "group_best",
             "scale": "scale"}
    opts = nat.make_score_opts(dtype=dtype, **{names[n]: v for n, v in o.items()})
    ids = torch.full((L, T, k), 255, dtype=torch.uint8, device="cuda")
    w = torch.full((L, T, k), -7.0, device="cuda") if weights else None
    ss = torch.full((L, E), -7.0, device="cuda") if sums else None
    b = None if bias is None else torch.from_numpy(np.asarray(bias, dtype=np.float32)).cuda()
    n = nat.moer_score_workspace_bytes(d, T)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    nat.moer_score_topk(d, opts, dev, T, dev.stride(1), dev.stride(0), b, ids, w, ss, ws, n, stream)
    assert nat.moer_ws_status(ws, stream) == 0
    return (ids.cpu().numpy().astype(np.int64), None if w is None else w.double().cpu().numpy(),
            None if ss is None else ss.double().cpu().numpy())


def _check_forward(got, x, k, bias=None, **o):
    ids, w, ss = got
    b32 = None if bias is None else np.asarray(bias, dtype=np.float32)
    ref, rw, rs_, gap = router.score_topk(x, k, bias=b32, **o)
    c = router.scores(x, o.get("score", "softmax")) + (0 if bias is None else b32[:, None, :])
    tol = 1e-5 * (1 + (0 if bias is None else np.abs(b32[np.isfinite(b32)]).max(initial=0.0)))
    settled = gap > tol
    assert settled.mean() > 0.9
    assert np.array_equal(ids[settled], ref[settled])
    for l, t in zip(*np.nonzero(~settled)):
        assert len(set(ids[l, t])) == k
        if o.get("n_group", 1) == 1:
            assert np.allclose(c[l, t][ids[l, t]], c[l, t][ref[l, t]], atol=tol, equal_nan=True)
    if w is not None:
        want, have = rw[settled], w[settled]
        lim = 4e-6 * np.abs(want) + 1e-30
        if o.get("score", "softmax") == "sigmoid":
            lim = lim + 2.4e-38 * abs(o.get("scale", 1.0))  # scores under the normal range are 0
        assert np.isfinite(have).all() and (np.abs(have - want) <= lim).all()
    if ss is not None:
        assert (np.abs(ss - rs_) <= 6e-6 * rs_ + 1e-30).all()


CASES = [
    # L, T, E, k
    (1, 1, 128, 8), (2, 3, 64, 6), (1, 33, 128, 8), (3, 65, 256, 8), (2, 257, 128, 6), (1, 40, 4, 1), (1, 40, 4, 4),
    (1, 31, 60, 5), (2, 50, 100, 32), (1, 70, 256, 32), (1, 64, 160, 10), (1, 100, 8, 8), (1, 300, 36, 7), (2, 130, 192, 4),
]


@pytest.mark.parametrize("L,T,E,k", CASES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_plain_gate(env, L, T, E, k, dtype, score, renorm):
    torch, _ = env
    rs = np.random.RandomState(L * 1000 + T + E + k)
    dev, x = _logits(torch, rs, L, T, E, dtype)
    _check_forward(_forward(env, dev, E, k, dtype, score=score, renorm=renorm, scale=2.5), x, k, score=score, renorm=renorm,
                   scale=2.5)


@pytest.mark.parametrize("L,T,E,k,n,keep", [(1, 33, 256, 8, 8, 4), (2, 65, 128, 8, 4, 2), (1, 20, 60, 5, 4, 2),
                                            (1, 50, 64, 6, 8, 3), (1, 9, 64, 2, 32, 1), (1, 40, 256, 8, 4, 4), (2, 37, 96, 4, 3, 2),
                                            (1, 129, 256, 6, 16, 5)])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_groups_and_bias(env, L, T, E, k, n, keep, best, score, biased, dtype):
    torch, _ = env
    rs = np.random.RandomState(T + E + n)
    dev, x = _logits(torch, rs, L, T, E, dtype)
    bias = rs.normal(0, 0.05, size=(L, E)) if biased else None
    o = dict(score=score, renorm=True, n_group=n, top_group=keep, best=best, scale=1.5)
    _check_forward(_forward(env, dev, E, k, dtype, bias=bias, **o), x, k, bias=bias, **o)


@pytest.mark.parametrize("special", ["masks", "ties", "inf", "lowest"])
@pytest.mark.parametrize("E,k", [(64, 6), (128, 8), (256, 8), (60, 5), (256, 20)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_special_values(env, special, E, k, score, biased, dtype):
    torch, _ = env
    rs = np.random.RandomState(E + k)
    dev, x = _logits(torch, rs, 2, 70, E, dtype, special=special)
    bias = rs.normal(0, 0.5, size=(2, E)) if biased else None
    for renorm in (True, False):
        o = dict(score=score, renorm=renorm)
        _check_forward(_forward(env, dev, E, k, dtype, bias=bias, **o), x, k, bias=bias, **o)


def test_masked_groups(env):
    torch, _ = env
    rs = np.random.RandomState(5)
    dev, x = _logits(torch, rs, 1, 64, 64, "f32", special="masks")
    for best in (1, 2):
        for bias in (None, rs.normal(0, 0.1, size=(1, 64))):
            o = dict(score="sigmoid", n_group=8, top_group=4, best=best)
            _check_forward(_forward(env, dev, 64, 8, "f32", bias=bias, **o), x, 8, bias=bias, **o)


def test_infinite_bias(env):
    """-inf keeps an expert out (its weight stays its score's), +inf puts it first, NaN is below both."""
    torch, _ = env
    rs = np.random.RandomState(6)
    dev, x = _logits(torch, rs, 1, 40, 64, "f32")
    bias = rs.normal(0, 0.1, size=(1, 64))
    bias[0, 3], bias[0, 7], bias[0, 9] = -np.inf, np.inf, np.nan
    ids, w, _ = _forward(env, dev, 64, 6, "f32", bias=bias, score="sigmoid")
    assert (ids[0, :, 0] == 7).all() and not np.isin(ids, (3, 9)).any()
    _check_forward((ids, w, None), x, 6, bias=bias, score="sigmoid")


@pytest.mark.parametrize("layout", ["token", "odd"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E,k", [(64, 6), (128, 8), (256, 8), (100, 5)])
def test_layouts(env, layout, dtype, E, k):
    torch, _ = env
    rs = np.random.RandomState(9)
    dev, x = _logits(torch, rs, 3, 77, E, dtype, layout=layout)
    _check_forward(_forward(env, dev, E, k, dtype, renorm=False), x, k, renorm=False)
    bias = rs.normal(0, 0.1, size=(3, E))
    _check_forward(_forward(env, dev, E, k, dtype, bias=bias, score="sigmoid"), x, k, bias=bias, score="sigmoid")


def test_large_logits(env):
    """Logits of +-80 and more: scores under the normal range round to 0, none is NaN."""
    torch, _ = env
    rs = np.random.RandomState(10)
    dev, x = _logits(torch, rs, 1, 200, 128, "f32", std=60.0)
    for score in ("softmax", "sigmoid"):
        ids, w, ss = _forward(env, dev, 128, 8, "f32", score=score, renorm=False)
        ref, rw, rss, _ = router.score_topk(x, 8, score, False)
        assert np.array_equal(ids, ref)
        # x - m up to 400: the exponent's argument carries 400 * 2^-24 = 2.4e-5
        assert (np.abs(w - rw) <= 3e-5 * rw + 2.4e-38).all() and np.isfinite(ss).all()


def test_many_rows_against_the_logits_pass(env):
    """Without bias or groups the ids are those of moer_topk_signature, at sizes that fill the GPU."""
    torch, nat = env
    for E, k, L, T in ((128, 8, 3, 40001), (64, 6, 2, 30007), (256, 8, 2, 20011)):
        g = torch.Generator(device="cuda")
        g.manual_seed(E)
        x = torch.randn((L, T, E), device="cuda", generator=g)
        x[:, ::7] = x[:, ::7].round()
        d = nat.make_dims(E, k, L, [], 16)
        ref = torch.empty((L, T, k), dtype=torch.uint8, device="cuda")
        n = nat.moer_workspace_bytes(d, T, 0, 0, 0)
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        nat.moer_topk_signature(d, x, T, None, 0, ref, None, None, ws, n)
        ids, w, ss = _forward(env, x, E, k, "f32")
        assert np.array_equal(ids, ref.cpu().numpy())
        q = torch.softmax(x.double(), -1).gather(-1, ref.long())
        q = (q / q.sum(-1, keepdim=True)).cpu().numpy()
        assert (np.abs(w - q) <= 4e-6 * q).all()
        p = torch.softmax(x.double(), -1).sum(1).cpu().numpy()
        assert (np.abs(ss - p) <= 1e-5 * p).all()


# Sizes at which the throughput kernel runs (4,096 rows and more), with a ragged last tile
@pytest.mark.parametrize("E,k", [(16, 3), (24, 8), (32, 8), (60, 5), (64, 6), (72, 4), (96, 8), (128, 8), (128, 1), (160, 7), (192, 8),
                                 (256, 8), (256, 2)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True)])
def test_throughput_sizes(env, E, k, dtype, score, renorm):
    torch, _ = env
    rs = np.random.RandomState(E + k)
    dev, x = _logits(torch, rs, 2, 2051, E, dtype)
    for biased in (False, True):
        bias = rs.normal(0, 0.05, size=(2, E)) if biased else None
        o = dict(score=score, renorm=renorm, scale=2.5)
        _check_forward(_forward(env, dev, E, k, dtype, bias=bias, **o), x, k, bias=bias, **o)


@pytest.mark.parametrize("E,k,n,keep", [(256, 8, 8, 4), (128, 8, 8, 3), (128, 6, 4, 2), (64, 4, 8, 2), (64, 6, 2, 1), (256, 8, 4, 3), (160, 4, 5, 2),
                                        (32, 2, 4, 1)])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_throughput_groups(env, E, k, n, keep, best, score, dtype):
    torch, _ = env
    rs = np.random.RandomState(E + n)
    dev, x = _logits(torch, rs, 1, 4100, E, dtype)
    for biased in (False, True):
        bias = rs.normal(0, 0.05, size=(1, E)) if biased else None
        o = dict(score=score, renorm=True, n_group=n, top_group=keep, best=best)
        _check_forward(_forward(env, dev, E, k, dtype, bias=bias, sums=biased, **o), x, k, bias=bias, **o)


# groups of quads that are no whole blocks of the throughput kernel's lanes
@pytest.mark.parametrize("E,k,n,keep", [(160, 6, 8, 3), (96, 8, 8, 4), (96, 5, 4, 2), (192, 8, 8, 4), (192, 4, 2, 1), (192, 8, 4, 3), (32, 8, 8, 4),
                                        (16, 2, 4, 2), (252, 8, 7, 3), (60, 4, 3, 2)])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_throughput_odd_groups(env, E, k, n, keep, best, score, dtype):
    torch, _ = env
    rs = np.random.RandomState(E + n + 1)
    for special in (None, "masks"):
        dev, x = _logits(torch, rs, 2, 1060, E, dtype, special=special)
        for biased in (False, True):
            bias = rs.normal(0, 0.05, size=(2, E)) if biased else None
            o = dict(score=score, renorm=not biased, n_group=n, top_group=keep, best=best)
            _check_forward(_forward(env, dev, E, k, dtype, bias=bias, sums=biased, **o), x, k, bias=bias, **o)


@pytest.mark.parametrize("special", ["masks", "ties", "inf", "lowest"])
@pytest.mark.parametrize("E,k,n", [(64, 6, 1), (128, 8, 8), (256, 8, 8), (60, 5, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_throughput_special_values(env, special, E, k, n, score, dtype):
    torch, _ = env
    rs = np.random.RandomState(E + k + 1)
    dev, x = _logits(torch, rs, 2, 2100, E, dtype, special=special)
    for biased in (False, True):
        bias = rs.normal(0, 0.5, size=(2, E)) if biased else None
        o = dict(score=score, renorm=biased, n_group=n, top_group=max(1, n // 2), best=1 + (biased and n > 1))
        _check_forward(_forward(env, dev, E, k, dtype, bias=bias, **o), x, k, bias=bias, **o)


@pytest.mark.parametrize("layout", ["token", "odd"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_throughput_layouts(env, layout, dtype):
    torch, _ = env
    rs = np.random.RandomState(12)
    for E, k in ((64, 6), (100, 7), (256, 8)):
        dev, x = _logits(torch, rs, 3, 1500, E, dtype, layout=layout)
        bias = rs.normal(0, 0.05, size=(3, E))
        _check_forward(_forward(env, dev, E, k, dtype, bias=bias, score="sigmoid"), x, k, bias=bias, score="sigmoid")


def test_offsets_past_32_bits(env):
    """More than 2^31 logits: the first and the last rows' choices, weights and gradients."""
    torch, nat = env
    E, k, T = 128, 8, (1 << 24) + 4099
    x = torch.zeros((1, T, E), dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    ends = torch.cat([torch.arange(2000), torch.arange(T - 2000, T)]).cuda()
    x[0, ends] = torch.randn((4000, E), device="cuda", generator=gen).to(x.dtype)
    d, o = nat.make_dims(E, k, 1, [], 16), nat.make_score_opts(dtype="bf16")
    ids = torch.empty((1, T, k), dtype=torch.uint8, device="cuda")
    w = torch.empty((1, T, k), device="cuda")
    n = nat.moer_score_workspace_bytes(d, T)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    nat.moer_score_topk(d, o, x, T, E, T * E, None, ids, w, None, ws, n)
    ref, rw, _, _ = router.score_topk(x[:, ends].double().cpu().numpy(), k)
    assert np.array_equal(ids[:, ends].cpu().numpy(), ref)
    assert (np.abs(w[:, ends].double().cpu().numpy() - rw) <= 4e-6 * rw).all()
    assert (ids[0, T // 2] == torch.arange(k, device="cuda")).all()       # a row of ties
    w.normal_(generator=gen)
    dx = torch.empty_like(x)
    nat.moer_score_topk_grad(d, o, x, T, E, T * E, ids, w, None, dx, E, T * E, ws, n)
    assert nat.moer_ws_status(ws) == 0
    _check_grad(dx[:, ends].double().cpu().numpy(), x[:, ends].double().cpu().numpy(), ref, w[:, ends].cpu().numpy(), None, "bf16")


def test_same_bits_twice_and_on_another_stream(env):
    torch, _ = env
    rs = np.random.RandomState(11)
    dev, _ = _logits(torch, rs, 2, 5003, 128, "bf16")
    torch.cuda.synchronize()
    a = _forward(env, dev, 128, 8, "bf16", renorm=False)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = _forward(env, dev, 128, 8, "bf16", renorm=False, stream=side)
    side.synchronize()
    assert all(np.array_equal(u, v) for u, v in zip(a, b))


def test_no_tokens(env):
    torch, nat = env
    d = nat.make_dims(64, 6, 2, [], 16)
    ss = torch.full((2, 64), 3.0, device="cuda")
    nat.moer_score_topk(d, nat.make_score_opts(), None, 0, 64, 64, None, None, None, ss, None, 0)
    assert (ss.cpu() == 0).all()


# ------------------------------------------------------------------ the gradient
def _backward(env, dev, ids, dw, da, E, k, dtype, inplace=False, **o):
    torch, nat = env
    L, T = dev.shape[:2]
    d = nat.make_dims(E, k, L, [], 16)
    opts = nat.make_score_opts(dtype=dtype, **o)
    out = dev if inplace else torch.full_like(dev, 9.0)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    nat.moer_score_topk_grad(d, opts, dev, T, dev.stride(1), dev.stride(0), torch.from_numpy(ids.astype(np.uint8)).cuda(),
                             torch.from_numpy(dw.astype(np.float32)).cuda(),
                             None if da is None else torch.from_numpy(da.astype(np.float32)).cuda(), out, out.stride(1),
                             out.stride(0), ws, 256)
    return out.double().cpu().numpy(), nat.moer_ws_status(ws)


def _ids(rs, L, T, E, k):
    return np.argsort(rs.random_sample((L, T, E)), axis=-1)[..., :k]


def _check_grad(got, x, ids, dw, da, dtype, **o):
    dx, mag = router.score_topk_grad(x, ids, dw.astype(np.float32), None if da is None else da.astype(np.float32), **o)
    import torch
    lim = 1e-5 * mag + 1e-37
    lo, hi = (torch.from_numpy(v).to(getattr(torch, DT[dtype])).double().numpy() for v in (dx - lim, dx + lim))
    assert np.isfinite(got).all()
    bad = (got < lo) | (got > hi)
    assert not bad.any(), (int(bad.sum()), got[bad][:5], lo[bad][:5], hi[bad][:5])


@pytest.mark.parametrize("L,T,E,k", CASES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("sums", [True, False])
def test_gradient(env, L, T, E, k, dtype, score, renorm, sums):
    torch, _ = env
    rs = np.random.RandomState(T + E + k)
    dev, x = _logits(torch, rs, L, T, E, dtype)
    ids, dw, da = _ids(rs, L, T, E, k), rs.normal(size=(L, T, k)), rs.normal(size=(L, E)) if sums else None
    got, status = _backward(env, dev, ids, dw, da, E, k, dtype, score=score, renorm=renorm, scale=1.5)
    assert status == 0
    _check_grad(got, x, ids, dw, da, dtype, score=score, renorm=renorm, scale=1.5)


@pytest.mark.parametrize("special", ["masks", "inf", "lowest"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,k", [(128, 8), (60, 5), (256, 8)])
def test_gradient_special_values(env, special, score, renorm, E, k):
    torch, _ = env
    rs = np.random.RandomState(21)
    dev, x = _logits(torch, rs, 2, 70, E, "f32", special=special)
    ids, dw, da = _ids(rs, 2, 70, E, k), rs.normal(size=(2, 70, k)), rs.normal(size=(2, E))
    got, _ = _backward(env, dev, ids, dw, da, E, k, "f32", score=score, renorm=renorm)
    _check_grad(got, x, ids, dw, da, "f32", score=score, renorm=renorm)


@pytest.mark.parametrize("layout", ["token", "odd"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("sums", [True, False])
def test_gradient_layouts(env, layout, dtype, inplace, sums):
    torch, _ = env
    rs = np.random.RandomState(22)
    dev, x = _logits(torch, rs, 3, 77, 128, dtype, layout=layout)
    ids, dw, da = _ids(rs, 3, 77, 128, 8), rs.normal(size=(3, 77, 8)), rs.normal(size=(3, 128)) if sums else None
    got, _ = _backward(env, dev, ids, dw, da, 128, 8, dtype, inplace=inplace, score="sigmoid")
    _check_grad(got, x, ids, dw, da, dtype, score="sigmoid")
    if layout == "odd" and inplace:      # what lies between the rows is left alone
        buf = dev._base
        assert (buf[:, :, 0] == 7).all() and (buf[:, :, 129:] == 7).all()


@pytest.mark.parametrize("E", [64, 100])
def test_gradient_bad_ids(env, E):
    torch, _ = env
    rs = np.random.RandomState(23)
    dev, x = _logits(torch, rs, 1, 50, E, "f32")
    ids, dw = _ids(rs, 1, 50, E, 6), rs.normal(size=(1, 50, 6))
    ids[0, 7, 2] = ids[0, 7, 0]           # repeated: counts as given
    ok = ids.copy()
    ids[0, 9, 3] = 255                    # no such expert: contributes nothing
    got, status = _backward(env, dev, ids, dw, None, E, 6, "f32", score="sigmoid", renorm=False)
    assert status == 6
    dw2 = dw.copy()
    dw2[0, 9, 3] = 0.0
    _check_grad(got, x, ok, dw2, None, "f32", score="sigmoid", renorm=False)


# ------------------------------------------------------------------ the block plan
def _plan(env, new, ctx, B, pages=None, free=None, room=0, want=None, **over):
    torch, nat = env
    i32 = torch.int32
    R = len(new)
    ref_pages = None if pages is None else pages.copy()
    n_free = 0 if free is None else len(free)
    ref = router.block_plan(new, ctx, B, ref_pages, free) if want is None else want
    T, nb, nc = (int(v) + room for v in ref["totals"][:3])
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()  # noqa: E731
    e = lambda *s, dtype=i32: torch.full(s, 77, dtype=dtype, device="cuda")  # noqa: E731
    b = {"new_len": t(new), "ctx_len": t(ctx), "req_off": e(R + 1), "req_blk_off": e(R + 1), "blk_tab": e(nb, 2),
         "req_cache_off": e(R + 1), "tok_req": e(T), "tok_pos": e(T), "totals": e(4)}
    if pages is not None:
        b.update(pages=t(pages), insert_slot=e(nb), cache_idx=e(nc), slot_map=e(T, dtype=torch.int64))
        if free is not None:
            b["free_pages"] = t(free)
    if not any(ctx):
        b["ctx_len"] = None
    size = dict(R=R, block=B, T=T, nblk=nb, ncached=nc, n_free=n_free, ld_pages=0 if pages is None else pages.shape[1])
    size.update(over)
    a = nat.make_block_plan(**size, **b)
    n = nat.moer_block_plan_workspace_bytes(R)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    nat.moer_block_plan(a, ws, n)
    return {k: v.cpu().numpy() for k, v in b.items() if v is not None}, ref, ref_pages, nat.moer_ws_status(ws)


def _batch(rs, R, B, most_new, most_ctx, aligned=False, zeros=0.1):
    new = rs.randint(1, most_new + 1, size=R)
    new[rs.random_sample(R) < zeros] = 0
    ctx = rs.randint(0, most_ctx + 1, size=R)
    if aligned:
        ctx = ctx // B * B
    have = -(-ctx // B)
    total = -(-(ctx + new) // B)
    width = int(total.max()) + 2 if R else 1
    pool = rs.permutation(int(total.sum()) + 9)
    pages = np.full((R, width), -5)
    at = 0
    for r in range(R):
        pages[r, :have[r]] = pool[at:at + have[r]]
        at += have[r]
    return new, ctx, pages, pool[at:]


@pytest.mark.parametrize("R,B,most_new,most_ctx", [(1, 16, 1, 0), (1, 16, 40, 100), (7, 16, 1, 500), (33, 1, 5, 9),
                                                    (300, 16, 50, 200), (1025, 16, 3, 40), (2500, 255, 700, 900), (5000, 8, 1, 70),
                                                    (70, 128, 4096, 3000), (3, 7, 20000, 11)])
@pytest.mark.parametrize("room", [0, 37])
@pytest.mark.parametrize("aligned", [True, False])
def test_block_plan(env, R, B, most_new, most_ctx, room, aligned):
    rs = np.random.RandomState(R + B)
    new, ctx, pages, free = _batch(rs, R, B, most_new, most_ctx, aligned)
    got, ref, ref_pages, status = _plan(env, new, ctx, B, pages, free, room)
    assert status == 0
    assert np.array_equal(got["pages"], ref_pages)
    for name in ("req_off", "req_blk_off", "req_cache_off", "totals"):
        assert np.array_equal(got[name], ref[name]), name
    for name in ("insert_slot", "cache_idx", "slot_map", "tok_req", "tok_pos", "blk_tab"):
        n = len(ref[name])
        assert np.array_equal(got[name][:n], ref[name]), name
        rest = got[name][n:]
        if name == "blk_tab":
            assert (rest == (ref["totals"][0], 0)).all()
        else:
            assert (rest == -1).all(), name


def test_block_plan_of_many_requests(env):
    """More requests than one block's sums reach."""
    rs = np.random.RandomState(7)
    new, ctx, pages, free = _batch(rs, 70001, 4, 2, 9)
    got, ref, ref_pages, status = _plan(env, new, ctx, 4, pages, free)
    assert status == 0 and np.array_equal(got["pages"], ref_pages)
    for name in ("req_off", "req_blk_off", "req_cache_off", "totals", "insert_slot", "cache_idx", "slot_map", "tok_req",
                 "tok_pos", "blk_tab"):
        assert np.array_equal(got[name], ref[name]), name


def test_block_plan_without_pages(env):
    rs = np.random.RandomState(3)
    new, ctx, _, _ = _batch(rs, 50, 16, 30, 60)
    got, ref, _, status = _plan(env, new, ctx, 16)
    assert status == 0 and np.array_equal(got["blk_tab"], ref["blk_tab"]) and np.array_equal(got["tok_pos"], ref["tok_pos"])
    assert np.array_equal(got["totals"], ref["totals"])


def test_block_plan_no_requests(env):
    got, _, _, status = _plan(env, np.zeros(0, int), np.zeros(0, int), 16, room=5)
    assert status == 0 and got["totals"].tolist() == [0, 0, 0, 0] and (got["tok_req"] == -1).all()
    assert got["req_off"].tolist() == [0] and (got["blk_tab"] == 0).all()


def test_block_plan_slots_past_32_bits(env):
    big = 2 ** 31 - 5
    got, _, _, status = _plan(env, np.array([3]), np.array([0]), 255, np.array([[-1]]), np.array([big]),
                              want={"totals": np.array([3, 1, 0, 1])})
    assert status == 0 and got["slot_map"].tolist() == [big * 255 + i for i in range(3)]


def test_block_plan_bad_data(env):
    rs = np.random.RandomState(4)
    new, ctx, pages, free = _batch(rs, 40, 16, 30, 60, zeros=0.0)
    full, ref, _, _ = _plan(env, new, ctx, 16, pages, free)
    # a negative length counts as 0
    neg = new.copy()
    neg[5] = -3
    got, want, _, status = _plan(env, neg, ctx, 16, pages, free)
    assert status == 6 and np.array_equal(got["slot_map"], want["slot_map"])
    # free pages run out: the last ones are -1, with their slots
    short, _, _, status = _plan(env, new, ctx, 16, pages, free, n_free=int(ref["totals"][3]) - 1, want=ref)
    assert status == 6
    assert (short["slot_map"] != full["slot_map"]).any()
    bad = short["slot_map"] != full["slot_map"]
    assert (short["slot_map"][bad] == -1).all() and (full["slot_map"][bad] // 16 == free[ref["totals"][3] - 1]).all()
    # too little room for blocks or tokens: what fits is written
    got, _, _, status = _plan(env, new, ctx, 16, pages, free, want=ref, nblk=int(ref["totals"][1]) - 3)
    assert status == 6 and np.array_equal(got["blk_tab"][:-3], ref["blk_tab"][:-3]) and (got["blk_tab"][-3:] == 77).all()
    got, _, _, status = _plan(env, new, ctx, 16, pages, free, want=ref, T=int(ref["totals"][0]) - 7)
    assert status == 6 and np.array_equal(got["slot_map"][:-7], ref["slot_map"][:-7]) and (got["slot_map"][-7:] == 77).all()


# ------------------------------------------------------------------ the experts' lists
@pytest.mark.parametrize("L,T,E,k", [(1, 1, 128, 8), (2, 3, 64, 6), (1, 513, 128, 8), (3, 700, 256, 8), (2, 5000, 60, 6), (1, 9001, 4, 1),
                                     (1, 900, 100, 32), (1, 70001, 128, 8), (48, 40, 128, 8), (1, 2049, 256, 2)])
@pytest.mark.parametrize("align", [1, 16, 100])
@pytest.mark.parametrize("skew", [0.0, 3.0])
def test_expert_order(env, L, T, E, k, align, skew):
    torch, nat = env
    rs = np.random.RandomState(T + E)
    pop = rs.normal(size=(L, 1, E)) * skew
    ids = np.argsort(-(pop + rs.gumbel(size=(L, T, E))), axis=-1)[..., :k].astype(np.uint8)
    _order_case(env, ids, E, k, align)


def _order_case(env, ids, E, k, align, extra=0, status=0):
    torch, nat = env
    L, T = ids.shape[:2]
    N = T * k
    ld = N + min(E, N) * (align - 1) + extra
    d = nat.make_dims(E, k, L, [], 16)
    off = torch.full((L, E + 1), 77, dtype=torch.int32, device="cuda")
    order = torch.full((L, ld), 77, dtype=torch.int32, device="cuda")
    inv = torch.full((L, T, k), 77, dtype=torch.int32, device="cuda")
    n = nat.moer_expert_order_workspace_bytes(d, T)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    dev = torch.from_numpy(ids).cuda()
    ro, rr, ri = router.expert_order(ids, E, align, ld)
    for o, i in ((order, inv), (order, None), (None, inv), (None, None)):
        off.fill_(77), order.fill_(77), inv.fill_(77)
        nat.moer_expert_order(d, dev, T, align, off, o, ld if o is not None else 0, i, ws, n)
        assert nat.moer_ws_status(ws) == status
        assert np.array_equal(off.cpu().numpy(), ro)
        assert o is None or np.array_equal(order.cpu().numpy(), rr)
        assert i is None or np.array_equal(inv.cpu().numpy(), ri)


def test_expert_order_odd_data(env):
    rs = np.random.RandomState(8)
    ids = rs.randint(0, 64, size=(2, 3000, 6)).astype(np.uint8)    # with repeats within a token
    _order_case(env, ids, 64, 6, 16, extra=5)
    ids[1, 17, 3] = 200                                            # no such expert
    _order_case(env, ids, 64, 6, 16, extra=5, status=6)
    _order_case(env, np.full((1, 4000, 8), 3, dtype=np.uint8), 128, 8, 128)   # one expert takes all
    _order_case(env, np.zeros((2, 0, 8), dtype=np.uint8), 128, 8, 16, extra=9)


# More than eight experts to a token at the sizes of the throughput kernel
@pytest.mark.parametrize("E,k", [(16, 9), (16, 16), (24, 12), (32, 16), (60, 13), (64, 9), (64, 16), (72, 10), (100, 15), (128, 10), (128, 16),
                                 (160, 12), (192, 11), (256, 9), (256, 16)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True)])
def test_throughput_many_choices(env, E, k, dtype, score, renorm):
    torch, _ = env
    rs = np.random.RandomState(E + k)
    dev, x = _logits(torch, rs, 2, 1031, E, dtype)
    for biased in (False, True):
        bias = rs.normal(0, 0.05, size=(2, E)) if biased else None
        for sums in (False, True):
            o = dict(score=score, renorm=renorm, scale=1.5)
            _check_forward(_forward(env, dev, E, k, dtype, bias=bias, sums=sums, **o), x, k, bias=bias, **o)


# groups of whole blocks and groups of quads; as many choices as the kept groups have experts
@pytest.mark.parametrize("E,k,n,keep", [(256, 16, 8, 4), (256, 10, 8, 1), (128, 16, 8, 1), (128, 12, 4, 2), (64, 9, 8, 2), (64, 16, 2, 1),
                                        (32, 16, 4, 2), (160, 12, 5, 2), (96, 10, 8, 4), (160, 16, 8, 3)])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_throughput_many_choices_in_groups(env, E, k, n, keep, best, score, dtype):
    torch, _ = env
    rs = np.random.RandomState(E + n + k)
    dev, x = _logits(torch, rs, 1, 2100, E, dtype)
    for biased in (False, True):
        bias = rs.normal(0, 0.05, size=(1, E)) if biased else None
        o = dict(score=score, renorm=not biased, n_group=n, top_group=keep, best=best)
        _check_forward(_forward(env, dev, E, k, dtype, bias=bias, sums=biased, **o), x, k, bias=bias, **o)


@pytest.mark.parametrize("special", ["masks", "ties", "inf", "lowest"])
@pytest.mark.parametrize("E,k,n", [(64, 12, 1), (128, 16, 8), (256, 10, 8), (60, 9, 1)])
@pytest.mark.parametrize("layout", ["token", "odd"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_throughput_many_choices_special_values(env, special, E, k, n, layout, dtype):
    torch, _ = env
    rs = np.random.RandomState(E + k + 1)
    dev, x = _logits(torch, rs, 2, 1060, E, dtype, layout=layout, special=special)
    for biased in (False, True):
        bias = rs.normal(0, 0.5, size=(2, E)) if biased else None
        o = dict(score="sigmoid" if biased else "softmax", renorm=biased, n_group=n, top_group=max(1, n // 2), best=1 + (n > 1))
        ids, w, ss = _forward(env, dev, E, k, dtype, bias=bias, **o)
        # Groups tie where their logits do, and the oracle leaves those rows open: every
        # row's choice is that of the few rows' kernel, and the others are the oracle's
        few = [_forward(env, dev[:, a:a + 530], E, k, dtype, bias=bias, sums=False, **o) for a in (0, 530)]
        assert np.array_equal(ids, np.concatenate([f[0] for f in few], axis=1))
        ws = np.concatenate([f[1] for f in few], axis=1)
        assert (np.abs(w - ws) <= 8e-6 * np.abs(ws) + 4.8e-38).all()
        b32 = None if bias is None else bias.astype(np.float32)
        _, _, sums, gap = router.score_topk(x, k, bias=b32, **o)
        assert (np.abs(ss - sums) <= 6e-6 * sums + 1e-30).all()
        tol = 1e-5 * (1 + (0 if bias is None else np.abs(b32).max()))
        for l in range(2):
            at = gap[l] > tol
            _check_forward((ids[l:l + 1, at], w[l:l + 1, at], None), x[l:l + 1, at], k,
                           bias=None if bias is None else bias[l:l + 1], **o)


# Groups whose two best scores nearly add up to the same: small logits, and sigmoids near 1
@pytest.mark.parametrize("E,k,n,keep", [(256, 8, 8, 4), (128, 16, 8, 3), (64, 6, 4, 2), (160, 6, 8, 3)])
@pytest.mark.parametrize("std", [0.003, 0.1, 9.0])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_throughput_near_groups(env, E, k, n, keep, std, score, dtype):
    torch, _ = env
    rs = np.random.RandomState(E + k)
    dev, x = _logits(torch, rs, 1, 2600, E, dtype, std=std)
    o = dict(score=score, renorm=True, n_group=n, top_group=keep, best=2)
    ids, w, _ = _forward(env, dev, E, k, dtype, sums=False, **o)
    few = [_forward(env, dev[:, a:a + 1300], E, k, dtype, sums=False, **o) for a in (0, 1300)]
    assert np.array_equal(ids, np.concatenate([f[0] for f in few], axis=1))
    gap = router.score_topk(x, k, **o)[3]
    at = gap[0] > 1e-5
    _check_forward((ids[:, at], w[:, at], None), x[:, at], k, **o)


# groups that share quads of experts with their neighbours
@pytest.mark.parametrize("E,k,n,keep", [(72, 6, 4, 2), (72, 8, 4, 3), (36, 4, 6, 2), (100, 8, 4, 1), (60, 5, 4, 2), (20, 3, 4, 2), (252, 8, 4, 2),
                                        (28, 2, 4, 3), (132, 7, 3, 2), (200, 8, 8, 4), (12, 3, 4, 2), (252, 8, 2, 1)])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_throughput_shared_quads(env, E, k, n, keep, best, score, dtype):
    torch, _ = env
    rs = np.random.RandomState(E + n + 2)
    for special in (None, "masks"):
        dev, x = _logits(torch, rs, 2, 1060, E, dtype, special=special)
        for biased in (False, True):
            bias = rs.normal(0, 0.05, size=(2, E)) if biased else None
            o = dict(score=score, renorm=not biased, n_group=n, top_group=keep, best=best)
            _check_forward(_forward(env, dev, E, k, dtype, bias=bias, sums=biased, **o), x, k, bias=bias, **o)


# Runs of equal and nearly equal choice scores: rounded logits with no, equal or nearly equal biases
@pytest.mark.parametrize("E,k,n,keep", [(256, 8, 1, 1), (256, 7, 8, 4), (64, 16, 1, 1), (64, 5, 1, 1), (128, 12, 4, 2), (128, 8, 4, 2)])
@pytest.mark.parametrize("scale", [0.25, 64.0])
@pytest.mark.parametrize("spread", [0.0, 1e-6, 1e-3])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_throughput_runs(env, E, k, n, keep, scale, spread, score, dtype):
    torch, _ = env
    rs = np.random.RandomState(E + k)
    x = np.round(rs.normal(0.0, 2.0, size=(1, 2400, E)) * scale) / scale
    t = torch.from_numpy(x).to(getattr(torch, DT[dtype]))
    dev, x = t.cuda(), t.double().numpy()
    bias = rs.normal(0, 1, size=(1, E)) * spread + 0.25
    o = dict(score=score, renorm=True, n_group=n, top_group=keep, best=1)
    ids, w, _ = _forward(env, dev, E, k, dtype, bias=bias, sums=False, **o)
    b32 = bias.astype(np.float32)
    if spread == 0.0:  # the few rows' kernel breaks the ties alike
        few = [_forward(env, dev[:, a:a + 1200], E, k, dtype, bias=bias, sums=False, **o) for a in (0, 1200)]
        assert np.array_equal(ids, np.concatenate([f[0] for f in few], axis=1))
    _, _, _, gap = router.score_topk(x, k, bias=b32, **o)
    # whatever the order of scores that fp32 cannot tell apart: the choice falls off, and no
    # expert of a kept group that was passed over stands above its last one
    c = (router.scores(x, score) + b32[:, None, :])[0]
    mine = np.take_along_axis(c, ids[0], axis=1)
    assert (np.diff(mine, axis=1) <= 2e-6).all()
    taken = np.zeros(c.shape, dtype=bool)
    np.put_along_axis(taken, ids[0], True, axis=1)
    assert (taken.sum(1) == k).all()
    kept = taken.reshape(-1, n, E // n).any(2)
    assert (kept.sum(1) <= keep).all()
    over = np.where(taken | ~np.repeat(kept, E // n, axis=1), -np.inf, c).max(1)
    assert (over <= mine[:, -1] + 2e-6).all()
    at = gap[0] > 2e-5
    if at.any():
        _check_forward((ids[:, at], w[:, at], None), x[:, at], k, bias=bias, **o)
