"""The router operators at the ends of their inputs' ranges, against oracle/router.py.

Tolerances and comparisons are those of test_gpu_router.py, whose header derives them.
"""
import math
import time

import numpy as np
import pytest

from oracle import router
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


# Lengths that a batch cannot have: what fits is written, in a time that goes by the room
@pytest.mark.parametrize("B", [1, 16, 255])
@pytest.mark.parametrize("R,at", [(3, 0), (1000, 2), (3000, 2)])
@pytest.mark.parametrize("maps", [True, False])
def test_block_plan_of_absurd_lengths(env, B, R, at, maps):
    torch, nat = env
    rs = np.random.RandomState(B + R)
    new, ctx = rs.randint(1, 20, size=R).astype(np.int64), rs.randint(0, 30, size=R).astype(np.int64)
    ctx[at] = 2 * B + 1 if B > 1 else 2
    new[at:] = 2 ** 31 - 1 - ctx[at:]
    have, total = -(-ctx // B), -(-(ctx + new) // B)
    width = int(max(have.max(), total[:at].max(initial=0))) + 4
    pages = np.full((R, width), -5, dtype=np.int32)
    for r in range(R):
        pages[r, :have[r]] = 7 * r + np.arange(have[r])
    free = (1000000 + np.arange(int((total - have)[:at].sum()) + 2)).astype(np.int32)
    taken = np.concatenate([[0], np.cumsum(total - have)])
    want = pages.copy()
    for r in range(R):
        for i in range(int(have[r]), int(min(total[r], width))):
            f = taken[r] + i - have[r]
            want[r, i] = free[f] if f < len(free) else -1
    blocks = np.where(new > 0, -(-(ctx % B + new) // B), 0)
    nb, T = int(blocks[:at].sum()) + 5, int(new[:at].sum()) + 3
    tab, tok = [], []
    for r in range(at + 1):
        p, t = int(ctx[r]), int(new[:r].sum())
        while p < ctx[r] + new[r] and len(tab) < nb:
            end = min(int(ctx[r] + new[r]), (p // B + 1) * B)
            tab.append((t, end - p))
            t, p = t + end - p, end
        tok += [(r, int(ctx[r]) + i) for i in range(min(int(new[r]), T - len(tok)))]
    t32 = lambda a: torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()  # noqa: E731
    e = lambda *s, dtype=torch.int32: torch.full(s, 77, dtype=dtype, device="cuda")  # noqa: E731
    b = {"new_len": t32(new), "ctx_len": t32(ctx), "pages": t32(pages), "free_pages": t32(free), "req_off": e(R + 1),
         "req_blk_off": e(R + 1), "blk_tab": e(nb, 2), "insert_slot": e(nb), "totals": e(4)}
    if maps:
        b.update(tok_req=e(T), tok_pos=e(T), slot_map=e(T, dtype=torch.int64))
    n = nat.moer_block_plan_workspace_bytes(R)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    args = nat.make_block_plan(R=R, block=B, T=T, nblk=nb, ld_pages=width, n_free=len(free), **b)
    torch.cuda.synchronize()
    start = time.perf_counter()
    nat.moer_block_plan(args, ws, n)
    assert nat.moer_ws_status(ws) == 6
    assert time.perf_counter() - start < 0.5
    assert np.array_equal(b["pages"].cpu().numpy(), want)
    assert b["blk_tab"].cpu().numpy().tolist() == [list(x) for x in tab]
    assert b["totals"].cpu().numpy().tolist()[0] == min(int(new.sum()), 2 ** 31 - 1)
    if maps:
        assert list(zip(b["tok_req"].tolist(), b["tok_pos"].tolist())) == tok


# More than eight choices at sizes past the rule's 2,816 rows, and the same rows a few at a time
@pytest.mark.parametrize("E,k,n,keep", [(16, 9, 1, 1), (24, 12, 1, 1), (64, 16, 1, 1), (72, 10, 1, 1), (128, 10, 1, 1), (160, 12, 1, 1), (256, 16, 1, 1),
                                        (256, 10, 8, 4), (128, 16, 8, 3), (64, 9, 8, 2), (160, 12, 5, 2)])
@pytest.mark.parametrize("special,dtype", [(None, "f32"), ("masks", "bf16"), ("ties", "f16"), ("ties", "f32"), ("inf", "f32"), ("lowest", "bf16")])
def test_many_choices(env, E, k, n, keep, special, dtype):
    torch, _ = env
    rs = np.random.RandomState(E + k + 5)
    dev, x = _logits(torch, rs, 2, 1500, E, dtype, special=special)
    for biased, score, renorm in ((False, "softmax", False), (True, "softmax", True), (True, "sigmoid", True), (False, "sigmoid", False)):
        bias = rs.normal(0, 0.3, size=(2, E)) if biased else None
        o = dict(score=score, renorm=renorm, n_group=n, top_group=keep, best=1 + biased)
        ids, w, ss = _forward(env, dev, E, k, dtype, bias=bias, sums=renorm, **o)
        few = [_forward(env, dev[:, a:a + 750], E, k, dtype, bias=bias, sums=False, **o) for a in (0, 750)]
        gap = router.score_topk(x, k, bias=None if bias is None else bias.astype(np.float32), **o)[3]
        tol = 1e-5 * (1 + (0 if bias is None else np.abs(bias).max()))
        for l in range(2):
            at = gap[l] > tol  # other rows may go either way in fp32
            assert np.array_equal(ids[l, at], np.concatenate([f[0][l] for f in few])[at])
            if at.any():
                _check_forward((ids[l:l + 1, at], w[l:l + 1, at], None), x[l:l + 1, at], k, bias=None if bias is None else bias[l:l + 1], **o)
        if renorm:
            sums = router.scores(x, score).sum(1)
            assert (np.abs(ss - sums) <= 6e-6 * sums + 1e-30).all()


# Several tiles to a warp (4,864 units share the rows: from 155,648 rows with k <= 8, 77,824 with
# k <= 16 and 38,912 beyond): the loads ahead and the shared rows of the second and later tiles
@pytest.mark.parametrize("E,k,L,T", [(64, 6, 3, 70001), (128, 8, 1, 200003), (256, 8, 2, 90007), (60, 5, 2, 100001), (128, 12, 2, 50003), (256, 20, 1, 50021)])
@pytest.mark.parametrize("score,renorm,sums", [("softmax", False, True), ("softmax", False, False), ("softmax", True, True), ("softmax", True, False),
                                               ("sigmoid", False, True), ("sigmoid", True, True), ("sigmoid", True, False)])
@pytest.mark.parametrize("dtype,layout", [("f32", "layer"), ("bf16", "token")])
def test_gradient_of_many_rows(env, E, k, L, T, score, renorm, sums, dtype, layout):
    """The whole result against the formulas in 64 bits, with masks, on the GPU; the bounds are _check_grad's."""
    torch, nat = env
    gen = torch.Generator(device="cuda")
    gen.manual_seed(E + k)
    x = torch.randn((L, T, E) if layout == "layer" else (T, L, E), device="cuda", generator=gen)
    x = x if layout == "layer" else x.permute(1, 0, 2)
    x = x.mul_(2.0).masked_fill_(torch.rand((L, T, E), device="cuda", generator=gen) < 0.02, -math.inf).to(getattr(torch, DT[dtype]))
    ids = torch.rand((L, T, E), device="cuda", generator=gen).topk(k, -1).indices
    dw = torch.randn((L, T, k), device="cuda", generator=gen)
    da = torch.randn((L, E), device="cuda", generator=gen) if sums else None
    d, o = nat.make_dims(E, k, L, [], 16), nat.make_score_opts(dtype=dtype, score=score, renorm=renorm, scale=1.5)
    out = torch.full_like(x, 9.0)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    nat.moer_score_topk_grad(d, o, x, T, x.stride(1), x.stride(0), ids.to(torch.uint8), dw, da, out, out.stride(1), out.stride(0), ws, 256)
    assert nat.moer_ws_status(ws) == 0
    for l in range(L):
        z = x[l].double()
        s = torch.sigmoid(z) if score == "sigmoid" else torch.softmax(z, -1)
        at, g = ids[l], dw[l].double() * 1.5
        p = s.gather(1, at)
        q = p / p.sum(-1, keepdim=True).clamp_min(1e-300)
        dx, mag = torch.zeros_like(s), torch.zeros_like(s)
        for to, sign, gg, a in ((dx, -1.0, g, None if da is None else da[l].double()), (mag, 1.0, g.abs(), None if da is None else da[l].double().abs())):
            part = q * (gg + sign * (gg * q).sum(-1, keepdim=True)) if renorm else gg * p
            if score == "sigmoid":
                part = part * (1 - p)
                if a is not None:
                    to += a * s * (1 - s)
            else:
                if a is not None:
                    to += s * (a + sign * (a * s).sum(-1, keepdim=True))
                if not renorm:
                    to += sign * s * (gg * p).sum(-1, keepdim=True)
            to.scatter_add_(1, at, part)
        lim = 1e-5 * mag + 1e-37
        lo, hi = ((dx + f * lim).to(x.dtype).double() for f in (-1.0, 1.0))
        got = out[l].double()
        assert bool(((got >= lo) & (got <= hi)).all()), (l, int((~((got >= lo) & (got <= hi))).sum()))


# Groups without a live expert score -inf and tie, whether their logits are -inf or NaN
@pytest.mark.parametrize("E,k,n,keep", [(16, 4, 8, 4), (64, 6, 8, 3), (128, 8, 4, 2), (256, 8, 8, 4)])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("T", [70, 2100])
def test_groups_of_masks(env, E, k, n, keep, best, T):
    torch, _ = env
    rs = np.random.RandomState(E + T)
    x = rs.normal(size=(1, T, n, E // n))
    x[rs.random_sample((1, T, n)) < 0.4] = -np.inf
    x[rs.random_sample((1, T, n)) < 0.4] = np.nan
    dev, x = _device(torch, x.reshape(1, T, E), "f32")
    for bias in (None, rs.normal(0, 0.3, size=(1, E))):
        o = dict(score="sigmoid", renorm=True, n_group=n, top_group=keep, best=best)
        _check_forward(_forward(env, dev, E, k, "f32", bias=bias, **o), x, k, bias=bias, **o)
