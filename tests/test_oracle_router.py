"""The 64-bit statements of the router operators against brute force and against differences."""
import itertools

import numpy as np
import pytest

from oracle import router


def test_choice_is_the_best_subset():
    rs = np.random.RandomState(0)
    x = rs.normal(size=(1, 20, 8))
    bias = rs.normal(size=(1, 8)) * 0.1
    ids, w, _, _ = router.score_topk(x, 3, "sigmoid", True, bias)
    c = router.scores(x, "sigmoid") + bias
    for t in range(20):
        best = max(itertools.combinations(range(8), 3), key=lambda s: sum(c[0, t, i] for i in s))
        assert set(ids[0, t]) == set(best)
    assert np.allclose(w.sum(-1), 1.0)


def test_groups_keep_the_best_two():
    x = np.array([[[3.0, 0.0, 2.0, 1.9, 1.0, 1.0]]])  # three groups of two
    one, _, _, _ = router.score_topk(x, 2, "softmax", n_group=3, top_group=1, best=1)
    two, _, _, _ = router.score_topk(x, 2, "sigmoid", n_group=3, top_group=1, best=2)
    assert one.tolist() == [[[0, 1]]] and two.tolist() == [[[2, 3]]]


def test_masked_rows_have_no_weight():
    x = np.full((1, 3, 4), -np.inf)
    x[0, 1, 2], x[0, 2, 1] = 1.0, np.nan
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            ids, w, s, _ = router.score_topk(x, 2, score, renorm, np.full((1, 4), 5.0))
            assert ids[0].tolist() == [[0, 1], [2, 0], [0, 2]]
            assert w[0, 0].tolist() == [0, 0] and w[0, 2].tolist() == [0, 0] and w[0, 1, 1] == 0 and w[0, 1, 0] > 0
            assert np.isfinite(s).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("sums", [True, False])
def test_gradient_against_differences(score, renorm, sums):
    """Central differences with step h: error O(h^2) of the third derivative, which these
    functions keep below 1; h = 1e-4 leaves 1e-8 and rounding 1e-16 / h = 1e-12."""
    rs = np.random.RandomState(1)
    L, T, E, k = 2, 3, 8, 3
    x = rs.normal(size=(L, T, E))
    x[0, 0, 5] = -np.inf
    ids = np.stack([[rs.permutation(E)[:k] for _ in range(T)] for _ in range(L)])
    dw, da = rs.normal(size=(L, T, k)), rs.normal(size=(L, E)) if sums else None

    def loss(z):
        s = router.scores(z, score)
        w = np.take_along_axis(s, ids, -1)
        if renorm:
            w = w / w.sum(-1, keepdims=True)
        return (1.7 * w * dw).sum() + (0 if da is None else (s.sum(1) * da).sum())

    dx, mag = router.score_topk_grad(x, ids, dw, da, score, renorm, 1.7)
    assert (np.abs(dx) <= mag + 1e-12).all()
    h = 1e-4
    for at in np.ndindex(L, T, E):
        if np.isinf(x[at]):
            assert dx[at] == 0
            continue
        hi, lo = x.copy(), x.copy()
        hi[at] += h
        lo[at] -= h
        assert abs((loss(hi) - loss(lo)) / (2 * h) - dx[at]) < 1e-7


def test_plan_matches_the_workloads_tables():
    """The batch tables that the workload generator makes on the host, from lengths alone."""
    import gen
    wl = gen.make_workload("c4", R=40)
    b = wl.batch()
    new = np.array([wl.computed_tokens(r) for r in range(40)])
    ctx = wl.cached_blocks[:40] * wl.B
    width = int(max(len(s) for s in wl.slot_of_block))
    pages = np.full((40, width), -1)
    for r, s in enumerate(wl.slot_of_block[:40]):
        pages[r, :len(s)] = s
    p = router.block_plan(new, ctx, wl.B, pages)
    assert np.array_equal(p["req_off"], b.req_off) and np.array_equal(p["blk_tab"], b.blk_tab)
    assert np.array_equal(p["req_blk_off"], b.req_blk_off) and np.array_equal(p["cache_idx"], b.cache_idx)
    assert np.array_equal(p["req_cache_off"], b.req_cache_off) and np.array_equal(p["insert_slot"], b.insert_slot)


def test_plan_continues_a_page():
    pages = np.array([[7, 9, -1], [3, -1, -1]])
    p = router.block_plan([3, 0], [6, 4], 4, pages, [5])
    assert p["blk_tab"].tolist() == [[0, 2], [2, 1]] and p["insert_slot"].tolist() == [-1, -1]
    assert p["slot_map"].tolist() == [38, 39, 20] and pages.tolist() == [[7, 9, 5], [3, -1, -1]]
    assert p["cache_idx"].tolist() == [7, 3] and p["totals"].tolist() == [3, 2, 2, 1]


def test_order_by_hand():
    ids = np.array([[[2, 0], [2, 9], [0, 1]]])
    off, order, inv = router.expert_order(ids, 4, 2, 9)
    assert off.tolist() == [[0, 2, 4, 6, 6]]
    assert order.tolist() == [[1, 4, 5, -1, 0, 2, -1, -1, -1]]
    assert inv.tolist() == [[[4, 0], [5, -1], [1, 2]]]
