"""The router operators together: the tables from lengths against the host-made ones, the scored
step against the raw-logits step where both compute the same, and the example end to end."""
import importlib.util
import os

import numpy as np
import pytest

import gen
from oracle import router

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_routing_top_gb300 import _native as nat
    from moe_expert_routing_top_gb300 import pipeline
    from tests import gpu_util
    return torch, nat, pipeline, gpu_util


def _lengths(wl):
    new = np.array([wl.computed_tokens(r) for r in range(wl.R)])
    ctx = np.asarray(wl.cached_blocks[:wl.R]) * wl.B
    pages = np.full((wl.R, max(len(s) for s in wl.slot_of_block)), -1, dtype=np.int32)
    for r, s in enumerate(wl.slot_of_block[:wl.R]):
        pages[r, :len(s)] = s
    return new, ctx, pages


def test_tables_from_lengths(env):
    torch, _, pipeline, _ = env
    wl = gen.make_workload("c4", R=300)
    host = pipeline.BatchDev.from_host(wl.batch())
    new, ctx, pages = _lengths(wl)
    bd = pipeline.BatchDev.from_lengths(new, ctx, wl.B, torch.from_numpy(pages).cuda())
    assert (bd.T, bd.R, bd.nblk, bd.ncached) == (host.T, host.R, host.nblk, host.ncached)
    for name in ("blk_tab", "req_blk_off", "cache_idx", "req_cache_off", "insert_slot"):
        assert torch.equal(getattr(bd, name).reshape(-1), getattr(host, name).reshape(-1)), name


@pytest.mark.parametrize("cfg,R", [("c1", None), ("c4", 60)])
def test_scored_step_equals_the_raw_step(env, cfg, R):
    """A softmax gate without bias or groups chooses what the raw logits choose, so counts,
    signatures, loads, skew and decoder choices are the raw step's."""
    torch, nat, pipeline, gu = env
    wl = gen.make_workload(cfg, R=R)
    b = wl.batch()
    logits = gu.device_logits(wl, b)
    raw = pipeline.RoutingStats.for_workload(wl, max_T=b.T, max_nblk=b.nblk, max_R=b.R)
    raw.step(logits, pipeline.BatchDev.from_host(b))
    new, ctx, pages = _lengths(wl)
    bd = pipeline.BatchDev.from_lengths(new, ctx, wl.B, torch.from_numpy(pages).cuda())
    rs = pipeline.RoutingStats.for_workload(wl)
    rs.set_gate(nat.make_score_opts(renorm=False))
    off, order, inv = rs.score_step(logits, bd, align=16)
    assert raw.status() == 0 and rs.status() == 0
    assert torch.equal(rs.topk_for(b.T), raw.topk_for(b.T))
    for name in ("affinity", "W", "Wg", "rho_g", "rho_e"):
        assert torch.equal(getattr(rs, name), getattr(raw, name)), name
    assert torch.equal(rs.blk_cnt[:b.nblk], raw.blk_cnt[:b.nblk]) and torch.equal(rs.choice[:b.R], raw.choice[:b.R])
    assert torch.equal(rs.loads, raw.loads)
    ids = raw.topk_for(b.T)
    p = torch.softmax(logits.double(), -1).gather(-1, ids.long())
    assert ((rs.weights_for(b.T) - p).abs() <= 4e-6 * p).all()   # a score's bound (test_gpu_router.py)
    ro, rr, ri = router.expert_order(ids.cpu().numpy(), wl.E, 16, order.shape[1])
    assert np.array_equal(off.cpu().numpy(), ro) and np.array_equal(order.cpu().numpy(), rr)
    assert np.array_equal(inv.cpu().numpy(), ri)


def test_scored_step_of_256_experts(env):
    torch, nat, pipeline, _ = env
    L, E, k, B, R = 2, 256, 8, 16, 9
    rs_ = np.random.RandomState(2)
    new = rs_.randint(1, 90, size=R)
    bd = pipeline.BatchDev.from_lengths(new, np.zeros(R, int), B)
    st = pipeline.RoutingStats(E, k, L, [0, 1], B, D=3, tau=0.1, centroids=rs_.rand(3, 2 * E), idf=np.ones((2, E)), loads=np.zeros(3),
                               live=False, G=4, group_of=np.zeros((L, E)))
    bias = rs_.normal(0, 0.05, size=(L, E)).astype(np.float32)
    o = dict(score="sigmoid", n_group=8, top_group=4)
    st.set_gate(nat.make_score_opts(group_best=2, scale=2.5, **o), bias)
    x = rs_.normal(size=(L, bd.T, E)).astype(np.float32)
    st.score_step(torch.from_numpy(x).cuda(), bd)
    assert st.status() == 0
    ids, w, _, gap = router.score_topk(x, k, bias=bias, best=2, scale=2.5, **o)
    ok = gap > 2e-5
    got = st.topk_for(bd.T).cpu().numpy()
    assert ok.mean() > 0.9 and np.array_equal(got[ok], ids[ok])
    cnt = np.stack([np.bincount(got[l].reshape(-1), minlength=E) for l in range(L)])
    assert np.array_equal(st.req_cnt[:R].sum(0).cpu().numpy(), cnt)


def test_example(env):
    torch, _, _, _ = env
    spec = importlib.util.spec_from_file_location("scored_router", os.path.join(ROOT, "examples", "scored_router.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    out = m.main(R=20)
    bd, st = out["batch"], out["stats"]
    ids = st.topk_for(bd.T).cpu().numpy().astype(np.int64)
    x = out["logits"].double().cpu().numpy()
    dx, mag = router.score_topk_grad(x, ids, out["d_weights"].cpu().numpy(), out["d_sums"].cpu().numpy(), "sigmoid", True, 2.5)
    assert (np.abs(out["d_logits"].cpu().numpy() - dx) <= 1e-5 * mag + 1e-30).all()
    # every pair is listed once, in its expert's segment
    off, order, inv = (out[n].cpu().numpy() for n in ("off", "order", "inv"))
    for l in range(ids.shape[0]):
        flat = ids[l].reshape(-1)
        assert np.array_equal(order[l][inv[l].reshape(-1)], np.arange(len(flat)))
        assert (off[l][flat] <= inv[l].reshape(-1)).all() and (inv[l].reshape(-1) < off[l][flat + 1]).all()
    # slots are those of the block table
    slot = bd.slot_map.cpu().numpy()
    pos, req, pages = bd.tok_pos.cpu().numpy(), bd.tok_req.cpu().numpy(), out["pages"].cpu().numpy()
    assert np.array_equal(slot, pages[req, pos // 16].astype(np.int64) * 16 + pos % 16)
