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


def test_batches_larger_than_the_buffers(env):
    torch, nat, pipeline = env
    L, E, k = 3, 64, 6
    rs = _stats(pipeline, nat, L, E, k, max_T=10, renorm=False)
    for T in (10, 3000, 41):
        x = torch.randn((L, T, E), device="cuda")
        rs.score_topk(x)
        _check(rs, x.double().cpu().numpy(), T, k, renorm=False)
        off, order, inv = rs.expert_order(T)
        assert (order.sort(1).values.cpu() == torch.arange(T * k, dtype=torch.int32)).all()
        dw = torch.randn((L, T, k), device="cuda")
        dx = rs.score_grad(x, dw)
        g, mag = router.score_topk_grad(x.double().cpu().numpy(), rs.topk_for(T).cpu().numpy(), dw.cpu().numpy(), renorm=False)
        assert (np.abs(dx.cpu().numpy() - g) <= 1e-5 * mag + 1e-37).all()
    assert rs.status() == 0


def test_step_of_padded_logits(env):
    torch, nat, pipeline = env
    L, E, k = 2, 128, 8
    new = np.array([30, 17, 40])
    bd = pipeline.BatchDev.from_lengths(new, np.zeros(3, int), 16)
    x = torch.randn((L, 128, E), device="cuda")
    a, b = (_stats(pipeline, nat, L, E, k) for _ in range(2))
    off, order, inv = a.score_step(x, bd)
    off2, order2, inv2 = b.score_step(x[:, :bd.T].contiguous(), bd)
    assert a.status() == 0 and b.status() == 0
    assert torch.equal(a.topk_for(bd.T), b.topk_for(bd.T)) and torch.equal(a.affinity, b.affinity)
    assert torch.equal(order, order2) and torch.equal(inv, inv2) and torch.equal(off, off2)
    assert torch.equal(a.req_cnt[:3], b.req_cnt[:3])


def test_gradient_of_a_sum_and_of_other_layouts(env):
    torch, nat, pipeline = env
    L, T, E, k = 2, 70, 64, 6
    rs = _stats(pipeline, nat, L, E, k)
    x = torch.randn((L, T, E), device="cuda")
    rs.score_topk(x)
    for dw in (torch.ones((), device="cuda").expand(L, T, k), torch.randn((T, L, k), device="cuda").transpose(0, 1),
               torch.randn((L, T, k), device="cuda").to(torch.bfloat16)):
        dx = rs.score_grad(x, dw)
        g, mag = router.score_topk_grad(x.double().cpu().numpy(), rs.topk_for(T).cpu().numpy(), dw.float().cpu().numpy())
        assert (np.abs(dx.cpu().numpy() - g) <= 1e-5 * mag + 1e-37).all()


def test_gradients_of_two_batches_under_way(env):
    torch, nat, pipeline = env
    L, T, E, k = 2, 70, 64, 6
    rs = _stats(pipeline, nat, L, E, k)
    x = [torch.randn((L, T, E), device="cuda") for _ in range(2)]
    ids = []
    for b in range(2):
        rs.score_topk(x[b])
        ids.append(rs.topk_for(T).clone())
    dw = torch.randn((L, T, k), device="cuda")
    for b in range(2):
        dx = rs.score_grad(x[b], dw, topk=ids[b])
        g, mag = router.score_topk_grad(x[b].double().cpu().numpy(), ids[b].cpu().numpy(), dw.cpu().numpy())
        assert (np.abs(dx.cpu().numpy() - g) <= 1e-5 * mag + 1e-37).all()


def _lengths(rs, R, B, most_new, most_ctx):
    new, ctx = rs.randint(0, most_new, size=R), rs.randint(0, most_ctx, size=R)
    have, total = -(-ctx // B), -(-(ctx + new) // B)
    pool = rs.permutation(int(total.sum()) + 5).astype(np.int32)
    pages, at = np.full((R, int(total.max()) + 1), -1, dtype=np.int32), 0
    for r in range(R):
        pages[r, :have[r]] = pool[at:at + have[r]]
        at += have[r]
    return new, ctx, pages, pool[at:]


@pytest.mark.parametrize("R", [9, 3000])
@pytest.mark.parametrize("slice_", ["columns", "transposed"])
def test_block_table_that_is_a_slice(env, R, slice_):
    torch, nat, pipeline = env
    new, ctx, pages, free = _lengths(np.random.RandomState(R), R, 16, 60, 100)
    W = pages.shape[1]
    wide = torch.full((R, W + 9), 12345, dtype=torch.int32, device="cuda") if slice_ == "columns" else torch.full((W + 9, R), 12345, dtype=torch.int32, device="cuda")
    t = wide[:, 4:4 + W] if slice_ == "columns" else wide[4:4 + W].t()
    t.copy_(torch.from_numpy(pages).cuda())
    bd = pipeline.BatchDev.from_lengths(new, ctx, 16, t, torch.from_numpy(free).cuda())
    ref = router.block_plan(new, ctx, 16, pages, free)
    assert np.array_equal(t.cpu().numpy(), pages) and np.array_equal(bd.slot_map.cpu().numpy(), ref["slot_map"])
    assert np.array_equal(bd.cache_idx.cpu().numpy()[:bd.ncached], ref["cache_idx"]) and np.array_equal(bd.insert_slot.cpu().numpy(), ref["insert_slot"])
    t.fill_(12345)
    assert (wide == 12345).all()


def _busy(torch):
    """Some milliseconds of work on the current stream."""
    a = torch.randn((4096, 4096), device="cuda")
    for _ in range(40):
        a = (a @ a).mul_(1e-2)
    return a


@pytest.mark.parametrize("handle", [False, True])
def test_tables_on_another_stream(env, handle):
    """What the current stream still has to do (the workspace's zeroing, the table's making) comes first."""
    torch, nat, pipeline = env
    side = torch.cuda.Stream()
    for R in (9, 3000):
        new, ctx, pages, free = _lengths(np.random.RandomState(R + 1), R, 16, 60, 100)
        host, fr = torch.from_numpy(pages).cuda(), torch.from_numpy(free).cuda()
        torch.cuda.synchronize()
        busy = _busy(torch)
        t = host + 0 * busy[0, 0].nan_to_num(0.0, 0.0, 0.0).int()
        bd = pipeline.BatchDev.from_lengths(new, ctx, 16, t, fr, stream=side.cuda_stream if handle else side)
        ref = router.block_plan(new, ctx, 16, pages, free)
        assert np.array_equal(t.cpu().numpy(), pages) and np.array_equal(bd.slot_map.cpu().numpy(), ref["slot_map"])
        assert np.array_equal(bd.req_off.cpu().numpy(), ref["req_off"]) and np.array_equal(bd.blk_tab.cpu().numpy(), ref["blk_tab"])


@pytest.mark.parametrize("handle", [False, True])
def test_buffers_on_the_launches_stream(env, handle):
    """A RoutingStats on a stream of its own, while the current one still has to fill memory that it
    has given back: neither side's writes reach the other's tensors."""
    torch, nat, pipeline = env
    L, T, E, k = 2, 4000, 64, 6
    side = torch.cuda.Stream()
    rs = _stats(pipeline, nat, L, E, k, max_T=T, stream=side.cuda_stream if handle else side)
    x = torch.randn((L, T, E), device="cuda")
    dw = torch.randn((T, L, k), device="cuda").transpose(0, 1)
    torch.cuda.synchronize()
    _busy(torch)
    sizes = [(L * (E + 1), torch.int32), (L * T * k, torch.int32), (L * T * k, torch.int32), (L * T * E, torch.float32), (L * T * k, torch.float32)]
    late = [torch.empty(n, dtype=d, device="cuda").fill_(77) for n, d in sizes]
    del late  # the fills are still to come
    rs.score_topk(x)
    off, order, inv = rs.expert_order(T)
    dx = rs.score_grad(x, dw)
    torch.cuda.synchronize()
    assert rs.status() == 0
    ids = rs.topk_for(T).cpu().numpy()
    ro, rr, ri = router.expert_order(ids, E, 1, T * k)
    assert np.array_equal(off.cpu().numpy(), ro) and np.array_equal(order.cpu().numpy(), rr) and np.array_equal(inv.cpu().numpy(), ri)
    g, mag = router.score_topk_grad(x.double().cpu().numpy(), ids, dw.cpu().numpy())
    assert (np.abs(dx.cpu().numpy() - g) <= 1e-5 * mag + 1e-37).all()


def test_step_on_a_stream_of_its_own(env):
    torch, nat, pipeline = env
    L, E, k = 2, 64, 6
    side = torch.cuda.Stream()
    new = np.array([300, 17, 40])
    bd = pipeline.BatchDev.from_lengths(new, np.zeros(3, int), 16)
    x = torch.randn((L, bd.T, E), device="cuda")
    torch.cuda.synchronize()
    a = _stats(pipeline, nat, L, E, k, stream=side)
    b = _stats(pipeline, nat, L, E, k)
    out = [s.score_step(x, bd) for s in (a, b)]
    torch.cuda.synchronize()
    assert a.status() == 0 and b.status() == 0
    assert all(torch.equal(u, v) for u, v in zip(*out)) and torch.equal(a.affinity, b.affinity) and torch.equal(a.W, b.W)


def test_current_streams_handle(env):
    """The library's default stream is torch's current one, inside and outside a stream's context."""
    torch, nat, pipeline = env
    assert nat.current_handle() == torch.cuda.current_stream().cuda_stream == nat.current_handle(torch.cuda.current_device())
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert nat.current_handle() == side.cuda_stream
