"""The router entry points' refusals, on the CPU: every call here is rejected on the host."""
import ctypes

import pytest

nat = pytest.importorskip("moe_expert_routing_top_gb300._native")

BADPTR = 0x1001  # misaligned, never dereferenced


def _code(fn, *args):
    with pytest.raises(nat.MoerError) as ei:
        fn(*args)
    return ei.value.code


@pytest.mark.parametrize("E,k,over,code", [
    (128, 8, dict(dtype=3), 1), (128, 8, dict(score=2), 1), (128, 8, dict(renorm=2), 1),
    (128, 8, dict(scale=float("inf")), 3), (128, 8, dict(scale=float("nan")), 3),
    (128, 8, dict(n_group=0), 3), (128, 8, dict(n_group=33), 3), (128, 8, dict(n_group=3), 3),
    (128, 8, dict(n_group=8, top_group=9), 3), (128, 8, dict(n_group=8, top_group=0), 3),
    (128, 8, dict(n_group=8, top_group=4, group_best=3), 3),
    (32, 8, dict(n_group=8, top_group=1), 2),                      # fewer experts than k
    (16, 1, dict(n_group=16, top_group=4, group_best=2), 2),       # no second expert in a group
    (260, 8, {}, 3), (64, 33, {}, 3)])
def test_options(E, k, over, code):
    d = nat.make_dims(E, k, 2, [], 16)
    o = nat.make_score_opts(**over)
    assert _code(nat.moer_score_topk, d, o, 64, 10, E, 10 * E, None, 64, None, None, 64, 1 << 20, 0) == code
    assert _code(nat.moer_score_topk_grad, d, o, 64, 10, E, 10 * E, 64, 64, None, 64, E, 10 * E, 64, 256, 0) == code


def test_score_topk_arguments():
    d, o = nat.make_dims(128, 8, 2, [], 16), nat.make_score_opts()
    n = nat.moer_score_workspace_bytes(d, 100)
    f = nat.moer_score_topk

    def call(logits=64, T=100, lt=128, ll=12800, bias=None, topk=64, w=64, ss=None, ws=64, wb=n, dims=d, opts=o):
        return f(dims, opts, logits, T, lt, ll, bias, topk, w, ss, ws, wb, 0)
    assert _code(lambda: call(logits=None)) == 1
    assert _code(lambda: call(logits=0x1002)) == 1             # fp32 on 2 bytes
    assert _code(lambda: call(topk=None)) == 1
    assert _code(lambda: call(topk=0x1004)) == 1
    assert _code(lambda: call(bias=BADPTR)) == 1
    assert _code(lambda: call(w=BADPTR)) == 1
    assert _code(lambda: call(ss=BADPTR)) == 1
    assert _code(lambda: call(ws=None)) == 1
    assert _code(lambda: call(ws=0x1008)) == 1
    assert _code(lambda: call(wb=n - 1)) == 5
    assert _code(lambda: call(T=-1)) == 3
    assert _code(lambda: call(T=1 << 31)) == 3
    assert _code(lambda: call(lt=127)) == 2
    assert _code(lambda: call(ll=100)) == 2
    assert _code(lambda: call(lt=1 << 60)) == 2
    assert nat.LIB.moer_score_topk(ctypes.byref(d), None, 64, 1, 128, 128, None, 64, None, None, 64, n, None) == 1
    assert nat.LIB.moer_score_topk(None, ctypes.byref(o), 64, 1, 128, 128, None, 64, None, None, 64, n, None) == 1
    f(d, o, None, 0, 128, 128, None, None, None, None, None, 0, 0)   # no tokens, no sums: nothing to do
    assert nat.moer_score_workspace_bytes(nat.make_dims(1000, 8, 2, [], 16), 100) == 256


def test_grad_arguments():
    d, o = nat.make_dims(128, 8, 2, [], 16), nat.make_score_opts(dtype="bf16")
    f = nat.moer_score_topk_grad

    def call(logits=64, T=100, lt=128, ll=12800, topk=64, dw=64, da=None, out=64, gt=128, gl=12800, ws=64, wb=256):
        return f(d, o, logits, T, lt, ll, topk, dw, da, out, gt, gl, ws, wb, 0)
    for over, code in ((dict(logits=None), 1), (dict(logits=BADPTR), 1), (dict(topk=None), 1), (dict(topk=BADPTR), 1),
                       (dict(dw=None), 1), (dict(dw=0x1002), 1), (dict(da=0x1002), 1), (dict(out=None), 1),
                       (dict(out=BADPTR), 1), (dict(lt=64), 2), (dict(gt=64), 2), (dict(gl=0), 2), (dict(ws=None), 1),
                       (dict(wb=255), 5), (dict(T=-5), 3)):
        assert _code(lambda: call(**over)) == code, over
    call(T=0)


def test_block_plan_arguments():
    f = nat.moer_block_plan
    n = nat.moer_block_plan_workspace_bytes(10)
    ok = dict(R=10, block=16, T=100, nblk=10, ncached=4, ld_pages=8, n_free=5, new_len=64, ctx_len=64, pages=64,
              free_pages=64, req_off=64, req_blk_off=64, blk_tab=64, insert_slot=64, req_cache_off=64, cache_idx=64,
              slot_map=64, tok_req=64, tok_pos=64, totals=64)

    def code(ws=64, wb=n, **over):
        return _code(f, nat.make_block_plan(**{**ok, **over}), ws, wb, 0)
    for over, want in ((dict(R=-1), 3), (dict(R=(1 << 20) + 1), 3), (dict(block=0), 3), (dict(block=256), 3), (dict(T=-1), 3),
                       (dict(T=1 << 31), 3), (dict(nblk=-1), 3), (dict(ncached=-1), 3), (dict(ld_pages=-1), 3),
                       (dict(n_free=-1), 3), (dict(req_off=None), 1), (dict(req_blk_off=None), 1), (dict(new_len=None), 1),
                       (dict(pages=None), 1), (dict(pages=None, ld_pages=0), 1), (dict(blk_tab=None), 1),
                       (dict(req_cache_off=None), 1), (dict(free_pages=None), 1), (dict(tok_pos=BADPTR), 1),
                       (dict(slot_map=0x1004), 1), (dict(new_len=0x1002), 1), (dict(ws=None), 1), (dict(ws=0x1008), 1),
                       (dict(wb=n - 1), 5)):
        assert code(**over) == want, over
    assert nat.LIB.moer_block_plan(None, 64, n, None) == 1
    with pytest.raises(TypeError):
        nat.make_block_plan(R=1, block=16, no_such_buffer=64)


def test_expert_order_arguments():
    d = nat.make_dims(128, 8, 2, [], 16)
    n = nat.moer_expert_order_workspace_bytes(d, 100)
    f = nat.moer_expert_order

    def call(topk=64, T=100, align=16, off=64, order=64, ld=800 + 128 * 15, inv=64, ws=64, wb=n, dims=d):
        return f(dims, topk, T, align, off, order, ld, inv, ws, wb, 0)
    for over, code in ((dict(topk=None), 1), (dict(topk=0x1004), 1), (dict(off=None), 1), (dict(off=BADPTR), 1),
                       (dict(order=BADPTR), 1), (dict(inv=BADPTR), 1), (dict(align=0), 3), (dict(align=1025), 3), (dict(T=-1), 3),
                       (dict(T=1 << 28), 3), (dict(ld=800 + 128 * 15 - 1), 2), (dict(ws=None), 1), (dict(wb=n - 1), 5),
                       (dict(dims=nat.make_dims(128, 40, 2, [], 16)), 3)):
        assert _code(lambda: call(**over)) == code, over
    assert nat.moer_expert_order_workspace_bytes(nat.make_dims(64, 1000, 2, [], 16), 100) == 256
