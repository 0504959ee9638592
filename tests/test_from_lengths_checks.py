"""What BatchDev.from_lengths hands to the library, and what it refuses, on the CPU: the call is
replaced by a recorder that fills the block table as the oracle does."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
nat = pytest.importorskip("moe_expert_routing_top_gb300._native")
from moe_expert_routing_top_gb300 import pipeline  # noqa: E402
from oracle import router  # noqa: E402

B = 16
NEW, CTX = np.array([20, 0, 5, 33]), np.array([16, 40, 0, 3])


@pytest.fixture
def plans(monkeypatch):
    seen = []

    def plan(args, ws, ws_bytes, stream=None):
        b = args._keepalive
        seen.append((args, b))
        if b.get("pages") is not None:
            assert args.ld_pages == b["pages"].shape[1] and b["pages"].is_contiguous()
            free = b["free_pages"]
            router.block_plan(b["new_len"].numpy(), b["ctx_len"].numpy(), args.block, b["pages"].numpy(),
                              None if free is None else free.numpy())
    monkeypatch.setattr(nat, "moer_block_plan", plan)
    monkeypatch.setattr(nat, "moer_ws_status", lambda ws, stream=None: 0)
    return seen


def _table(rows=4, width=4):
    t = torch.full((rows, width), -1, dtype=torch.int32)
    for r, c in enumerate(CTX):
        t[r, :-(-int(c) // B)] = torch.arange(-(-int(c) // B), dtype=torch.int32) + 100 * r
    return t


FREE = torch.arange(50, 60, dtype=torch.int32)


def _want():
    t = _table().numpy()
    router.block_plan(NEW, CTX, B, t, FREE.numpy())
    return torch.from_numpy(t)


def test_a_tables_rows(plans):
    t = _table()
    pipeline.BatchDev.from_lengths(NEW, CTX, B, t, FREE, device="cpu")
    assert plans[0][1]["pages"] is t and torch.equal(t, _want())


@pytest.mark.parametrize("cut", ["columns", "rows", "transposed"])
def test_a_slice_of_a_wider_table(plans, cut):
    wide = torch.full((8, 12), 7, dtype=torch.int32)
    t = {"columns": wide[:4, 3:7], "rows": wide[::2, :4], "transposed": wide.t()[:4, :4]}[cut]
    t.copy_(_table())
    before = wide.clone()
    pipeline.BatchDev.from_lengths(NEW, CTX, B, t, FREE, device="cpu")
    assert torch.equal(t, _want())
    t.copy_(_table())
    assert torch.equal(wide, before)  # nothing else was written


@pytest.mark.parametrize("new,ctx,pages,free", [
    (NEW, CTX[:1], None, None), (NEW, np.append(CTX, 3), None, None), (NEW.reshape(2, 2), CTX.reshape(2, 2), None, None),
    (NEW, np.array([0, 0, 0, 2 ** 31]), None, None), (np.array([2 ** 32 + 5, 0, 0, 0]), CTX, None, None),
    (NEW, CTX, _table()[:3], FREE), (NEW, CTX, _table().long(), FREE), (NEW, CTX, _table().reshape(-1), FREE), (NEW, CTX, _table().to("meta"), FREE),
    (NEW, CTX, _table(), FREE.long()), (NEW, CTX, _table(), FREE.reshape(2, 5)), (NEW, CTX, _table(), FREE.to("meta")),
    (NEW, CTX, None, FREE)])
def test_arguments_that_do_not_fit(plans, new, ctx, pages, free):
    with pytest.raises(ValueError):
        pipeline.BatchDev.from_lengths(new, ctx, B, pages, free, device="cpu")
    assert not plans


def test_every_other_free_page(plans):
    t = _table()
    pipeline.BatchDev.from_lengths(NEW, CTX, B, t, torch.stack([FREE, -FREE], 1)[:, 0], device="cpu")
    assert torch.equal(t, _want())
