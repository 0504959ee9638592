"""Workspace sizes of the router operators: a program asks once, for its largest batch."""
import pytest

nat = pytest.importorskip("moe_expert_routing_top_gb300._native")


@pytest.mark.parametrize("E,k,L", [(128, 8, 48), (256, 8, 26), (64, 6, 26), (128, 8, 1), (60, 4, 7), (16, 2, 256)])
def test_sizes_grow_with_the_batch(E, k, L):
    d = nat.make_dims(E, k, L, [], 16)
    tokens = list(range(0, 9000)) + list(range(9001, 2_000_000, 997)) + [1 << n for n in range(15, 31)] + [2 ** 31 - 1]
    for size in (nat.moer_score_workspace_bytes, nat.moer_expert_order_workspace_bytes):
        last = 0
        for T in sorted(tokens):
            n = size(d, T)
            assert n >= last, (size.__name__, T)
            last = n


def test_block_plan_sizes_grow():
    sizes = [nat.moer_block_plan_workspace_bytes(R) for R in range(5000)]
    assert sizes == sorted(sizes)


@pytest.mark.parametrize("E,k,L", [(128, 8, 48), (256, 8, 26), (16, 2, 256)])
def test_score_size_holds_every_unit(E, k, L):
    """A partial sum of every span of tokens that the gate may take: L T / 4864 tokens, rounded
    up to a multiple of the eight rows that a block takes at a time."""
    d = nat.make_dims(E, k, L, [], 16)
    for T in list(range(1, 6000)) + [65536, 131072, 1_000_003]:
        span = (T * L + 4863) // 4864
        span = (span + 7) // 8 * 8
        assert nat.moer_score_workspace_bytes(d, T) >= 256 + L * ((T + span - 1) // span) * E * 4, T
