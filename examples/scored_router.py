"""One prefill batch through a scored router and one layer's experts, as a serving engine would run
them, and one training step of both.

From the requests' lengths the GPU makes the batch's block tables and KV slots; the router's
logits become expert ids and weights (sigmoid scores, a balance bias, 4 of 8 expert groups);
the ids go on to the signature and decoder choice and into the experts' token lists; and the
weights' and score sums' gradients come back to the logits.  At the first layer the hidden states
pass the norm, the experts' products over those lists and the combination per token, and the
gradients come back through all of them; the weights' one goes on to that layer's logits.

    python examples/scored_router.py
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from moe_expert_routing_top_gb300 import _native as nat  # noqa: E402
from moe_expert_routing_top_gb300 import pipeline  # noqa: E402


def main(E=128, k=8, L=4, R=64, B=16, D=4, H=512, I=128, seed=0):
    rs = np.random.RandomState(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    # the batch: new and cached tokens of each request, the KV cache's block table and free pages
    new = rs.randint(1, 200, size=R)
    ctx = rs.randint(0, 20, size=R) * B
    held = ctx // B
    need = -(-(ctx + new) // B) - held
    ids = rs.permutation(int((held + need).sum()) + 32).astype(np.int32)
    table = np.full((R, int((held + need).max())), -1, dtype=np.int32)
    at = 0
    for r in range(R):
        table[r, :held[r]] = ids[at:at + held[r]]
        at += held[r]
    pages, free = torch.from_numpy(table).cuda(), torch.from_numpy(ids[at:]).cuda()
    bd = pipeline.BatchDev.from_lengths(new, ctx, B, pages, free)

    # the router's state: signature mask, decoders, expert groups of the load statistics
    mask = [0, L - 1]
    rs_ = pipeline.RoutingStats(E, k, L, mask, B, D=D, tau=0.1, centroids=rs.rand(D, len(mask) * E), idf=np.ones((len(mask), E)),
                                loads=np.zeros(D), live=True, G=8, group_of=np.tile(np.arange(E) % 8, (L, 1)), nslots=len(ids),
                                max_T=bd.T, max_nblk=bd.nblk, max_R=bd.R)
    bias = torch.zeros((L, E), device="cuda")
    rs_.set_gate(nat.make_score_opts(score="sigmoid", renorm=True, n_group=8, top_group=4, group_best=2, scale=2.5), bias)

    logits = torch.randn((L, bd.T, E), device="cuda", generator=gen)
    sums = torch.empty((L, E), device="cuda")
    off, order, inv = rs_.score_step(logits, bd, align=16, score_sum=sums)

    # the first layer's experts, on the hidden states
    dtype = torch.bfloat16
    w1 = (torch.randn((E, 2 * I, H), device="cuda", generator=gen) * H ** -0.5).to(dtype)
    w2 = (torch.randn((E, H, I), device="cuda", generator=gen) * I ** -0.5).to(dtype)
    experts = pipeline.ExpertLayer(w1, w2, norm_weight=torch.ones(H, device="cuda", dtype=dtype))
    attention = torch.randn((bd.T, H), device="cuda", generator=gen).to(dtype)
    x, hidden, rstd = experts.norm(attention, torch.randn((bd.T, H), device="cuda", generator=gen).to(dtype))
    weights = rs_.weights_for(bd.T)[0].clone()
    out, kept = experts.forward(x, off[0], order[0], inv[0], weights, add=hidden)
    grads = experts.backward(kept, torch.randn((bd.T, H), device="cuda", generator=gen).to(dtype))
    d_attention, d_norm = experts.norm_grad(hidden, rstd, grads["x"])

    # balance: experts with more tokens than the mean are made less likely for the next batch
    load = rs_.W.float()
    rs_.bias -= 0.001 * torch.sign(load - load.mean(-1, keepdim=True))

    # training: the gradient of a loss in the weights and of a balance loss in the mean scores
    d_weights = torch.randn((L, bd.T, k), device="cuda", generator=gen)
    d_weights[0] = grads["weights"]
    d_sums = 0.01 * E * load / (load.sum(-1, keepdim=True) * bd.T)
    d_logits = rs_.score_grad(logits, d_weights, d_sums)
    torch.cuda.synchronize()
    if rs_.status() != 0 or experts.status() != 0:
        raise RuntimeError("the workspace reports bad data")
    return {"batch": bd, "stats": rs_, "off": off, "order": order, "inv": inv, "sums": sums, "logits": logits,
            "d_weights": d_weights, "d_sums": d_sums, "d_logits": d_logits, "pages": pages,
            "experts": experts, "kept": kept, "weights": weights, "out": out, "hidden": hidden, "grads": grads, "d_attention": d_attention,
            "d_norm": d_norm}


if __name__ == "__main__":
    out = main()
    bd, stats = out["batch"], out["stats"]
    print(f"{bd.R} requests, {bd.T} tokens in {bd.nblk} KV blocks; decoders {stats.choice[:8].tolist()} ...; "
          f"largest expert load {int(stats.W.max())} of {bd.T}; |d_logits| {float(out['d_logits'].abs().mean()):.2e}; "
          f"experts' outputs {float(out['out'].float().std()):.2f}, |d_w1| {float(out['grads']['w1'].abs().mean()):.2e}")
