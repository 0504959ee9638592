"""One routing-statistics step over a batch, through the C ABI.

`RoutingStats` owns the caller-side buffers the C ABI expects (PyTorch
allocates them; the library allocates nothing) and issues, on one CUDA
stream:

  moer_topk_signature  top-k + per-KV-block counts + co-activation (one pass)
  moer_block_stitch    prefix-cache stitching into per-request counts
  moer_affinity_load   expert / group loads and skew from the co-activation
  moer_route           signatures, centroid distances, tau-band decoder choice

or, when the router logits are not materialised, `moer_gate_topk` (the bf16
gate GEMM with top-k, block counts and co-activation fused behind it) in
place of the first call.  `moer_ids_signature` derives the block counts and
co-activation from top-k ids already produced (the bench uses it to time the
dominant kernel's call alone).

With a scored gate (`set_gate`: softmax or sigmoid scores, a balance bias, expert
groups, renormalised weights) the step runs on the ids of `moer_score_topk`
instead and also gives the experts' weights and token lists (`score_step`;
`moer_expert_order`); `score_grad` is the gate's gradient for training.
`ExpertLayer` runs what a layer computes with those lists: the norm, the experts' products and
activation, the combination per token and the gradients (`moer_rms_norm`, `moer_expert_gemm`,
`moer_expert_act`, `moer_expert_combine`).
`BatchDev.from_lengths` makes a batch's tables on the GPU from its requests'
lengths (`moer_block_plan`).

`calibrate` runs the offline half (idf, greedy layer mask, balanced K-means
centroids, spectral expert groups) call by call on the GPU, and
`save_calibration` / `load_calibration` carry its result to the serving side.

This module only marshals arguments and orders calls; every step of the
path runs in the library's kernels.
"""
from __future__ import annotations

import contextlib
import dataclasses
from typing import Optional

import numpy as np
import torch

from . import _native as nat


_AS_IT_IS = contextlib.nullcontext()
_GATE_DTYPES = {0: torch.float32, 1: torch.bfloat16, 2: torch.float16}  # by moer_dtype


def _as_stream(stream, device):
    """A torch stream of a torch stream or a handle."""
    if not isinstance(stream, int):
        return stream
    return torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)


@dataclasses.dataclass
class BatchDev:
    """Device copies of one batch's metadata (see gen.workloads.Batch)."""
    T: int
    R: int
    nblk: int
    blk_tab: torch.Tensor
    req_blk_off: torch.Tensor
    cache_idx: Optional[torch.Tensor]
    req_cache_off: Optional[torch.Tensor]
    insert_slot: Optional[torch.Tensor]
    ncached: int = 0
    req_off: Optional[torch.Tensor] = None   # with from_lengths: [R+1] CSR of the computed tokens,
    slot_map: Optional[torch.Tensor] = None  # [T] int64 KV cache slot of each,
    tok_req: Optional[torch.Tensor] = None   # [T] its request
    tok_pos: Optional[torch.Tensor] = None   # [T] and its position there

    @staticmethod
    def from_lengths(new_len, ctx_len, block, pages=None, free_pages=None, device="cuda", stream=None) -> "BatchDev":
        """A batch's tables made on the GPU from the requests' lengths (host arrays: tokens to
        compute, tokens held in the KV cache).  `pages` [R][width] int32 (device) is the KV
        cache's block table, with the held tokens' pages in it; the pages newly needed come
        from `free_pages` [n] int32 (device) in request order and are written into it.  The call
        runs on `stream`, after what the current stream has under way, and waits for it.  A table
        that is a slice of a wider one is copied and written back.  Without `pages` the batch
        has no slots and no signature cache."""
        n, c = np.asarray(new_len, dtype=np.int64), np.asarray(ctx_len, dtype=np.int64)
        if n.ndim != 1 or n.shape != c.shape:
            raise ValueError(f"lengths of shapes {n.shape} and {c.shape}: expected one of each per request")
        new, ctx, B, R = n.astype(np.int32), c.astype(np.int32), int(block), len(n)
        if (new != n).any() or (ctx != c).any():
            raise ValueError("a length does not fit 32 bits")
        where = torch.device(device).type
        if pages is None and free_pages is not None:
            raise ValueError("free pages without a block table")
        if pages is not None and (pages.dtype != torch.int32 or pages.dim() != 2 or pages.shape[0] < R or pages.device.type != where):
            raise ValueError(f"pages has to be int32 [{R} requests or more][width] on {device}")
        if free_pages is not None and (free_pages.dtype != torch.int32 or free_pages.dim() != 1 or free_pages.device.type != where):
            raise ValueError(f"free_pages has to be int32 [n] on {device}")
        table = pages
        if pages is not None:
            pages = pages.contiguous()
        if free_pages is not None:
            free_pages = free_pages.contiguous()
        T, nblk = int(n.sum()), int(np.where(n > 0, -(-(c % B + n) // B), 0).sum())
        ncached = int((c // B).sum()) if pages is not None else 0
        i32 = torch.int32

        def empty(*shape, dtype=i32):
            return torch.empty(shape, dtype=dtype, device=device)
        b = {"new_len": torch.from_numpy(new).to(device), "ctx_len": torch.from_numpy(ctx).to(device),
             "req_off": empty(R + 1), "req_blk_off": empty(R + 1), "blk_tab": empty(max(nblk, 1), 2),
             "tok_req": empty(T), "tok_pos": empty(T)}
        if pages is not None:
            b.update(pages=pages, free_pages=free_pages, insert_slot=empty(max(nblk, 1)), req_cache_off=empty(R + 1),
                     cache_idx=empty(max(ncached, 1)), slot_map=empty(T, dtype=torch.int64))
        args = nat.make_block_plan(R=R, block=B, T=T, nblk=nblk, ncached=ncached,
                                   ld_pages=0 if pages is None else pages.shape[1],
                                   n_free=0 if free_pages is None else free_pages.numel(), **b)
        wsb = nat.moer_block_plan_workspace_bytes(R)
        ws = torch.zeros(wsb, dtype=torch.uint8, device=device)
        if stream is not None and where == "cuda":
            # the launch comes after the workspace's zeroing, the copies and the table's producer,
            # which are on the current stream; what is made there is safe to use after the wait below
            _as_stream(stream, ws.device).wait_stream(torch.cuda.current_stream(ws.device))
        nat.moer_block_plan(args, ws, wsb, stream)
        code = nat.moer_ws_status(ws, stream)
        if pages is not table:
            table.copy_(pages)
        if code != 0:
            raise nat.MoerError("moer_block_plan", code, nat.moer_status_str(code))
        return BatchDev(T=T, R=R, nblk=nblk, blk_tab=b["blk_tab"], req_blk_off=b["req_blk_off"],
                        cache_idx=b.get("cache_idx"), req_cache_off=b.get("req_cache_off"),
                        insert_slot=b.get("insert_slot"), ncached=ncached, req_off=b["req_off"],
                        slot_map=b.get("slot_map"), tok_req=b["tok_req"], tok_pos=b["tok_pos"])

    @staticmethod
    def from_host(b, device="cuda", with_cache=True, pin=False) -> "BatchDev":
        def t(a, dt=torch.int32):
            x = torch.from_numpy(np.ascontiguousarray(a)).to(dt)
            if pin:
                x = x.pin_memory()
            return x.to(device, non_blocking=pin)
        ci = t(b.cache_idx) if with_cache and len(b.cache_idx) else None
        return BatchDev(T=b.T, R=b.R, nblk=b.nblk, blk_tab=t(b.blk_tab.reshape(-1)),
                        req_blk_off=t(b.req_blk_off),
                        cache_idx=ci if with_cache else None,
                        req_cache_off=t(b.req_cache_off) if with_cache else None,
                        insert_slot=t(b.insert_slot) if with_cache else None,
                        ncached=int(len(b.cache_idx)) if with_cache else 0)


class _OnStream:
    """What owns buffers on `self.device` and launches on `self.stream`."""

    def _on_stream(self):
        """Makes the launches' stream the current one: what is allocated, filled or copied within
        is in order with them, and its memory goes back to that stream."""
        return torch.cuda.stream(_as_stream(self.stream, self.device)) if self._elsewhere() else _AS_IT_IS

    def _elsewhere(self):
        if self.device.type != "cuda":
            return False
        if self.device.index is not None and torch.cuda.current_device() != self.device.index:
            return True
        return nat.current_handle(self.device.index) != (self.stream if isinstance(self.stream, int) else self.stream.cuda_stream)

    def _results(self, *tensors):
        """Tensors made on the launches' stream, for a caller on the current one."""
        if self._elsewhere():
            for t in tensors:
                t.record_stream(torch.cuda.current_stream(self.device))
        return tensors


class RoutingStats(_OnStream):
    """Holds the model/serving state of the path and runs steps over batches on `stream` (the one
    that is current when it is made, if none is given).  Inputs have to be ready on that stream,
    and a reader on another one has to wait for it."""

    def __init__(self, E, k, L, mask, block, *, D, tau, centroids, idf, loads, live, G, group_of,
                 nslots=0, max_T=0, max_nblk=0, max_R=0, device="cuda", stream=None):
        self.dims = nat.make_dims(E, k, L, list(mask), block)
        self.E, self.k, self.L, self.m, self.B = E, k, L, len(mask), block
        self.D, self.tau, self.live, self.G = D, float(tau), bool(live), G
        dev = torch.device(device)
        self.device = dev
        self.stream = stream if stream is not None else torch.cuda.current_stream(dev)
        with self._on_stream():
            f32, i32 = torch.float32, torch.int32
            self.centroids = torch.as_tensor(np.asarray(centroids), dtype=f32).to(dev).contiguous()
            self.idf = torch.as_tensor(np.asarray(idf), dtype=f32).to(dev).contiguous()
            self.loads = torch.as_tensor(np.asarray(loads), dtype=i32).to(dev).contiguous()
            self.group_of = torch.as_tensor(np.asarray(group_of), dtype=i32).to(dev).contiguous()
            self.affinity = torch.zeros((L, E, E), dtype=i32, device=dev)
            self.W = torch.empty((L, E), dtype=torch.int64, device=dev)
            self.Wg = torch.empty((L, G), dtype=torch.int64, device=dev)
            self.rho_g = torch.empty(L, dtype=torch.float64, device=dev)
            self.rho_e = torch.empty(L, dtype=torch.float64, device=dev)
            self.n_rep = torch.empty(L, dtype=i32, device=dev)
            self.rep_src = torch.empty(L, dtype=i32, device=dev)
            self.hot = torch.empty((L, E), dtype=torch.uint8, device=dev)
            self.rep_dst = torch.empty((L, G), dtype=i32, device=dev)
            self.w_pred = torch.empty((L, G), dtype=torch.float64, device=dev)
            self.cache = (torch.zeros((nslots, self.m, E), dtype=torch.uint8, device=dev)
                          if nslots > 0 else None)
        self.nslots = nslots
        self.gate_H = 0
        self.score_opts = self.bias = None
        self._alloc(max_T, max_nblk, max_R)

    def _alloc(self, T, nblk, R):
        self.cap = (T, nblk, R)
        self.ids_T = None  # tokens of the batch whose ids self.topk holds
        with self._on_stream():
            self._make(T, nblk, R)

    def _make(self, T, nblk, R):
        dev, E, k, L, m, D = self.device, self.E, self.k, self.L, self.m, self.D
        self.topk = torch.empty(L * max(T, 1) * k, dtype=torch.uint8, device=dev)
        self.blk_cnt = torch.empty((max(nblk, 1), m, E), dtype=torch.uint8, device=dev)
        self.req_cnt = torch.empty((max(R, 1), m, E), dtype=torch.int32, device=dev)
        self.sig = torch.empty((max(R, 1), m * E), dtype=torch.float32, device=dev)
        self.dist = torch.empty((max(R, 1), D), dtype=torch.float32, device=dev)
        self.choice = torch.empty(max(R, 1), dtype=torch.int32, device=dev)
        self.ws_bytes = nat.moer_workspace_bytes(self.dims, T, nblk, R, D)
        if self.gate_H:
            self.ws_bytes = max(self.ws_bytes, nat.moer_gate_workspace_bytes(self.dims, self.gate_H))
        if self.score_opts is not None:
            self.weights = torch.empty(L * max(T, 1) * k, dtype=torch.float32, device=dev)
            self.ws_bytes = max(self.ws_bytes, nat.moer_score_workspace_bytes(self.dims, T),
                                nat.moer_expert_order_workspace_bytes(self.dims, T))
        self.ws = torch.zeros(self.ws_bytes, dtype=torch.uint8, device=dev)

    def ensure(self, T, nblk, R, H=0):
        grow_gate = H > self.gate_H
        if grow_gate:
            self.gate_H = H
        if grow_gate or T > self.cap[0] or nblk > self.cap[1] or R > self.cap[2]:
            self._alloc(max(T, self.cap[0]), max(nblk, self.cap[1]), max(R, self.cap[2]))

    def topk_for(self, T: int) -> torch.Tensor:
        """The top-k ids of the last batch of T tokens, as [L][T][k]."""
        return self.topk[:self.L * T * self.k].view(self.L, T, self.k)

    # ------------------------------------------------------ scored gates
    def set_gate(self, opts: "nat.moer_score_opts", bias=None):
        """The scored gate of `score_step` (options from make_score_opts) and its balance bias
        ([L][E], or None).  The tensor in use is `self.bias`, which may be changed in place: the
        given one if it is contiguous fp32 on this device, else a copy of it."""
        with self._on_stream():
            if bias is not None:
                bias = torch.as_tensor(bias, dtype=torch.float32).to(self.device).contiguous()
                if tuple(bias.shape) != (self.L, self.E):
                    raise ValueError(f"bias has shape {tuple(bias.shape)}, expected {(self.L, self.E)}")
        self.score_opts, self.bias = opts, bias
        self._alloc(*self.cap)

    def weights_for(self, T: int) -> torch.Tensor:
        """The weights of the last batch of T tokens, as [L][T][k]."""
        return self.weights[:self.L * T * self.k].view(self.L, T, self.k)

    def _check_logits(self, logits, what="logits"):
        """The library takes addresses: a tensor of another type, shape or layout than the gate's
        would be read, or written, past its end."""
        if self.score_opts is None:
            raise ValueError("no scored gate: call set_gate first")
        if logits.dtype != _GATE_DTYPES.get(self.score_opts.dtype):
            raise ValueError(f"{what} are {logits.dtype}, the gate's options say {_GATE_DTYPES.get(self.score_opts.dtype)}")
        shape = logits.shape
        if len(shape) != 3 or shape[0] != self.L or shape[2] != self.E:
            raise ValueError(f"{what} have shape {tuple(shape)}, expected ({self.L}, T, {self.E})")
        if logits.stride(2) != 1:
            raise ValueError(f"{what}: the logits of a row have to be contiguous")
        if logits.device != self.ws.device:
            raise ValueError(f"{what} are on {logits.device}, expected {self.ws.device}")

    def _is(self, x, dtype, shape) -> bool:
        return x.dtype == dtype and x.shape == shape and x.is_contiguous() and x.device == self.ws.device

    def _as_f32(self, x, shape, what):
        """x as contiguous fp32, itself where it is that already."""
        if self._is(x, torch.float32, shape):
            return x
        if not x.is_floating_point() or x.shape != shape or x.device != self.ws.device:
            raise ValueError(f"{what} has to be a floating tensor of shape {shape} on {self.ws.device}")
        with self._on_stream():
            return x.to(torch.float32).contiguous()

    def score_topk(self, logits, score_sum=None):
        """Top-k ids and weights of the scored gate; logits [L][T][E] of the gate's type with any
        strides between rows; score_sum [L][E] fp32, if given, receives the scores' sums."""
        self._check_logits(logits)
        self.ensure(logits.shape[1], 0, 0)
        self._score_topk(logits, logits.shape[1], score_sum)

    def _score_topk(self, logits, T, score_sum):
        if score_sum is not None and not self._is(score_sum, torch.float32, (self.L, self.E)):
            raise ValueError(f"score_sum has to be contiguous fp32 {(self.L, self.E)} on {self.ws.device}")
        self.ids_T = T
        nat.moer_score_topk(self.dims, self.score_opts, logits, T, logits.stride(1), logits.stride(0), self.bias,
                            self.topk, self.weights, score_sum, self.ws, self.ws_bytes, self.stream)

    def score_grad(self, logits, d_weights, d_score_sum=None, out=None, topk=None) -> torch.Tensor:
        """The logits' gradient from that of the weights ([L][T][k]) and, if given, of the
        score sums ([L][E]), for the ids `topk` ([L][T][k] uint8) that the weights belong to.
        Without `topk` they are those of the last score_topk call: with several batches under
        way, keep a copy of each one's ids (topk_for(T).clone()) and give it here.  Gradients
        that are not contiguous fp32 are copied to it."""
        self._check_logits(logits)
        T = logits.shape[1]
        if topk is None:
            if T != self.ids_T:
                raise ValueError(f"logits of {T} tokens, but the ids held are of {self.ids_T}")
            topk = self.topk
        elif not self._is(topk, torch.uint8, (self.L, T, self.k)):
            raise ValueError(f"topk has to be contiguous uint8 {(self.L, T, self.k)} on {self.ws.device}")
        d_weights = self._as_f32(d_weights, (self.L, T, self.k), "d_weights")
        if d_score_sum is not None:
            d_score_sum = self._as_f32(d_score_sum, (self.L, self.E), "d_score_sum")
        made = out is None
        if made:
            with self._on_stream():
                out = torch.empty_like(logits)
        else:
            self._check_logits(out, "out's entries")
            if out.shape != logits.shape:
                raise ValueError("out has to have the logits' shape")
        nat.moer_score_topk_grad(self.dims, self.score_opts, logits, T, logits.stride(1), logits.stride(0), topk,
                                 d_weights, d_score_sum, out, out.stride(1), out.stride(0), self.ws, self.ws_bytes,
                                 self.stream)
        if made:
            self._results(out)
        return out

    def expert_order(self, T: int, align: int = 1):
        """The experts' token lists of the last batch: offsets [L][E+1], pairs in expert order
        [L][rows] (segments padded to `align`) and each pair's row [L][T][k]."""
        if T > self.cap[0]:
            raise ValueError(f"{T} tokens, but the ids' buffer holds {self.cap[0]}")
        n = T * self.k
        ld = n + min(self.E, n) * (align - 1)
        i32, dev = torch.int32, self.device
        with self._on_stream():
            off = torch.empty((self.L, self.E + 1), dtype=i32, device=dev)
            order = torch.empty((self.L, ld), dtype=i32, device=dev)
            inv = torch.empty((self.L, T, self.k), dtype=i32, device=dev)
        nat.moer_expert_order(self.dims, self.topk, T, align, off, order, ld, inv, self.ws, self.ws_bytes, self.stream)
        return self._results(off, order, inv)

    def score_step(self, logits, bd: BatchDev, align=1, score_sum=None, write_sig=True):
        """All rows of the path over one batch through the scored gate, and the experts' token
        lists (returned).  Co-activation and loads need E <= 128 and k in {6, 8}
        (moer_ids_signature's limit) and are left as they are otherwise.  Logits padded past
        the batch's tokens are taken up to them."""
        self._check_logits(logits)
        T = logits.shape[1]
        if T < bd.T:
            raise ValueError(f"logits of {T} tokens, but the batch has {bd.T}")
        self.ensure(bd.T, bd.nblk, bd.R)
        self._score_topk(logits if T == bd.T else logits[:, :bd.T], bd.T, score_sum)
        counted = self.E <= 128 and self.k in (6, 8)
        self.ids_signature(bd, blk_counts=True, affinity=counted)
        self.block_stitch(bd)
        if counted:
            self.affinity_load()
        self.route(bd.R, write_sig)
        return self.expert_order(bd.T, align)

    def reset_stats(self):
        with self._on_stream():
            self.affinity.zero_()

    # ------------------------------------------------------------ the step
    def topk_signature(self, logits, bd: BatchDev, write_topk=True, blk_counts=True):
        """Top-k ids and co-activation, plus the block counts unless ``blk_counts`` is False
        (then ``ids_signature`` can produce them from the ids)."""
        if write_topk:
            self.ids_T = bd.T
        nat.moer_topk_signature(self.dims, logits, bd.T, bd.blk_tab, bd.nblk,
                                self.topk if write_topk else None,
                                self.blk_cnt if blk_counts else None, self.affinity,
                                self.ws, self.ws_bytes, self.stream)

    def gate_topk(self, hidden, w_gate, bd: BatchDev, logits=None, counts=True):
        """hidden bf16 [T][H] x w_gate bf16 [L][H][E] -> top-k and, unless ``counts`` is False,
        block counts and co-activation (else ``ids_signature`` produces them from the ids)."""
        H = hidden.shape[-1]
        self.ids_T = bd.T
        nat.moer_gate_topk(self.dims, hidden, bd.T, H, w_gate, bd.blk_tab, bd.nblk, logits,
                           self.topk, self.blk_cnt if counts else None,
                           self.affinity if counts else None, self.ws, self.ws_bytes,
                           self.stream)

    def ids_signature(self, bd: BatchDev, blk_counts=True, affinity=False):
        """Block counts (and, if asked, co-activation) from the top-k ids in ``self.topk``."""
        T = bd.T
        nat.moer_ids_signature(self.dims, self.topk, T, bd.blk_tab, bd.nblk,
                               self.blk_cnt if blk_counts else None,
                               self.affinity if affinity else None, self.ws, self.ws_bytes, self.stream)

    def block_stitch(self, bd: BatchDev):
        use_cache = self.cache is not None and bd.req_cache_off is not None
        nat.moer_block_stitch(self.dims, self.blk_cnt, bd.blk_tab, bd.nblk, bd.req_blk_off, bd.R,
                              bd.cache_idx if use_cache else None,
                              bd.ncached if use_cache else 0,
                              bd.req_cache_off if use_cache else None,
                              self.cache if use_cache else None, self.nslots,
                              bd.insert_slot if use_cache else None, self.req_cnt, self.ws,
                              self.ws_bytes, self.stream)

    def affinity_load(self):
        nat.moer_affinity_load(self.dims, self.affinity, self.group_of, self.G, self.W, self.Wg,
                               self.rho_g, self.rho_e, self.stream)

    def replication_plan(self):
        """GRACE replication plan per layer from the current loads (after affinity_load)."""
        nat.moer_replication_plan(self.dims, self.W, self.group_of, self.G, self.n_rep, self.rep_src,
                                  self.hot, self.rep_dst, self.w_pred, self.ws, self.ws_bytes,
                                  self.stream)

    def route(self, R, write_sig=True):
        nat.moer_route(self.dims, self.req_cnt, R, self.idf, self.centroids, self.D, self.tau,
                       self.loads, int(self.live), self.sig if write_sig else None, self.dist,
                       self.choice, self.ws, self.ws_bytes, self.stream)

    def step(self, logits, bd: BatchDev, write_topk=True, write_sig=True):
        """All rows of the path over one batch (loads and co-activation accumulate)."""
        self.ensure(bd.T, bd.nblk, bd.R)
        self.topk_signature(logits, bd, write_topk)
        self.block_stitch(bd)
        self.affinity_load()
        self.route(bd.R, write_sig)

    def gate_step(self, hidden, w_gate, bd: BatchDev, write_sig=True):
        """All rows of the path over one batch, starting from hidden states (gate GEMM)."""
        self.ensure(bd.T, bd.nblk, bd.R, hidden.shape[-1])
        self.gate_topk(hidden, w_gate, bd)
        self.block_stitch(bd)
        self.affinity_load()
        self.route(bd.R, write_sig)

    def capture_step(self, logits, bd: BatchDev, write_topk=True, write_sig=True):
        """A CUDA graph of one ``step`` on these buffers and inputs (their device addresses
        are baked in): ``replay()`` runs the whole step again with no per-call host work.

        One eager step runs first, on the pipeline's stream, so that the library's one-time
        set-up (kernel attributes, the tensor-map encoder) and any buffer growth happen
        outside the capture; its counts accumulate like any step's.  The capture itself
        runs on a side stream (the legacy default stream cannot be captured)."""
        self.step(logits, bd, write_topk, write_sig)
        torch.cuda.synchronize(self.affinity.device)
        graph = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream(device=self.affinity.device)
        own = self.stream
        self.stream = side
        try:
            with torch.cuda.graph(graph, stream=side):
                self.step(logits, bd, write_topk, write_sig)
        finally:
            self.stream = own
        return graph

    def status(self) -> int:
        return nat.moer_ws_status(self.ws, self.stream)

    @staticmethod
    def for_workload(wl, *, max_T=0, max_nblk=0, max_R=0, device="cuda", stream=None):
        return RoutingStats(wl.E, wl.k, wl.L, wl.mask, wl.B, D=wl.D, tau=wl.tau,
                            centroids=wl.centroids, idf=wl.idf, loads=wl.loads0, live=wl.live,
                            G=wl.G, group_of=wl.group_of, nslots=wl.nslots, max_T=max_T,
                            max_nblk=max_nblk, max_R=max_R, device=device, stream=stream)


def to_8bit_blocks(w):
    """Weights [E][N][K] as e4m3 with an fp32 scale for each block of 128 x 128 (moer_expert_gemm's
    layout), by torch operations: done once, when a model is loaded."""
    E, N, K = w.shape
    pad = torch.nn.functional.pad(w.float(), (0, -K % 128, 0, -N % 128))
    b = pad.view(E, -(-N // 128), 128, -(-K // 128), 128)
    scale = (b.abs().amax((2, 4)) / 448.0).clamp_(min=1e-30)
    q = (b / scale[:, :, None, :, None]).view(E, pad.shape[1], pad.shape[2])[:, :N, :K]
    return q.to(torch.float8_e4m3fn).contiguous(), scale.contiguous()


@dataclasses.dataclass
class ExpertPass:
    """What a forward pass of ExpertLayer leaves for its backward pass: x and the lists as they were
    given (they have to stay as they are until then), its own tensors, and a copy of the weights."""
    x: torch.Tensor
    h: torch.Tensor
    a: torch.Tensor
    z: torch.Tensor
    off: torch.Tensor
    order: torch.Tensor
    inv: torch.Tensor
    weights: torch.Tensor


class ExpertLayer(_OnStream):
    """One layer's experts behind a router: the norm in front (`norm`, if it has a weight), the gated
    products over the experts' token lists and their combination per token (`forward`), and the
    gradients (`norm_grad`, `backward`).  The lists are one layer's of RoutingStats.expert_order or
    score_step, the weights one layer's of weights_for:

        off, order, inv = rs.score_step(logits, batch, align=128)
        y, hidden, _ = layer.norm(x, hidden)
        out, kept = layer.forward(y, off[l], order[l], inv[l], rs.weights_for(T)[l], add=hidden)

    w1 [E][2 I][H] (the halves a and b of the activation one after the other) and w2 [E][H][I], both
    bf16 or fp16; or both e4m3 with `scales` (of w1 and w2, from to_8bit_blocks), which serve only:
    the rows then go through both products in 8 bits.  Calls run on `stream` (the current one when
    the layer is made, if none is given); inputs have to be ready there, and a reader on another one
    has to wait for it."""

    def __init__(self, w1, w2, scales=None, norm_weight=None, eps=1e-6, dtype=torch.bfloat16, stream=None):
        self.device = w1.device
        if w1.dim() != 3 or w2.dim() != 3 or w1.shape[1] % 2 or w2.shape != (w1.shape[0], w1.shape[2], w1.shape[1] // 2):
            raise ValueError(f"weights of shapes {tuple(w1.shape)} and {tuple(w2.shape)}: expected [E][2 I][H] and [E][H][I]")
        self.E, self.H, self.I = w1.shape[0], w1.shape[2], w2.shape[2]
        self.eight = w1.dtype == torch.float8_e4m3fn
        self.dtype = dtype if self.eight else w1.dtype
        if not 1 <= self.H <= 16384:
            raise ValueError(f"H {self.H}: at most 16384")
        if w1.dtype != w2.dtype or self.dtype not in (torch.bfloat16, torch.float16) or w2.device != self.device:
            raise ValueError("weights have to be bf16, fp16 or e4m3, both of one type, on one device")
        if not (w1.is_contiguous() and w2.is_contiguous()):
            raise ValueError("weights have to be contiguous")
        unit = 16 if self.eight else 8
        if self.H % unit or self.I % unit:
            raise ValueError(f"H {self.H} and I {self.I} have to be multiples of {unit}: a row starts on 16 bytes")
        if self.eight != (scales is not None):
            raise ValueError("e4m3 weights need their scales, and no others have any")
        if self.eight:
            for w, s in zip((w1, w2), scales):
                want = (self.E, -(-w.shape[1] // 128), -(-w.shape[2] // 128))
                if tuple(s.shape) != want or s.dtype != torch.float32 or not s.is_contiguous() or s.device != self.device:
                    raise ValueError(f"scales have to be contiguous fp32 {want} on {self.device}")
        if norm_weight is not None and (norm_weight.shape != (self.H,) or norm_weight.dtype != self.dtype or
                                        not norm_weight.is_contiguous() or norm_weight.device != self.device):
            raise ValueError(f"the norm's weight has to be contiguous {self.dtype} of {self.H} on {self.device}")
        self.w1, self.w2, self.scales, self.norm_weight, self.eps = w1, w2, scales, norm_weight, float(eps)
        self.stream = stream if stream is not None or self.device.type != "cuda" else torch.cuda.current_stream(self.device)
        if self.device.type == "cuda":  # a layer may go, with its weights, while its last launches read them
            for t in (w1, w2, *(scales or ()), norm_weight):
                if t is not None:
                    t.record_stream(_as_stream(self.stream, self.device))
        # the calls' status word; what a call writes besides (norm_grad's partial sums) is its own, since graphs captured
        # of one layer may run at the same time
        with self._on_stream():
            self.ws = torch.zeros(nat.moer_expert_gemm_workspace_bytes(nat.make_expert_gemm()), dtype=torch.uint8, device=self.device)
        self.ws_bytes = self.ws.numel()

    # ---------------------------------------------------------------- pieces
    def _takes(self, *tensors):
        """Inputs from the current stream, for launches on another: their memory stays theirs until those ran."""
        if self._elsewhere():
            for t in tensors:
                if t is not None:
                    t.record_stream(_as_stream(self.stream, self.device))

    def _name(self):
        return "bf16" if self.dtype == torch.bfloat16 else "f16"

    def _rows(self, x, cols, what, rows=None, dtype=None):
        dtype = dtype or self.dtype
        if x.dim() != 2 or x.shape[1] != cols or (rows is not None and x.shape[0] != rows) or x.dtype != dtype or x.device != self.device:
            raise ValueError(f"{what} has to be {dtype} [{'rows' if rows is None else rows}][{cols}] on {self.device}, "
                             f"got {x.dtype} {tuple(x.shape)} on {x.device}")
        if x.stride(1) != 1 and cols > 1:
            raise ValueError(f"{what}: the elements of a row have to be contiguous")
        return x

    def _lists(self, off, order, inv, weights):
        def ints(t, shape, what):
            if t.dtype != torch.int32 or tuple(t.shape) != shape or not t.is_contiguous() or t.device != self.device:
                raise ValueError(f"{what} has to be contiguous int32 {shape} on {self.device}")
        ints(off, (self.E + 1,), "off")
        if order.dim() != 1 or inv.dim() != 2:
            raise ValueError("the lists are one layer's: off [E + 1], order [rows], inv [T][k]")
        ints(order, tuple(order.shape), "order")
        ints(inv, tuple(inv.shape), "inv")
        if weights is not None and (weights.dtype != torch.float32 or weights.shape != inv.shape or not weights.is_contiguous() or
                                    weights.device != self.device):
            raise ValueError(f"weights have to be contiguous fp32 {tuple(inv.shape)} on {self.device}")

    def _new(self, *shape, dtype=None):
        return torch.empty(shape, dtype=dtype or self.dtype, device=self.device)

    def _gemm(self, op, out, **values):
        a = nat.make_expert_gemm(op=op, E=self.E, out=out, dtype="e4m3" if self.eight else self._name(),
                                 out_dtype="f32" if out.dtype == torch.float32 else self._name(), **values)
        nat.moer_expert_gemm(a, self.ws, self.ws_bytes, self.stream)
        return out

    def _combine(self, z, inv, weights, add):
        T, k = inv.shape
        out = self._new(T, self.H)
        nat.moer_expert_combine(nat.make_expert_combine(T=T, H=self.H, k=k, rows=z.shape[0], dtype=self._name(), z=z, inv=inv, weights=weights,
                                                        add=add, out=out), self.ws, self.ws_bytes, self.stream)
        return out

    # ------------------------------------------------------------------ norm
    def norm(self, x, residual=None):
        """(y, sum, rstd): the norm's output, the residual stream x + residual, and what norm_grad
        needs.  With 8-bit weights y is (e4m3 rows, scales, 16-bit rows): the first two for
        `forward`, the last for the router's gate."""
        if self.norm_weight is None:
            raise ValueError("the layer was made without a norm's weight")
        self._rows(x, self.H, "x")
        T = x.shape[0]
        if residual is not None:
            self._rows(residual, self.H, "residual", T)
        self._takes(x, residual)
        with self._on_stream():
            y, rstd = self._new(T, self.H), self._new(T, dtype=torch.float32)
            s = x if residual is None else self._new(T, self.H)
            q, scale = (self._new(T, self.H, dtype=torch.float8_e4m3fn), self._new(T, -(-self.H // 128), dtype=torch.float32)) if self.eight else (None, None)
            nat.moer_rms_norm(nat.make_norm(T=T, H=self.H, dtype=self._name(), eps=self.eps, x=x, residual=residual, weight=self.norm_weight,
                                            sum=s if residual is not None else None, y=y, q=q, scale=scale, rstd=rstd), None, 0, self.stream)
        self._results(*(t for t in (y, s, rstd, q, scale) if t is not None))
        return (y if not self.eight else (q, scale, y)), s, rstd

    def norm_grad(self, s, rstd, d_y, d_sum=None):
        """(d_x, d_weight): the gradient by x and the residual alike, and by the norm's weight."""
        if self.norm_weight is None:
            raise ValueError("the layer was made without a norm's weight")
        T = s.shape[0]
        for t, what in ((s, "sum"), (d_y, "d_y"), (d_sum, "d_sum")):
            if t is not None:
                self._rows(t, self.H, what, T)
        if rstd.shape != (T,) or rstd.dtype != torch.float32 or not rstd.is_contiguous() or rstd.device != self.device:
            raise ValueError(f"rstd has to be contiguous fp32 of {T} on {self.device}")
        self._takes(s, rstd, d_y, d_sum)
        with self._on_stream():
            d_x, d_w = self._new(T, self.H), self._new(self.H, dtype=torch.float32)
            ws = self._new(nat.moer_rms_norm_workspace_bytes(T, self.H), dtype=torch.uint8)
            nat.moer_rms_norm_grad(nat.make_norm(T=T, H=self.H, dtype=self._name(), eps=self.eps, sum=s, weight=self.norm_weight, rstd=rstd, d_y=d_y,
                                                 d_sum=d_sum, d_x=d_x, d_weight=d_w), ws, ws.numel(), self.stream)
        return self._results(d_x, d_w)

    # --------------------------------------------------------------- experts
    def forward(self, x, off, order, inv, weights=None, add=None):
        """(out, kept): the combined outputs [T][H] of rows x [T][H] (8-bit weights: of a pair of e4m3
        rows and scales, as `norm` gives them), on top of `add` if given, and what `backward` needs
        (None with 8-bit weights)."""
        self._lists(off, order, inv, weights)
        T, rows, k = inv.shape[0], order.shape[0], inv.shape[1]
        if self.eight:
            x, sx = x[0], x[1]
            self._rows(x, self.H, "x", T, torch.float8_e4m3fn)
            self._rows(sx, -(-self.H // 128), "x's scales", T, torch.float32)
        else:
            self._rows(x, self.H, "x", T)
        if add is not None:
            self._rows(add, self.H, "add", T)
        used = off[self.E:]
        self._takes(x, sx if self.eight else None, off, order, inv, weights, add)
        with self._on_stream():
            lists = dict(expert_off=off, rows=rows)
            h = self._gemm("forward", self._new(rows, 2 * self.I), N=2 * self.I, K=self.H, k=k, tokens=T, order=order, x=x, w=self.w1, **lists,
                           **({"x_scale": sx, "w_scale": self.scales[0]} if self.eight else {}))
            act = dict(rows=rows, I=self.I, dtype=self._name(), h=h, used=used)
            if self.eight:
                a, sa = self._new(rows, self.I, dtype=torch.float8_e4m3fn), self._new(rows, -(-self.I // 128), dtype=torch.float32)
                nat.moer_expert_act(nat.make_expert_act(q=a, scale=sa, **act), self.stream)
                more = {"x_scale": sa, "w_scale": self.scales[1]}
            else:
                a, more = self._new(rows, self.I), {}
                nat.moer_expert_act(nat.make_expert_act(y=a, **act), self.stream)
            z = self._gemm("forward", self._new(rows, self.H), N=self.H, K=self.I, tokens=rows, x=a, w=self.w2, **lists, **more)
            out = self._combine(z, inv, weights, add)
            # its own copy of the weights: those of weights_for lie in the router's one buffer, which the next batch overwrites
            kept = None if self.eight else ExpertPass(x, h, a, z, off, order, inv, None if weights is None else weights.detach().clone())
        self._results(out)
        return out, kept

    def backward(self, kept: ExpertPass, d_out):
        """The gradients of a forward pass, by name: x [T][H], w1 and w2 (fp32) and weights [T][k]
        (that of `add` is d_out itself)."""
        if self.eight:
            raise ValueError("8-bit weights serve only")
        off, order, inv, (T, k), rows = kept.off, kept.order, kept.inv, kept.inv.shape, kept.order.shape[0]
        self._rows(d_out, self.H, "d_out", T)
        self._takes(d_out)
        with self._on_stream():
            f32 = torch.float32
            lists = dict(expert_off=off, rows=rows)
            d_z, d_weights = self._new(rows, self.H), self._new(T, k, dtype=f32)
            nat.moer_expert_combine_grad(nat.make_expert_combine(
                T=T, H=self.H, k=k, rows=rows, dtype=self._name(), z=kept.z, inv=inv, order=order, weights=kept.weights, d_out=d_out, d_z=d_z,
                d_weights=d_weights), self.ws, self.ws_bytes, self.stream)
            w2 = dict(N=self.H, K=self.I, tokens=rows)
            d_a = self._gemm("grad_input", self._new(rows, self.I), x=d_z, w=self.w2, **w2, **lists)
            d_w2 = self._gemm("grad_weight", self._new(self.E, self.H, self.I, dtype=f32), x=kept.a, d_y=d_z, **w2, **lists)
            d_h = self._new(rows, 2 * self.I)
            nat.moer_expert_act_grad(nat.make_expert_act(rows=rows, I=self.I, dtype=self._name(), h=kept.h, used=off[self.E:], d_y=d_a, d_h=d_h),
                                     self.stream)
            w1 = dict(N=2 * self.I, K=self.H)
            d_w1 = self._gemm("grad_weight", self._new(self.E, 2 * self.I, self.H, dtype=f32), tokens=T, k=k, order=order, x=kept.x, d_y=d_h, **w1, **lists)
            d_rows = self._gemm("grad_input", self._new(rows, self.H), tokens=rows, x=d_h, w=self.w1, **w1, **lists)
            d_x = self._combine(d_rows, inv, None, None)
        self._results(d_x, d_w1, d_w2, d_weights)
        return {"x": d_x, "w1": d_w1, "w2": d_w2, "weights": d_weights}

    def status(self) -> int:
        return nat.moer_ws_status(self.ws, self.stream)


@dataclasses.dataclass
class Calibration:
    """What the offline half of the method hands to serving (device tensors unless noted)."""
    mask: np.ndarray          # host [m] sorted layer ids: the signature's layer mask
    mask_order: np.ndarray    # host [m] the layers in the order the greedy selection chose them
    quality: np.ndarray       # host [m] fp64 proxy quality after each addition
    idf: torch.Tensor         # [m][E] fp32 idf of the mask layers
    sig: torch.Tensor         # [N][m*E] fp32 signatures of the calibration prompts
    centroids: torch.Tensor   # [D][m*E] fp32 balanced K-means centroids: one per decoder
    assign: torch.Tensor      # [N] int32 cluster of each calibration prompt
    kmeans_info: np.ndarray   # host [3] steps, cancellations, step-bound flag
    affinity: torch.Tensor    # [L][E][E] int32 co-activation over the calibration prompts
    group_of: torch.Tensor    # [L][E] int32 spectral expert groups
    knee: np.ndarray          # host [L] knee grid point of each layer's grouping


def calibrate(E, k, L, block, logits, bd: BatchDev, req_off, *, m, D, G, seed_rows, max_iter=100,
              tau=0.1, device="cuda", stream=None) -> Calibration:
    """The offline calibration on the GPU, call by call: the prompts' top-k ids, per-block
    counts and co-activation over every layer (moer_topk_signature), their request counts
    (moer_block_stitch) and idf (moer_idf_fit); the greedy layer mask (moer_mask_select);
    the counts, idf and count.idf signatures over that mask (moer_ids_signature,
    moer_block_stitch, moer_idf_fit, moer_route with one zero centroid, whose choice is
    not used); the balanced K-means centroids from the rows `seed_rows` of those
    signatures (moer_kmeans_balanced); and the spectral expert groups of the
    co-activation (moer_spectral_groups).  This function orders calls and holds buffers;
    the arithmetic is the library's.

    logits [L][T][E] fp32 (device) and bd / req_off (host [R+1]) describe the calibration
    prompts, one request each, without prefix reuse."""
    dev = torch.device(device)
    st = stream if stream is not None else torch.cuda.current_stream(dev)
    f32, i32, u8 = torch.float32, torch.int32, torch.uint8
    T, R, nblk = bd.T, bd.R, bd.nblk
    d_all = nat.make_dims(E, k, L, list(range(L)), block)
    topk = torch.empty((L, T, k), dtype=u8, device=dev)
    blk_all = torch.empty((nblk, L, E), dtype=u8, device=dev)
    aff = torch.zeros((L, E, E), dtype=i32, device=dev)
    wsb = nat.moer_workspace_bytes(d_all, T, nblk, R, 1)
    ws = torch.zeros(wsb, dtype=u8, device=dev)
    nat.moer_topk_signature(d_all, logits, T, bd.blk_tab, nblk, topk, blk_all, aff, ws, wsb, st)
    req_all = torch.empty((R, L, E), dtype=i32, device=dev)
    nat.moer_block_stitch(d_all, blk_all, bd.blk_tab, nblk, bd.req_blk_off, R, None, 0, None, None, 0,
                          None, req_all, ws, wsb, st)
    del blk_all
    idf_all = torch.empty((L, E), dtype=f32, device=dev)
    nat.moer_idf_fit(d_all, req_all, R, idf_all, st)
    del req_all
    # the greedy layer mask
    d_sel = nat.make_dims(E, k, L, [], block)
    mask_order = torch.empty(m, dtype=i32, device=dev)
    quality = torch.empty(m, dtype=torch.float64, device=dev)
    msb = nat.moer_mask_select_workspace_bytes(d_sel, R)
    ms_ws = torch.zeros(msb, dtype=u8, device=dev)
    off = torch.as_tensor(np.asarray(req_off, dtype=np.int32)).to(dev)
    nat.moer_mask_select(d_sel, topk, T, off, R, idf_all, m, mask_order, quality, ms_ws, msb, st)
    order = mask_order.cpu().numpy()
    mask = np.sort(order)  # the dims take the mask as a sorted host array
    # counts, idf and signatures over the mask
    d_m = nat.make_dims(E, k, L, mask.tolist(), block)
    blk_m = torch.empty((nblk, m, E), dtype=u8, device=dev)
    nat.moer_ids_signature(d_m, topk, T, bd.blk_tab, nblk, blk_m, None, ws, wsb, st)
    req_m = torch.empty((R, m, E), dtype=i32, device=dev)
    nat.moer_block_stitch(d_m, blk_m, bd.blk_tab, nblk, bd.req_blk_off, R, None, 0, None, None, 0, None,
                          req_m, ws, wsb, st)
    idf_m = torch.empty((m, E), dtype=f32, device=dev)
    nat.moer_idf_fit(d_m, req_m, R, idf_m, st)
    sig = torch.empty((R, m * E), dtype=f32, device=dev)
    zero_c = torch.zeros((1, m * E), dtype=f32, device=dev)
    zero_l = torch.zeros(1, dtype=i32, device=dev)
    unused = torch.empty(R, dtype=i32, device=dev)
    nat.moer_route(d_m, req_m, R, idf_m, zero_c, 1, tau, zero_l, 0, sig, None, unused, None, 0, st)
    # balanced K-means from the caller's seed rows
    init = sig.index_select(0, torch.as_tensor(np.asarray(seed_rows, dtype=np.int64)).to(dev)).contiguous()
    cent = torch.empty((D, m * E), dtype=f32, device=dev)
    assign = torch.empty(R, dtype=i32, device=dev)
    info = torch.zeros(3, dtype=i32, device=dev)
    kmb = nat.moer_kmeans_workspace_bytes(R, m * E, D)
    km_ws = torch.zeros(kmb, dtype=u8, device=dev)
    nat.moer_kmeans_balanced(sig, R, m * E, D, init, max_iter, cent, assign, info, None, km_ws, kmb, st)
    # spectral expert groups of the co-activation
    group_of = torch.empty((L, E), dtype=i32, device=dev)
    knee = torch.empty(L, dtype=i32, device=dev)
    u = torch.empty((L, 17), dtype=torch.float64, device=dev)
    s = torch.empty((L, 17), dtype=torch.float64, device=dev)
    spb = nat.moer_spectral_workspace_bytes(d_all, G)
    sp_ws = torch.zeros(spb, dtype=u8, device=dev)
    nat.moer_spectral_groups(d_all, aff, G, group_of, knee, u, s, sp_ws, spb, st)
    for w in (ws, ms_ws, km_ws, sp_ws):
        code = nat.moer_ws_status(w, st)
        if code != 0:
            raise nat.MoerError("calibrate", code, nat.moer_status_str(code))
    return Calibration(mask=mask, mask_order=order, quality=quality.cpu().numpy(), idf=idf_m, sig=sig,
                       centroids=cent, assign=assign, kmeans_info=info.cpu().numpy(), affinity=aff,
                       group_of=group_of, knee=knee.cpu().numpy())


# ---------------------------------------------------------------- artefacts
CALIB_MAGIC = b"MOERCAL1"
CALIB_VERSION = 1
_CALIB_HEADER = "<8s8Id"  # magic, version, E, k, L, m, D, G, block, tau


def save_calibration(path, cal: Calibration, *, E, k, L, block, G, tau) -> None:
    """Writes what serving needs from a calibration, as little-endian binary: a header
    (magic, version, E, k, L, m, D, G, block, tau), then the mask int32 [m], idf fp32 [m][E],
    centroids fp32 [D][m*E] and expert groups int32 [L][E], then a CRC-32 of all of it.
    The calibration must be refitted when the model, the traffic or the decoder count changes;
    the file only carries it from the offline fit to the serving process."""
    import struct
    import zlib
    mask = np.ascontiguousarray(cal.mask, dtype="<i4")
    idf = np.ascontiguousarray(cal.idf.cpu().numpy() if torch.is_tensor(cal.idf) else cal.idf, dtype="<f4")
    cen = np.ascontiguousarray(cal.centroids.cpu().numpy() if torch.is_tensor(cal.centroids) else cal.centroids,
                               dtype="<f4")
    grp = np.ascontiguousarray(cal.group_of.cpu().numpy() if torch.is_tensor(cal.group_of) else cal.group_of,
                               dtype="<i4")
    m, D = int(mask.shape[0]), int(cen.shape[0])
    if idf.shape != (m, E) or cen.shape != (D, m * E) or grp.shape != (L, E):
        raise ValueError("calibration arrays do not match E, L and the mask")
    if grp.size and (grp.min() < 0 or grp.max() >= G):
        raise ValueError("expert group ids outside [0, G)")
    body = struct.pack(_CALIB_HEADER, CALIB_MAGIC, CALIB_VERSION, E, k, L, m, D, G, block, float(tau))
    body += mask.tobytes() + idf.tobytes() + cen.tobytes() + grp.tobytes()
    with open(path, "wb") as f:
        f.write(body + struct.pack("<I", zlib.crc32(body)))


def load_calibration(path) -> dict:
    """Reads a file written by save_calibration; raises ValueError when the magic, the
    version, the sizes or the CRC do not match.  Returns the header fields and host arrays
    (mask, idf, centroids, group_of), ready for RoutingStats."""
    import struct
    import zlib
    with open(path, "rb") as f:
        data = f.read()
    hs = struct.calcsize(_CALIB_HEADER)
    if len(data) < hs + 4:
        raise ValueError("calibration file too short")
    magic, ver, E, k, L, m, D, G, block, tau = struct.unpack_from(_CALIB_HEADER, data, 0)
    if magic != CALIB_MAGIC or ver != CALIB_VERSION:
        raise ValueError("not a calibration file of this version")
    sizes = [m * 4, m * E * 4, D * m * E * 4, L * E * 4]
    if len(data) != hs + sum(sizes) + 4:
        raise ValueError("calibration file size does not match its header")
    (crc,) = struct.unpack_from("<I", data, len(data) - 4)
    if zlib.crc32(data[:-4]) != crc:
        raise ValueError("calibration file checksum mismatch")
    off = hs
    out = {"E": E, "k": k, "L": L, "m": m, "D": D, "G": G, "block": block, "tau": tau}
    for name, n, dt, shape in (("mask", sizes[0], "<i4", (m,)), ("idf", sizes[1], "<f4", (m, E)),
                               ("centroids", sizes[2], "<f4", (D, m * E)), ("group_of", sizes[3], "<i4", (L, E))):
        out[name] = np.frombuffer(data, dtype=dt, count=n // 4, offset=off).reshape(shape).astype(dt[1:])
        off += n
    return out
