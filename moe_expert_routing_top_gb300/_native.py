"""ctypes binding of libmoeroute's C ABI (argument marshalling only).

Every function here has the name of the C entry point it calls and forwards
device pointers (torch tensors' `data_ptr()`), sizes and the CUDA stream
handle.  There is no fallback: if the shared library is missing the import
fails, and a non-zero status raises `MoerError`.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("MOER_LIBRARY", os.path.join(HERE, "_build", "libmoeroute.so"))

STATUS = {0: "MOER_OK", 1: "MOER_EINVAL", 2: "MOER_ESHAPE", 3: "MOER_ERANGE", 4: "MOER_ECUDA",
          5: "MOER_ENOMEM", 6: "MOER_EDATA", 7: "MOER_ETIMEOUT", 8: "MOER_EEXTENT"}


class MoerError(RuntimeError):
    def __init__(self, fn: str, code: int, text: str):
        super().__init__(f"{fn} failed: {STATUS.get(code, code)} ({text})")
        self.code = code


class moer_dims(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int32), ("k", ctypes.c_int32), ("L", ctypes.c_int32),
                ("m", ctypes.c_int32), ("mask", ctypes.POINTER(ctypes.c_int32)),
                ("block", ctypes.c_int32)]


class moer_score_opts(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("score", ctypes.c_int32), ("renorm", ctypes.c_int32),
                ("n_group", ctypes.c_int32), ("top_group", ctypes.c_int32), ("group_best", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class moer_block_plan_args(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("R", "block")] + [("T", ctypes.c_int64)] +
                [(n, ctypes.c_int32) for n in ("nblk", "ncached", "ld_pages", "n_free")] +
                [(n, ctypes.c_void_p) for n in ("new_len", "ctx_len", "pages", "free_pages", "req_off", "req_blk_off",
                                                "blk_tab", "insert_slot", "req_cache_off", "cache_idx", "slot_map",
                                                "tok_req", "tok_pos", "totals")])


def _fields(i32="", i64="", ptr="", f32="", order=None):
    kinds = {n: t for names, t in ((i32, ctypes.c_int32), (i64, ctypes.c_int64), (f32, ctypes.c_float), (ptr, ctypes.c_void_p))
             for n in names.split()}
    return [(n, kinds[n]) for n in (order or " ".join((i32, i64, f32, ptr))).split()]


class moer_norm_args(ctypes.Structure):
    _fields_ = _fields(i64="T ld_x ld_residual ld_sum ld_y ld_q ld_scale ld_d_y ld_d_sum ld_d_x", i32="H dtype", f32="eps",
                       ptr="x residual weight sum y q scale rstd d_y d_sum d_x d_weight",
                       order="T H dtype eps ld_x ld_residual ld_sum ld_y ld_q ld_scale ld_d_y ld_d_sum ld_d_x "
                             "x residual weight sum y q scale rstd d_y d_sum d_x d_weight")


class moer_expert_gemm_args(ctypes.Structure):
    _fields_ = _fields(i32="op E N K k dtype out_dtype", i64="rows tokens ld_x ld_d_y ld_w ld_out stride_w stride_out ld_x_scale",
                       ptr="expert_off order x x_scale w w_scale d_y out")


class moer_expert_act_args(ctypes.Structure):
    _fields_ = _fields(i64="rows ld_h ld_y ld_q ld_scale ld_d_y ld_d_h", i32="I dtype", ptr="used h y q scale d_y d_h",
                       order="rows I dtype ld_h ld_y ld_q ld_scale ld_d_y ld_d_h used h y q scale d_y d_h")


class moer_expert_combine_args(ctypes.Structure):
    _fields_ = _fields(i64="T rows ld_z ld_add ld_out ld_d_out ld_d_z", i32="H k dtype",
                       ptr="inv order weights z add out d_out d_z d_weights",
                       order="T H k rows dtype ld_z ld_add ld_out ld_d_out ld_d_z inv order weights z add out d_out d_z d_weights")


DTYPES = {"f32": 0, "bf16": 1, "f16": 2, "e4m3": 3}
GEMM_OPS = {"forward": 0, "grad_input": 1, "grad_weight": 2}
SCORES = {"softmax": 0, "sigmoid": 1}


def make_score_opts(dtype="f32", score="softmax", renorm=True, n_group=1, top_group=1, group_best=1,
                    scale=1.0) -> moer_score_opts:
    """Options of a scored gate; `dtype` and `score` by name (DTYPES, SCORES) or by number."""
    return moer_score_opts(DTYPES.get(dtype, dtype), SCORES.get(score, score), int(renorm), n_group, top_group,
                           group_best, scale)


def make_block_plan(*, R, block, T=0, nblk=0, ncached=0, ld_pages=0, n_free=0, **buffers) -> moer_block_plan_args:
    """Arguments of moer_block_plan; the buffers (tensors or addresses, by field name) are kept
    alive on the struct."""
    a = moer_block_plan_args(R=R, block=block, T=T, nblk=nblk, ncached=ncached, ld_pages=ld_pages, n_free=n_free)
    names = {n for n, t in moer_block_plan_args._fields_ if t is ctypes.c_void_p}
    for n, x in buffers.items():
        if n not in names:
            raise TypeError(f"moer_block_plan has no buffer {n!r}")
        setattr(a, n, _ptr(x))
    a._keepalive = buffers
    return a


def _make(cls, values, strides):
    """A struct of arguments from values, tensors and addresses by field name.  A tensor's row
    stride goes to its ld field unless that is given; its elements in a row have to be contiguous.
    The buffers are kept alive on the struct."""
    a, kinds = cls(), dict(cls._fields_)
    for n, x in values.items():
        if n not in kinds:
            raise TypeError(f"{cls.__name__} has no field {n!r}")
        if kinds[n] is not ctypes.c_void_p:
            setattr(a, n, DTYPES.get(x, x) if n in ("dtype", "out_dtype") else GEMM_OPS.get(x, x) if n == "op" else x)
            continue
        setattr(a, n, _ptr(x))
        if n in strides and hasattr(x, "stride"):
            if x.dim() < 2 or x.shape[-1] > 1 and x.stride(-1) != 1:
                raise ValueError(f"{n}: the elements of a row have to be contiguous")
            for ld, dim in strides[n]:
                if ld not in values and x.dim() >= -dim:
                    setattr(a, ld, max(x.stride(dim), x.shape[-1]) if x.shape[dim] == 1 else x.stride(dim))
        elif hasattr(x, "is_contiguous") and not x.is_contiguous():
            raise ValueError(f"{n} has to be contiguous")
    a._keepalive = values
    return a


def _rows_of(*names):
    return {n: [("ld_" + n, -2)] for n in names}


def make_norm(**values) -> moer_norm_args:
    """Arguments of moer_rms_norm and moer_rms_norm_grad by field name (dtype by name or number)."""
    return _make(moer_norm_args, values, _rows_of("x", "residual", "sum", "y", "q", "scale", "d_y", "d_sum", "d_x"))


def make_expert_gemm(**values) -> moer_expert_gemm_args:
    """Arguments of moer_expert_gemm by field name (op and types by name or number)."""
    return _make(moer_expert_gemm_args, values,
                 {**_rows_of("x", "d_y", "x_scale"), "w": [("ld_w", -2), ("stride_w", -3)], "out": [("ld_out", -2), ("stride_out", -3)]})


def make_expert_act(**values) -> moer_expert_act_args:
    """Arguments of moer_expert_act and moer_expert_act_grad by field name."""
    return _make(moer_expert_act_args, values, _rows_of("h", "y", "q", "scale", "d_y", "d_h"))


def make_expert_combine(**values) -> moer_expert_combine_args:
    """Arguments of moer_expert_combine and moer_expert_combine_grad by field name."""
    return _make(moer_expert_combine_args, values, _rows_of("z", "add", "out", "d_out", "d_z"))


def make_dims(E: int, k: int, L: int, mask, block: int = 16) -> moer_dims:
    """Builds the dims struct; the mask array is kept alive on the struct."""
    mask = [int(x) for x in mask]
    arr = (ctypes.c_int32 * max(len(mask), 1))(*mask)
    d = moer_dims(E, k, L, len(mask), ctypes.cast(arr, ctypes.POINTER(ctypes.c_int32)), block)
    d._mask_keepalive = arr
    return d


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libmoeroute is not built ({LIB_PATH} missing); run "
                          "`python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                             ctypes.c_size_t)
    dp = ctypes.POINTER(moer_dims)
    op = ctypes.POINTER(moer_score_opts)
    sigs = {
        "moer_workspace_bytes": ([dp, i64, i32, i32, i32], sz),
        "moer_topk_signature": ([dp, vp, i64, vp, i32, vp, vp, vp, vp, sz, vp], ctypes.c_int),
        "moer_topk_signature_noalloc": ([dp, vp, i64, vp, i32, vp, vp, vp, vp], ctypes.c_int),
        "moer_block_stitch": ([dp, vp, vp, i32, vp, i32, vp, i32, vp, vp, i32, vp, vp, vp, sz, vp],
                              ctypes.c_int),
        "moer_affinity_load": ([dp, vp, vp, i32, vp, vp, vp, vp, vp], ctypes.c_int),
        "moer_route": ([dp, vp, i32, vp, vp, i32, f32, vp, i32, vp, vp, vp, vp, sz, vp],
                       ctypes.c_int),
        "moer_idf_fit": ([dp, vp, i32, vp, vp], ctypes.c_int),
        "moer_gate_workspace_bytes": ([dp, i32], sz),
        "moer_gate_topk": ([dp, vp, i64, i32, vp, vp, i32, vp, vp, vp, vp, vp, sz, vp], ctypes.c_int),
        "moer_ids_signature": ([dp, vp, i64, vp, i32, vp, vp, vp, sz, vp], ctypes.c_int),
        "moer_spectral_workspace_bytes": ([dp, i32], sz),
        "moer_spectral_groups": ([dp, vp, i32, vp, vp, vp, vp, vp, sz, vp], ctypes.c_int),
        "moer_mask_select_workspace_bytes": ([dp, i32], sz),
        "moer_mask_select": ([dp, vp, i64, vp, i32, vp, i32, vp, vp, vp, sz, vp], ctypes.c_int),
        "moer_replication_plan": ([dp, vp, vp, i32, vp, vp, vp, vp, vp, vp, sz, vp], ctypes.c_int),
        "moer_kmeans_workspace_bytes": ([i32, i32, i32], sz),
        "moer_kmeans_balanced": ([vp, i32, i32, i32, vp, i32, vp, vp, vp, vp, vp, sz, vp], ctypes.c_int),
        "moer_score_workspace_bytes": ([dp, i64], sz),
        "moer_score_topk": ([dp, op, vp, i64, i64, i64, vp, vp, vp, vp, vp, sz, vp], ctypes.c_int),
        "moer_score_topk_grad": ([dp, op, vp, i64, i64, i64, vp, vp, vp, vp, i64, i64, vp, sz, vp], ctypes.c_int),
        "moer_block_plan_workspace_bytes": ([i32], sz),
        "moer_block_plan": ([ctypes.POINTER(moer_block_plan_args), vp, sz, vp], ctypes.c_int),
        "moer_expert_order_workspace_bytes": ([dp, i64], sz),
        "moer_expert_order": ([dp, vp, i64, i32, vp, vp, i64, vp, vp, sz, vp], ctypes.c_int),
        "moer_rms_norm_workspace_bytes": ([i64, i32], sz),
        "moer_rms_norm": ([ctypes.POINTER(moer_norm_args), vp, sz, vp], ctypes.c_int),
        "moer_rms_norm_grad": ([ctypes.POINTER(moer_norm_args), vp, sz, vp], ctypes.c_int),
        "moer_expert_gemm_workspace_bytes": ([ctypes.POINTER(moer_expert_gemm_args)], sz),
        "moer_expert_gemm": ([ctypes.POINTER(moer_expert_gemm_args), vp, sz, vp], ctypes.c_int),
        "moer_expert_act": ([ctypes.POINTER(moer_expert_act_args), vp], ctypes.c_int),
        "moer_expert_act_grad": ([ctypes.POINTER(moer_expert_act_args), vp], ctypes.c_int),
        "moer_expert_combine": ([ctypes.POINTER(moer_expert_combine_args), vp, sz, vp], ctypes.c_int),
        "moer_expert_combine_grad": ([ctypes.POINTER(moer_expert_combine_args), vp, sz, vp], ctypes.c_int),
        "moer_ws_status": ([vp, vp], ctypes.c_int),
        "moer_wait_selftest": ([vp, sz, ctypes.c_uint32, vp], ctypes.c_int),
        "moer_status_str": ([ctypes.c_int], ctypes.c_char_p),
        "moer_version": ([], ctypes.c_int32),
        "moer_set_extent_checks": ([i32], None),
        "moer_extent_checks": ([], ctypes.c_int32),
        "moer_buffer_holds": ([vp, sz], ctypes.c_int32),
    }
    for name, (args, res) in sigs.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    return lib


LIB = _load()
EXPORTS = ("moer_workspace_bytes", "moer_topk_signature", "moer_topk_signature_noalloc",
           "moer_block_stitch", "moer_affinity_load",
           "moer_route", "moer_idf_fit", "moer_gate_workspace_bytes", "moer_gate_topk",
           "moer_ids_signature",
           "moer_replication_plan", "moer_kmeans_workspace_bytes", "moer_kmeans_balanced",
           "moer_mask_select_workspace_bytes", "moer_mask_select", "moer_spectral_workspace_bytes",
           "moer_spectral_groups",
           "moer_score_workspace_bytes", "moer_score_topk", "moer_score_topk_grad",
           "moer_block_plan_workspace_bytes", "moer_block_plan",
           "moer_expert_order_workspace_bytes", "moer_expert_order",
           "moer_rms_norm_workspace_bytes", "moer_rms_norm", "moer_rms_norm_grad",
           "moer_expert_gemm_workspace_bytes", "moer_expert_gemm", "moer_expert_act", "moer_expert_act_grad",
           "moer_expert_combine", "moer_expert_combine_grad",
           "moer_ws_status", "moer_wait_selftest",
           "moer_status_str", "moer_version", "moer_set_extent_checks", "moer_extent_checks",
           "moer_buffer_holds")


def _ptr(x):
    return x if x is None or isinstance(x, int) else x.data_ptr()


_current = None  # (current device, its current stream's handle), bound at the first call without a stream


def current_handle(index=None) -> int:
    """The handle of the current stream of a device (the current one, if none is given), without
    the stream object that torch.cuda.current_stream() makes (0.2 instead of 2.9 us a call, a
    third of a small call's time on the host)."""
    global _current
    if _current is None:
        import torch
        torch.cuda.init()
        _current = (torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream)
    return _current[1](_current[0]() if index is None else index)


def _stream(s):
    if s is None:
        return current_handle()
    return s if isinstance(s, int) else s.cuda_stream


def _check(fn: str, code: int) -> None:
    if code != 0:
        raise MoerError(fn, code, LIB.moer_status_str(code).decode())


def moer_workspace_bytes(dims, T: int = 0, nblk: int = 0, R: int = 0, D: int = 0) -> int:
    return int(LIB.moer_workspace_bytes(ctypes.byref(dims), T, nblk, R, D))


def moer_topk_signature(dims, logits, T, blk_tab, nblk, topk, blk_cnt, affinity, ws, ws_bytes,
                        stream=None) -> None:
    _check("moer_topk_signature", LIB.moer_topk_signature(
        ctypes.byref(dims), _ptr(logits), int(T), _ptr(blk_tab), int(nblk), _ptr(topk),
        _ptr(blk_cnt), _ptr(affinity), _ptr(ws), int(ws_bytes), _stream(stream)))


def moer_topk_signature_noalloc(dims, logits, T, blk_tab, nblk, topk, blk_cnt, affinity,
                                stream=None) -> None:
    """moer_topk_signature without a workspace: the scratch is a fixed array inside the library,
    for callers that cannot allocate device memory (see include/moeroute.h)."""
    _check("moer_topk_signature_noalloc", LIB.moer_topk_signature_noalloc(
        ctypes.byref(dims), _ptr(logits), int(T), _ptr(blk_tab), int(nblk), _ptr(topk),
        _ptr(blk_cnt), _ptr(affinity), _stream(stream)))


def moer_block_stitch(dims, blk_cnt, blk_tab, nblk, req_blk_off, R, cache_idx, ncached, req_cache_off,
                      cache, nslots, insert_slot, req_cnt, ws, ws_bytes, stream=None) -> None:
    _check("moer_block_stitch", LIB.moer_block_stitch(
        ctypes.byref(dims), _ptr(blk_cnt), _ptr(blk_tab), int(nblk), _ptr(req_blk_off), int(R),
        _ptr(cache_idx), int(ncached), _ptr(req_cache_off), _ptr(cache), int(nslots), _ptr(insert_slot),
        _ptr(req_cnt), _ptr(ws), int(ws_bytes), _stream(stream)))


def moer_affinity_load(dims, affinity, group_of, G, W_expert, W_group, rho_group, rho_expert,
                       stream=None) -> None:
    _check("moer_affinity_load", LIB.moer_affinity_load(
        ctypes.byref(dims), _ptr(affinity), _ptr(group_of), int(G), _ptr(W_expert),
        _ptr(W_group), _ptr(rho_group), _ptr(rho_expert), _stream(stream)))


def moer_route(dims, req_cnt, R, idf, centroids, D, tau, loads, live, sig, dist, choice, ws,
               ws_bytes, stream=None) -> None:
    _check("moer_route", LIB.moer_route(
        ctypes.byref(dims), _ptr(req_cnt), int(R), _ptr(idf), _ptr(centroids), int(D),
        float(tau), _ptr(loads), int(live), _ptr(sig), _ptr(dist), _ptr(choice), _ptr(ws),
        int(ws_bytes), _stream(stream)))


def moer_idf_fit(dims, req_cnt, R, idf, stream=None) -> None:
    _check("moer_idf_fit", LIB.moer_idf_fit(ctypes.byref(dims), _ptr(req_cnt), int(R), _ptr(idf),
                                            _stream(stream)))


def moer_spectral_workspace_bytes(dims, G: int) -> int:
    return int(LIB.moer_spectral_workspace_bytes(ctypes.byref(dims), int(G)))


def moer_spectral_groups(dims, affinity, G, group_of, knee, u_curve, s_curve, ws, ws_bytes,
                         stream=None) -> None:
    _check("moer_spectral_groups", LIB.moer_spectral_groups(
        ctypes.byref(dims), _ptr(affinity), int(G), _ptr(group_of), _ptr(knee), _ptr(u_curve),
        _ptr(s_curve), _ptr(ws), int(ws_bytes), _stream(stream)))


def moer_mask_select_workspace_bytes(dims, R: int) -> int:
    return int(LIB.moer_mask_select_workspace_bytes(ctypes.byref(dims), int(R)))


def moer_mask_select(dims, topk, T, req_off, R, idf, m, mask_out, quality_out, ws, ws_bytes,
                     stream=None) -> None:
    _check("moer_mask_select", LIB.moer_mask_select(
        ctypes.byref(dims), _ptr(topk), int(T), _ptr(req_off), int(R), _ptr(idf), int(m),
        _ptr(mask_out), _ptr(quality_out), _ptr(ws), int(ws_bytes), _stream(stream)))


def moer_replication_plan(dims, W, group_of, G, n_rep, src, hot, dst, w_pred, ws, ws_bytes,
                          stream=None) -> None:
    _check("moer_replication_plan", LIB.moer_replication_plan(
        ctypes.byref(dims), _ptr(W), _ptr(group_of), int(G), _ptr(n_rep), _ptr(src), _ptr(hot),
        _ptr(dst), _ptr(w_pred), _ptr(ws), int(ws_bytes), _stream(stream)))


def moer_kmeans_workspace_bytes(N: int, dim: int, D: int) -> int:
    return int(LIB.moer_kmeans_workspace_bytes(int(N), int(dim), int(D)))


def moer_kmeans_balanced(sig, N, dim, D, init_centroids, max_iter, centroids, assign, info, objective,
                         ws, ws_bytes, stream=None) -> None:
    _check("moer_kmeans_balanced", LIB.moer_kmeans_balanced(
        _ptr(sig), int(N), int(dim), int(D), _ptr(init_centroids), int(max_iter), _ptr(centroids),
        _ptr(assign), _ptr(info), _ptr(objective), _ptr(ws), int(ws_bytes), _stream(stream)))


def moer_gate_workspace_bytes(dims, H: int) -> int:
    return int(LIB.moer_gate_workspace_bytes(ctypes.byref(dims), int(H)))


def moer_gate_topk(dims, hidden, T, H, w_gate, blk_tab, nblk, logits, topk, blk_cnt, affinity, ws,
                   ws_bytes, stream=None) -> None:
    _check("moer_gate_topk", LIB.moer_gate_topk(
        ctypes.byref(dims), _ptr(hidden), int(T), int(H), _ptr(w_gate), _ptr(blk_tab), int(nblk),
        _ptr(logits), _ptr(topk), _ptr(blk_cnt), _ptr(affinity), _ptr(ws), int(ws_bytes),
        _stream(stream)))


def moer_ids_signature(dims, topk, T, blk_tab, nblk, blk_cnt, affinity, ws, ws_bytes, stream=None) -> None:
    _check("moer_ids_signature", LIB.moer_ids_signature(
        ctypes.byref(dims), _ptr(topk), int(T), _ptr(blk_tab), int(nblk), _ptr(blk_cnt), _ptr(affinity),
        _ptr(ws), int(ws_bytes), _stream(stream)))


def moer_score_workspace_bytes(dims, T: int) -> int:
    return int(LIB.moer_score_workspace_bytes(ctypes.byref(dims), int(T)))


def moer_score_topk(dims, opts, logits, T, ld_token, ld_layer, bias, topk, weights, score_sum, ws, ws_bytes,
                    stream=None) -> None:
    _check("moer_score_topk", LIB.moer_score_topk(
        ctypes.byref(dims), ctypes.byref(opts), _ptr(logits), int(T), int(ld_token), int(ld_layer), _ptr(bias),
        _ptr(topk), _ptr(weights), _ptr(score_sum), _ptr(ws), int(ws_bytes), _stream(stream)))


def moer_score_topk_grad(dims, opts, logits, T, ld_token, ld_layer, topk, d_weights, d_score_sum, d_logits,
                         ldg_token, ldg_layer, ws, ws_bytes, stream=None) -> None:
    _check("moer_score_topk_grad", LIB.moer_score_topk_grad(
        ctypes.byref(dims), ctypes.byref(opts), _ptr(logits), int(T), int(ld_token), int(ld_layer), _ptr(topk),
        _ptr(d_weights), _ptr(d_score_sum), _ptr(d_logits), int(ldg_token), int(ldg_layer), _ptr(ws),
        int(ws_bytes), _stream(stream)))


def moer_block_plan_workspace_bytes(R: int) -> int:
    return int(LIB.moer_block_plan_workspace_bytes(int(R)))


def moer_block_plan(args, ws, ws_bytes, stream=None) -> None:
    """The tables of a batch from its requests' lengths; `args` from make_block_plan."""
    _check("moer_block_plan", LIB.moer_block_plan(ctypes.byref(args), _ptr(ws), int(ws_bytes), _stream(stream)))


def moer_expert_order_workspace_bytes(dims, T: int) -> int:
    return int(LIB.moer_expert_order_workspace_bytes(ctypes.byref(dims), int(T)))


def moer_expert_order(dims, topk, T, align, expert_off, order, ld_order, inv, ws, ws_bytes, stream=None) -> None:
    _check("moer_expert_order", LIB.moer_expert_order(
        ctypes.byref(dims), _ptr(topk), int(T), int(align), _ptr(expert_off), _ptr(order), int(ld_order),
        _ptr(inv), _ptr(ws), int(ws_bytes), _stream(stream)))


def moer_rms_norm_workspace_bytes(T: int, H: int) -> int:
    return int(LIB.moer_rms_norm_workspace_bytes(int(T), int(H)))


def moer_rms_norm(args, ws=None, ws_bytes=0, stream=None) -> None:
    """Residual addition, norm and 8-bit rows; `args` from make_norm."""
    _check("moer_rms_norm", LIB.moer_rms_norm(ctypes.byref(args), _ptr(ws), int(ws_bytes), _stream(stream)))


def moer_rms_norm_grad(args, ws, ws_bytes, stream=None) -> None:
    _check("moer_rms_norm_grad", LIB.moer_rms_norm_grad(ctypes.byref(args), _ptr(ws), int(ws_bytes), _stream(stream)))


def moer_expert_gemm_workspace_bytes(args) -> int:
    return int(LIB.moer_expert_gemm_workspace_bytes(ctypes.byref(args)))


def moer_expert_gemm(args, ws, ws_bytes, stream=None) -> None:
    """The experts' products over their token lists; `args` from make_expert_gemm."""
    _check("moer_expert_gemm", LIB.moer_expert_gemm(ctypes.byref(args), _ptr(ws), int(ws_bytes), _stream(stream)))


def moer_expert_act(args, stream=None) -> None:
    """Gated activation of the experts' rows; `args` from make_expert_act."""
    _check("moer_expert_act", LIB.moer_expert_act(ctypes.byref(args), _stream(stream)))


def moer_expert_act_grad(args, stream=None) -> None:
    _check("moer_expert_act_grad", LIB.moer_expert_act_grad(ctypes.byref(args), _stream(stream)))


def moer_expert_combine(args, ws, ws_bytes, stream=None) -> None:
    """The experts' rows back to their tokens; `args` from make_expert_combine."""
    _check("moer_expert_combine", LIB.moer_expert_combine(ctypes.byref(args), _ptr(ws), int(ws_bytes), _stream(stream)))


def moer_expert_combine_grad(args, ws, ws_bytes, stream=None) -> None:
    _check("moer_expert_combine_grad", LIB.moer_expert_combine_grad(ctypes.byref(args), _ptr(ws), int(ws_bytes),
                                                                   _stream(stream)))


def moer_ws_status(ws, stream=None) -> int:
    """Waits for the stream and returns (and clears) the workspace status code."""
    return int(LIB.moer_ws_status(_ptr(ws), _stream(stream)))


def moer_wait_selftest(ws, ws_bytes, limit_us, stream=None) -> None:
    """One kernel whose bounded wait cannot complete: it gives up after limit_us and
    records MOER_ETIMEOUT in ws (read it with moer_ws_status)."""
    _check("moer_wait_selftest", LIB.moer_wait_selftest(_ptr(ws), int(ws_bytes), int(limit_us), _stream(stream)))


def moer_status_str(code: int) -> str:
    return LIB.moer_status_str(int(code)).decode()


def moer_version() -> int:
    return int(LIB.moer_version())


def moer_set_extent_checks(on: bool) -> None:
    LIB.moer_set_extent_checks(1 if on else 0)


def moer_extent_checks() -> bool:
    return bool(LIB.moer_extent_checks())


def moer_buffer_holds(p, nbytes: int) -> bool:
    """Host-side: whether one device allocation holds [p, p + nbytes)."""
    return bool(LIB.moer_buffer_holds(_ptr(p), nbytes))
