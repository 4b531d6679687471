"""GB300 (sm_103a) draft-correction library: thin Python binding of include/dcoco.h.

Every function here only marshals arguments (tensor data pointers, sizes,
the current CUDA stream) into the C ABI of libdcoco.so; every step of the
correction path runs in the library's CUDA kernels.  There is no CPU path:
importing the binding without the built library raises.

Build the library first:  python draft_correction_slot_gb300/build.py
"""
from __future__ import annotations

import ctypes as C
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libdcoco.so")

DCOCO_OK = 0
DCOCO_EINVAL = -1
DCOCO_EUNSUPPORTED = -2
DCOCO_EBATCH = -3
DCOCO_ECUDA = -4
DCOCO_ENOMEM = -5
DCOCO_EDEVICE = -6


class DcocoError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {dcoco_status_string(status)} ({status})")
        self.status = status


class dcoco_config(C.Structure):
    _fields_ = [("vocab", C.c_int), ("hidden", C.c_int), ("slots", C.c_int), ("topk", C.c_int),
                ("rank", C.c_int), ("mlp_hidden", C.c_int), ("max_batch", C.c_int),
                ("variant", C.c_int), ("sigma", C.c_float), ("ln_eps", C.c_float),
                ("host_staging", C.c_int), ("path_rule", C.c_int), ("beam_width", C.c_int),
                ("beam_topm", C.c_int)]


WEIGHT_NAMES = ("w_cand", "w_ctx", "w_fuse", "ln_gamma", "ln_beta", "w_pair", "w1", "b1", "w2",
                "b2", "w_io")


class dcoco_weight_ptrs(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in WEIGHT_NAMES] + [("on_device", C.c_int)]


class dcoco_inputs(C.Structure):
    _fields_ = [("logits", C.c_void_p), ("logits_slot_stride", C.c_int64), ("hidden", C.c_void_p),
                ("cand_embed", C.c_void_p), ("target_tokens", C.c_void_p)]


class dcoco_outputs(C.Structure):
    _fields_ = [("tokens", C.c_void_p), ("choice", C.c_void_p), ("scores", C.c_void_p),
                ("accept_len", C.c_void_p), ("topk_ids", C.c_void_p), ("topk_val", C.c_void_p),
                ("margin", C.c_void_p), ("cand_feat", C.c_void_p)]


EXPORTED = ("dcoco_version", "dcoco_status_string", "dcoco_create", "dcoco_weights_create",
            "dcoco_correct", "dcoco_correct_host", "dcoco_topk", "dcoco_get_device_status",
            "dcoco_selftest_wait_timeout",
            "dcoco_weights_destroy", "dcoco_destroy", "dcoco_kernel_launches",
            "dcoco_stage_timing", "dcoco_stage_read", "dcoco_stage_name", "dcoco_topk_noalloc",
            "dcoco_topk_noalloc_plan", "dcoco_verify_stochastic", "dcoco_host_range_covers",
            "dcoco_tree_create", "dcoco_tree_attention", "dcoco_tree_commit", "dcoco_tree_status",
            "dcoco_tree_launches", "dcoco_tree_destroy", "dcoco_sample", "dcoco_distill_loss",
            "dcoco_distill_grad", "dcoco_distill_step", "dcoco_tree_create_quant", "dcoco_tree_attention_quant",
            "dcoco_tree_commit_quant", "dcoco_tree_append_quant", "dcoco_pages_create", "dcoco_pages_reserve",
            "dcoco_pages_fork", "dcoco_pages_free", "dcoco_pages_compact", "dcoco_pages_status",
            "dcoco_pages_launches", "dcoco_pages_destroy")

DCOCO_BF16, DCOCO_FP16, DCOCO_FP32 = 0, 1, 2
_DTYPE = {torch.bfloat16: DCOCO_BF16, torch.float16: DCOCO_FP16, torch.float32: DCOCO_FP32}


class dcoco_tree_config(C.Structure):
    _fields_ = [(n, C.c_int) for n in ("max_batch", "max_tree", "q_heads", "kv_heads", "head_dim", "page_size",
                                       "max_pages", "dtype")]


def _strided(name, *axes):
    return [(name, C.c_void_p)] + [(f"{name}_stride_{a}", C.c_int64) for a in axes]


class dcoco_tree_attention_args(C.Structure):
    _fields_ = (_strided("q", "n", "t", "h") + _strided("k_new", "n", "t", "h") + _strided("v_new", "n", "t", "h")
                + _strided("k_cache", "page", "token", "h") + _strided("v_cache", "page", "token", "h")
                + [("page_table", C.c_void_p), ("page_table_stride", C.c_int64), ("ctx_len", C.c_void_p),
                   ("tree_len", C.c_void_p), ("tree_mask", C.c_void_p), ("tree_mask_stride_n", C.c_int64),
                   ("num_pages", C.c_int), ("scale", C.c_float)])


class dcoco_tree_commit_args(C.Structure):
    _fields_ = ([(n, C.c_void_p) for n in ("tokens", "parents", "sampled", "tree_len", "ctx_len", "page_table")]
                + [("page_table_stride", C.c_int64)]
                + _strided("k_new", "l", "n", "t", "h") + _strided("v_new", "l", "n", "t", "h")
                + _strided("k_cache", "l", "page", "token", "h") + _strided("v_cache", "l", "page", "token", "h")
                + [("num_pages", C.c_int), ("layers", C.c_int)])


class dcoco_quant_scales(C.Structure):
    _fields_ = _strided("k_scale", "l", "page", "block", "h") + _strided("v_scale", "l", "page", "block", "h")


class dcoco_tree_append_args(C.Structure):
    _fields_ = ([(n, C.c_void_p) for n in ("first", "ctx_len", "page_table")] + [("page_table_stride", C.c_int64)]
                + _strided("k_new", "l", "t", "h") + _strided("v_new", "l", "t", "h")
                + _strided("k_cache", "l", "page", "token", "h") + _strided("v_cache", "l", "page", "token", "h")
                + [("num_pages", C.c_int), ("layers", C.c_int), ("tokens", C.c_int)])


class dcoco_pages_config(C.Structure):
    _fields_ = [(n, C.c_int) for n in ("num_pages", "page_size", "max_pages", "max_rows")]


class dcoco_pages_state(C.Structure):
    _fields_ = [("page_table", C.c_void_p), ("page_table_stride", C.c_int64), ("held", C.c_void_p),
                ("len", C.c_void_p), ("refs", C.c_void_p)]


class dcoco_page_plane(C.Structure):
    _fields_ = [("base", C.c_void_p), ("layer_stride", C.c_int64), ("page_stride", C.c_int64),
                ("page_bytes", C.c_int64), ("layers", C.c_int)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python draft_correction_slot_gb300/build.py` (there is no CPU fallback)")
    L = C.CDLL(LIB_PATH)
    L.dcoco_version.restype = C.c_int
    L.dcoco_status_string.argtypes = [C.c_int]
    L.dcoco_status_string.restype = C.c_char_p
    L.dcoco_create.argtypes = [C.POINTER(dcoco_config), C.POINTER(C.c_void_p)]
    L.dcoco_weights_create.argtypes = [C.c_void_p, C.POINTER(dcoco_weight_ptrs), C.c_void_p,
                                       C.POINTER(C.c_void_p)]
    for f in (L.dcoco_correct, L.dcoco_correct_host):
        f.argtypes = [C.c_void_p, C.c_void_p, C.c_int, C.POINTER(dcoco_inputs),
                      C.POINTER(dcoco_outputs), C.c_void_p]
    L.dcoco_verify_stochastic.argtypes = [C.c_void_p, C.c_int, C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p,
                                          C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p]
    L.dcoco_topk.argtypes = [C.c_void_p, C.c_int, C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p,
                             C.c_void_p]
    L.dcoco_topk_noalloc.argtypes = [C.c_int, C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_int64,
                                     C.c_void_p, C.c_void_p, C.c_void_p]
    L.dcoco_topk_noalloc_plan.argtypes = [C.c_int, C.c_int, C.c_int, C.c_int, C.POINTER(C.c_int),
                                          C.POINTER(C.c_int)]
    L.dcoco_host_range_covers.argtypes = [C.c_uint64, C.c_uint64, C.c_uint64, C.c_uint64]
    L.dcoco_get_device_status.argtypes = [C.c_void_p]
    L.dcoco_selftest_wait_timeout.argtypes = [C.c_void_p, C.c_longlong, C.c_void_p]
    L.dcoco_weights_destroy.argtypes = [C.c_void_p]
    L.dcoco_weights_destroy.restype = None
    L.dcoco_destroy.argtypes = [C.c_void_p]
    L.dcoco_destroy.restype = None
    L.dcoco_kernel_launches.argtypes = [C.c_void_p]
    L.dcoco_kernel_launches.restype = C.c_longlong
    L.dcoco_stage_timing.argtypes = [C.c_void_p, C.c_int]
    L.dcoco_stage_read.argtypes = [C.c_void_p, C.c_int, C.POINTER(C.c_float), C.POINTER(C.c_int),
                                   C.POINTER(C.c_int)]
    L.dcoco_stage_name.argtypes = [C.c_void_p, C.c_int]
    L.dcoco_stage_name.restype = C.c_char_p
    P, I, I64, F = C.c_void_p, C.c_int, C.c_int64, C.c_float
    L.dcoco_tree_create.argtypes = [C.POINTER(dcoco_tree_config), C.POINTER(P)]
    L.dcoco_tree_attention.argtypes = [P, I, I, P, P, P, P]
    L.dcoco_tree_commit.argtypes = [P, I, I, P, P, P, P, P, P]
    L.dcoco_tree_status.argtypes = [P]
    L.dcoco_tree_launches.argtypes = [P]
    L.dcoco_tree_launches.restype = C.c_longlong
    L.dcoco_tree_destroy.argtypes = [P]
    L.dcoco_tree_destroy.restype = None
    L.dcoco_tree_create_quant.argtypes = [C.POINTER(dcoco_tree_config), I, C.POINTER(P)]
    L.dcoco_tree_attention_quant.argtypes = [P, I, I, P, P, P, P, P]
    L.dcoco_tree_commit_quant.argtypes = [P, I, I, P, P, P, P, P, P, P]
    L.dcoco_tree_append_quant.argtypes = [P, I, P, P, P, P]
    L.dcoco_pages_create.argtypes = [C.POINTER(dcoco_pages_config), C.POINTER(P)]
    L.dcoco_pages_reserve.argtypes = [P, P, I, P, P, P, P]
    L.dcoco_pages_fork.argtypes = [P, P, I, P, I, P, P, P, P]
    L.dcoco_pages_free.argtypes = [P, P, I, P, P]
    L.dcoco_pages_compact.argtypes = [P, P, I, P, P, I64, P, P, P]
    L.dcoco_pages_status.argtypes = [P]
    L.dcoco_pages_launches.argtypes = [P]
    L.dcoco_pages_launches.restype = C.c_longlong
    L.dcoco_pages_destroy.argtypes = [P]
    L.dcoco_pages_destroy.restype = None
    L.dcoco_sample.argtypes = [I, I, P, I, I64, P, P, P, P, P, P, P, P]
    teacher = [I, I, P, I, I64, I, P, P, P, F]
    L.dcoco_distill_loss.argtypes = teacher + [P, P, P]
    L.dcoco_distill_grad.argtypes = teacher + [P, P, P, I64, P]
    L.dcoco_distill_step.argtypes = teacher + [P, P, P, P, I64, P]
    return L


_lib = _load()


def lib():
    return _lib


def _check(rc: int, what: str):
    if rc != DCOCO_OK:
        raise DcocoError(rc, what)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        return t.data_ptr()
    return int(t)


# the current stream's handle, without the Stream object around it where torch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int | None:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


# ------------------------------------------------------------------ C ABI, same names
def dcoco_version() -> int:
    return _lib.dcoco_version()


def dcoco_status_string(status: int) -> str:
    return _lib.dcoco_status_string(status).decode()


def dcoco_create(vocab: int, hidden: int, slots: int = 16, topk: int = 16, max_batch: int = 32,
                 variant: int = 0, sigma: float = 1.0, ln_eps: float = 1e-5, rank: int = 128,
                 mlp_hidden: int = 256, host_staging: bool = False, path_rule: int = 0,
                 beam_width: int = 2, beam_topm: int = 0) -> C.c_void_p:
    """path_rule 0: prefix-first greedy walk; 1: highest-scoring path; 2: beam walk
    (beam_width partial paths, beam_topm successors each, 0 = all)."""
    cfg = dcoco_config(vocab, hidden, slots, topk, rank, mlp_hidden, max_batch, variant, sigma, ln_eps,
                       int(host_staging), int(path_rule), int(beam_width), int(beam_topm))
    h = C.c_void_p()
    _check(_lib.dcoco_create(C.byref(cfg), C.byref(h)), "dcoco_create")
    return h


def dcoco_weights_create(handle, weights: dict, stream=None) -> C.c_void_p:
    """weights: name -> fp32 tensor (all on the GPU, or all on the CPU)."""
    keep = {}
    on_dev = None
    for n in WEIGHT_NAMES:
        t = weights.get(n)
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            t = torch.as_tensor(t)
        t = t.detach().to(torch.float32).contiguous()
        dev = t.is_cuda
        if on_dev is None:
            on_dev = dev
        elif on_dev != dev:
            raise ValueError("weights must all be on the GPU or all on the CPU")
        keep[n] = t
    ptrs = dcoco_weight_ptrs(*[_ptr(keep.get(n)) for n in WEIGHT_NAMES], int(bool(on_dev)))
    w = C.c_void_p()
    _check(_lib.dcoco_weights_create(handle, C.byref(ptrs), _stream(stream) if on_dev else None,
                                     C.byref(w)), "dcoco_weights_create")
    return w


def _io(logits, hidden, cand_embed, target_tokens, logits_slot_stride, outs):
    stride = logits_slot_stride if logits_slot_stride is not None else logits.shape[-1]
    ins = dcoco_inputs(_ptr(logits), int(stride), _ptr(hidden), _ptr(cand_embed), _ptr(target_tokens))
    o = dcoco_outputs(*[_ptr(outs.get(k)) for k in ("tokens", "choice", "scores", "accept_len",
                                                    "topk_ids", "topk_val", "margin", "cand_feat")])
    return ins, o


def dcoco_correct(handle, weights, batch: int, logits, hidden, cand_embed, target_tokens=None, *,
                  tokens, choice=None, scores=None, accept_len=None, topk_ids=None, topk_val=None,
                  margin=None, cand_feat=None, logits_slot_stride: int | None = None, stream=None) -> None:
    """Device buffers in, device buffers out (see include/dcoco.h for layouts)."""
    ins, o = _io(logits, hidden, cand_embed, target_tokens, logits_slot_stride,
                 dict(tokens=tokens, choice=choice, scores=scores, accept_len=accept_len,
                      topk_ids=topk_ids, topk_val=topk_val, margin=margin, cand_feat=cand_feat))
    _check(_lib.dcoco_correct(handle, weights, batch, C.byref(ins), C.byref(o), _stream(stream)),
           "dcoco_correct")


def dcoco_correct_host(handle, weights, batch: int, logits, hidden, cand_embed, target_tokens=None,
                       *, tokens, choice=None, scores=None, accept_len=None, topk_ids=None,
                       topk_val=None, margin=None, logits_slot_stride: int | None = None,
                       stream=None) -> None:
    """Host (ideally pinned) logits/hidden/targets/outputs; cand_embed stays on the device."""
    ins, o = _io(logits, hidden, cand_embed, target_tokens, logits_slot_stride,
                 dict(tokens=tokens, choice=choice, scores=scores, accept_len=accept_len,
                      topk_ids=topk_ids, topk_val=topk_val, margin=margin))
    _check(_lib.dcoco_correct_host(handle, weights, batch, C.byref(ins), C.byref(o), _stream(stream)),
           "dcoco_correct_host")


def dcoco_topk(handle, batch: int, logits, topk_ids, topk_val, logits_slot_stride: int | None = None,
               stream=None) -> None:
    stride = logits_slot_stride if logits_slot_stride is not None else logits.shape[-1]
    _check(_lib.dcoco_topk(handle, batch, _ptr(logits), int(stride), _ptr(topk_ids), _ptr(topk_val),
                           _stream(stream)), "dcoco_topk")


def dcoco_verify_stochastic(handle, batch: int, target_logits, tokens, u_accept, u_draw, accept_len,
                            next_token, q_accept=None, target_stride: int | None = None, stream=None) -> None:
    """Stochastic verification (temperature 1) of the proposal `tokens` against
    target_logits [batch, B+1, stride] (bf16), with caller-drawn uniforms."""
    stride = target_stride if target_stride is not None else target_logits.shape[-1]
    _check(_lib.dcoco_verify_stochastic(handle, batch, _ptr(target_logits), int(stride), _ptr(tokens),
                                        _ptr(u_accept), _ptr(u_draw), _ptr(accept_len), _ptr(next_token),
                                        _ptr(q_accept) if q_accept is not None else None, _stream(stream)),
           "dcoco_verify_stochastic")


def dcoco_topk_noalloc(batch: int, slots: int, vocab: int, topk: int, logits, topk_ids, topk_val,
                       logits_slot_stride: int | None = None, stream=None) -> None:
    """Step 1 without a handle and without any device allocation (for callers
    that cannot allocate); same results as dcoco_topk."""
    stride = logits_slot_stride if logits_slot_stride is not None else logits.shape[-1]
    _check(_lib.dcoco_topk_noalloc(batch, slots, vocab, topk, _ptr(logits), int(stride), _ptr(topk_ids),
                                   _ptr(topk_val), _stream(stream)), "dcoco_topk_noalloc")


def dcoco_topk_noalloc_plan(batch: int, slots: int, vocab: int, topk: int) -> tuple[int, int]:
    """-> (segments per row dcoco_topk_noalloc would use, segments dcoco_topk would use)."""
    seg, planned = C.c_int(), C.c_int()
    _check(_lib.dcoco_topk_noalloc_plan(batch, slots, vocab, topk, C.byref(seg), C.byref(planned)),
           "dcoco_topk_noalloc_plan")
    return seg.value, planned.value


def dcoco_host_range_covers(range_start: int, range_size: int, ptr: int, nbytes: int) -> bool:
    """Whether [ptr, ptr + nbytes) lies inside the range (the host entry's in-place test)."""
    return bool(_lib.dcoco_host_range_covers(range_start, range_size, ptr, nbytes))


def dcoco_get_device_status(handle) -> int:
    return _lib.dcoco_get_device_status(handle)


def dcoco_selftest_wait_timeout(handle, limit_ns: int, stream: int = 0) -> None:
    """One block waits on an mbarrier nothing completes, with the kernels' own
    bounded wait (limit_ns); the handle's device status then reads DCOCO_EDEVICE."""
    _check(_lib.dcoco_selftest_wait_timeout(handle, int(limit_ns), C.c_void_p(stream)),
           "dcoco_selftest_wait_timeout")


def dcoco_weights_destroy(weights) -> None:
    _lib.dcoco_weights_destroy(weights)


def dcoco_destroy(handle) -> None:
    _lib.dcoco_destroy(handle)


def dcoco_kernel_launches(handle) -> int:
    return int(_lib.dcoco_kernel_launches(handle))


def dcoco_stage_timing(handle, enable: bool) -> None:
    _check(_lib.dcoco_stage_timing(handle, int(bool(enable))), "dcoco_stage_timing")


def dcoco_stage_read(handle) -> tuple[dict, int]:
    """-> ({stage name: summed ms}, number of calls summed)."""
    ms = (C.c_float * 8)()
    calls, ns = C.c_int(), C.c_int()
    _check(_lib.dcoco_stage_read(handle, 8, ms, C.byref(calls), C.byref(ns)), "dcoco_stage_read")
    return {dcoco_stage_name(handle, s): float(ms[s]) for s in range(ns.value)}, calls.value


def dcoco_stage_name(handle, s: int) -> str | None:
    r = _lib.dcoco_stage_name(handle, s)
    return None if r is None else r.decode()


# ------------------------------------------------------------------ the target's side of a drafted block
def _dense(t, name: str, shape: tuple, dtype) -> int:
    """The pointer of a contiguous CUDA tensor of that shape and type."""
    if t.dtype is not dtype or not t.is_cuda or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor of shape {tuple(shape)}")
    return t.data_ptr()


def _dense_or_none(t, name: str, shape: tuple, dtype) -> int:
    return 0 if t is None else _dense(t, name, shape, dtype)


def _heads(t, name: str, shape: tuple, dtype) -> tuple:
    """A CUDA tensor whose last axis (a head's elements) is dense: its pointer and the other axes' strides."""
    st = t.stride()
    if t.dtype is not dtype or not t.is_cuda or t.shape != shape or st[-1] != 1:
        raise ValueError(f"{name} must be a CUDA {dtype} tensor of shape {shape} whose last axis is dense")
    return (t.data_ptr(), *st[:-1])


# the C structures as bytes (a ctypes structure takes several times as long to fill)
_ATTENTION_ARGS = struct.Struct("@" + "P3q" * 5 + "PqPPPqif")
_COMMIT_ARGS = struct.Struct("@6Pq" + "P4q" * 4 + "ii")
assert _ATTENTION_ARGS.size == C.sizeof(dcoco_tree_attention_args) and _COMMIT_ARGS.size == C.sizeof(dcoco_tree_commit_args)


class _TreeHandle(C.c_void_p):
    """A dcoco_tree_handle and the sizes it was made for."""
    sizes: tuple = ()
    scale_tokens: int = 0  # of a cache in 8 bits; 0: in 16


def dcoco_tree_create(max_batch: int, max_tree: int, q_heads: int, kv_heads: int, head_dim: int, page_size: int,
                      max_pages: int, dtype: torch.dtype = torch.bfloat16) -> _TreeHandle:
    """Handle of the tree calls for one attention layout; see include/dcoco.h."""
    cfg = dcoco_tree_config(max_batch, max_tree, q_heads, kv_heads, head_dim, page_size, max_pages,
                            _DTYPE.get(dtype, -1))
    h = _TreeHandle()
    _check(_lib.dcoco_tree_create(C.byref(cfg), C.byref(h)), "dcoco_tree_create")
    h.sizes = (q_heads, kv_heads, head_dim, page_size, max_pages, dtype)
    return h


def _page_table(page_table, batch: int, max_pages: int) -> tuple:
    shape, st = page_table.shape, page_table.stride()
    if page_table.dtype is not torch.int32 or not page_table.is_cuda or len(shape) != 2 or shape[0] != batch \
            or shape[1] < max_pages or (st[1] != 1 and shape[1] > 1):
        raise ValueError(f"page_table must be a CUDA int32 tensor of shape ({batch}, >= {max_pages}) with dense rows")
    return page_table.data_ptr(), (st[0] if batch > 1 else max_pages)


def dcoco_tree_attention(handle, batch: int, q, k_new, v_new, k_cache, v_cache, page_table, ctx_len, *, out,
                         tree_mask=None, tree_len=None, lse=None, scale: float | None = None, stream=None) -> None:
    """Attention of batch trees of q.shape[1] nodes over a paged cache and the trees themselves.

    q [batch, nodes, q_heads, D], k_new and v_new [batch, nodes, kv_heads, D], k_cache and v_cache
    [pages, page_size, kv_heads, D] may be views (the last axis dense, strides multiples of 8);
    page_table [batch, max_pages], ctx_len and tree_len [batch] int32; tree_mask int32 words
    [batch or 1, nodes, ceil(nodes / 32)] (tree_mask() makes them from parents; None: causal);
    out [batch, nodes, q_heads, D] and lse fp32 [batch, nodes, q_heads] are written.  scale: 1/sqrt(D)."""
    hq, hkv, d, page, max_pages, dt = handle.sizes
    nodes, pages = q.shape[1], k_cache.shape[0]
    new, pool, one, i32 = (batch, nodes, hkv, d), (pages, page, hkv, d), (batch,), torch.int32
    mask_ptr = mask_stride = 0
    if tree_mask is not None:
        words = (nodes + 31) // 32
        shared = tree_mask.shape[0] == 1 and batch != 1
        mask_ptr = _dense(tree_mask, "tree_mask", (1 if shared else batch, nodes, words), i32)
        mask_stride = 0 if shared else nodes * words
    args = _ATTENTION_ARGS.pack(
        *_heads(q, "q", (batch, nodes, hq, d), dt), *_heads(k_new, "k_new", new, dt),
        *_heads(v_new, "v_new", new, dt), *_heads(k_cache, "k_cache", pool, dt),
        *_heads(v_cache, "v_cache", pool, dt), *_page_table(page_table, batch, max_pages),
        _dense(ctx_len, "ctx_len", one, i32), _dense_or_none(tree_len, "tree_len", one, i32),
        mask_ptr, mask_stride, pages, d ** -0.5 if scale is None else scale)
    _check(_lib.dcoco_tree_attention(handle, batch, nodes, args, _dense(out, "out", (batch, nodes, hq, d), dt),
                                     _dense_or_none(lse, "lse", (batch, nodes, hq), torch.float32), _stream(stream)),
           "dcoco_tree_attention")


def dcoco_tree_commit(handle, batch: int, tokens, parents, sampled, k_new, v_new, k_cache, v_cache, page_table,
                      ctx_len, *, path, accept_len, next_token, new_len, tree_len=None, stream=None) -> None:
    """Walk each tree along the target's tokens and append the path's K/V to the cache of every layer.

    tokens, parents, sampled and path int32 [batch, nodes]; k_new and v_new [layers, batch, nodes, kv_heads, D],
    k_cache and v_cache [layers, pages, page_size, kv_heads, D]; the others int32 [batch]."""
    _, hkv, d, page, max_pages, dt = handle.sizes
    nodes, layers, pages = tokens.shape[1], k_cache.shape[0], k_cache.shape[1]
    i32, tree, one = torch.int32, (batch, nodes), (batch,)
    new, pool = (layers, batch, nodes, hkv, d), (layers, pages, page, hkv, d)
    args = _COMMIT_ARGS.pack(
        _dense(tokens, "tokens", tree, i32), _dense(parents, "parents", tree, i32),
        _dense(sampled, "sampled", tree, i32), _dense_or_none(tree_len, "tree_len", one, i32),
        _dense(ctx_len, "ctx_len", one, i32), *_page_table(page_table, batch, max_pages),
        *_heads(k_new, "k_new", new, dt), *_heads(v_new, "v_new", new, dt),
        *_heads(k_cache, "k_cache", pool, dt), *_heads(v_cache, "v_cache", pool, dt), pages, layers)
    _check(_lib.dcoco_tree_commit(handle, batch, nodes, args, _dense(path, "path", tree, i32),
                                  _dense(accept_len, "accept_len", one, i32),
                                  _dense(next_token, "next_token", one, i32), _dense(new_len, "new_len", one, i32),
                                  _stream(stream)), "dcoco_tree_commit")


# the same on a cache in 8 bits
_E4M3 = torch.float8_e4m3fn
_SCALES = struct.Struct("@" + "P4q" * 2)
_APPEND_ARGS = struct.Struct("@3Pq" + "P3q" * 2 + "P4q" * 2 + "iii0q")
assert _SCALES.size == C.sizeof(dcoco_quant_scales) and _APPEND_ARGS.size == C.sizeof(dcoco_tree_append_args)


def dcoco_tree_create_quant(max_batch: int, max_tree: int, q_heads: int, kv_heads: int, head_dim: int, page_size: int,
                            max_pages: int, scale_tokens: int, dtype: torch.dtype = torch.bfloat16) -> _TreeHandle:
    """As dcoco_tree_create, for a cache of torch.float8_e4m3fn with an fp32 scale for each block of scale_tokens
    tokens and K/V head; dtype is that of q, the nodes' K/V and the outputs."""
    cfg = dcoco_tree_config(max_batch, max_tree, q_heads, kv_heads, head_dim, page_size, max_pages,
                            _DTYPE.get(dtype, -1))
    h = _TreeHandle()
    _check(_lib.dcoco_tree_create_quant(C.byref(cfg), scale_tokens, C.byref(h)), "dcoco_tree_create_quant")
    h.sizes, h.scale_tokens = (q_heads, kv_heads, head_dim, page_size, max_pages, dtype), scale_tokens
    return h


def _blocks(handle, what: str) -> int:
    """Scales of a page; refuses a handle for a cache in 16 bits."""
    if not handle.scale_tokens:
        raise DcocoError(DCOCO_EUNSUPPORTED, what)
    return handle.sizes[3] // handle.scale_tokens


def _scales(k_scale, v_scale, shape: tuple) -> bytes:
    """k_scale and v_scale of that shape ([layers,] pages, blocks, kv_heads), any positive strides."""
    packed = []
    for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if t.dtype is not torch.float32 or not t.is_cuda or t.shape != shape:
            raise ValueError(f"{name} must be a CUDA fp32 tensor of shape {tuple(shape)}")
        packed += [t.data_ptr(), *((0,) if len(shape) == 3 else ()), *t.stride()]
    return _SCALES.pack(*packed)


def dcoco_tree_attention_quant(handle, batch: int, q, k_new, v_new, k_cache, v_cache, k_scale, v_scale, page_table,
                               ctx_len, *, out, tree_mask=None, tree_len=None, lse=None, scale: float | None = None,
                               stream=None) -> None:
    """dcoco_tree_attention on k_cache and v_cache of torch.float8_e4m3fn (strides multiples of 16) with k_scale and
    v_scale fp32 [pages, page_size / scale_tokens, kv_heads]."""
    blocks = _blocks(handle, "dcoco_tree_attention_quant")
    hq, hkv, d, page, max_pages, dt = handle.sizes
    nodes, pages = q.shape[1], k_cache.shape[0]
    new, pool, one, i32 = (batch, nodes, hkv, d), (pages, page, hkv, d), (batch,), torch.int32
    mask_ptr = mask_stride = 0
    if tree_mask is not None:
        words = (nodes + 31) // 32
        shared = tree_mask.shape[0] == 1 and batch != 1
        mask_ptr = _dense(tree_mask, "tree_mask", (1 if shared else batch, nodes, words), i32)
        mask_stride = 0 if shared else nodes * words
    args = _ATTENTION_ARGS.pack(
        *_heads(q, "q", (batch, nodes, hq, d), dt), *_heads(k_new, "k_new", new, dt),
        *_heads(v_new, "v_new", new, dt), *_heads(k_cache, "k_cache", pool, _E4M3),
        *_heads(v_cache, "v_cache", pool, _E4M3), *_page_table(page_table, batch, max_pages),
        _dense(ctx_len, "ctx_len", one, i32), _dense_or_none(tree_len, "tree_len", one, i32),
        mask_ptr, mask_stride, pages, d ** -0.5 if scale is None else scale)
    _check(_lib.dcoco_tree_attention_quant(
        handle, batch, nodes, args, _scales(k_scale, v_scale, (pages, blocks, hkv)),
        _dense(out, "out", (batch, nodes, hq, d), dt), _dense_or_none(lse, "lse", (batch, nodes, hq), torch.float32),
        _stream(stream)), "dcoco_tree_attention_quant")


def dcoco_tree_commit_quant(handle, batch: int, tokens, parents, sampled, k_new, v_new, k_cache, v_cache, k_scale,
                            v_scale, page_table, ctx_len, *, path, accept_len, next_token, new_len, tree_len=None,
                            stream=None) -> None:
    """dcoco_tree_commit into k_cache and v_cache of torch.float8_e4m3fn with k_scale and v_scale fp32
    [layers, pages, page_size / scale_tokens, kv_heads], both written."""
    blocks = _blocks(handle, "dcoco_tree_commit_quant")
    _, hkv, d, page, max_pages, dt = handle.sizes
    nodes, layers, pages = tokens.shape[1], k_cache.shape[0], k_cache.shape[1]
    i32, tree, one = torch.int32, (batch, nodes), (batch,)
    new, pool = (layers, batch, nodes, hkv, d), (layers, pages, page, hkv, d)
    args = _COMMIT_ARGS.pack(
        _dense(tokens, "tokens", tree, i32), _dense(parents, "parents", tree, i32),
        _dense(sampled, "sampled", tree, i32), _dense_or_none(tree_len, "tree_len", one, i32),
        _dense(ctx_len, "ctx_len", one, i32), *_page_table(page_table, batch, max_pages),
        *_heads(k_new, "k_new", new, dt), *_heads(v_new, "v_new", new, dt),
        *_heads(k_cache, "k_cache", pool, _E4M3), *_heads(v_cache, "v_cache", pool, _E4M3), pages, layers)
    _check(_lib.dcoco_tree_commit_quant(
        handle, batch, nodes, args, _scales(k_scale, v_scale, (layers, pages, blocks, hkv)),
        _dense(path, "path", tree, i32), _dense(accept_len, "accept_len", one, i32),
        _dense(next_token, "next_token", one, i32), _dense(new_len, "new_len", one, i32), _stream(stream)),
        "dcoco_tree_commit_quant")


def dcoco_tree_append_quant(handle, batch: int, first, k_new, v_new, k_cache, v_cache, k_scale, v_scale, page_table,
                            ctx_len, *, new_len, stream=None) -> None:
    """Append ragged prompts: request n's tokens are rows first[n] .. first[n + 1] - 1 of k_new and v_new
    [layers, rows, kv_heads, D]; first int32 [batch + 1], ctx_len and new_len int32 [batch], the rest as above."""
    blocks = _blocks(handle, "dcoco_tree_append_quant")
    _, hkv, d, page, max_pages, dt = handle.sizes
    layers, pages, rows = k_cache.shape[0], k_cache.shape[1], k_new.shape[1]
    i32, one, new, pool = torch.int32, (batch,), (layers, rows, hkv, d), (layers, pages, page, hkv, d)
    args = _APPEND_ARGS.pack(
        _dense(first, "first", (batch + 1,), i32), _dense(ctx_len, "ctx_len", one, i32),
        *_page_table(page_table, batch, max_pages), *_heads(k_new, "k_new", new, dt), *_heads(v_new, "v_new", new, dt),
        *_heads(k_cache, "k_cache", pool, _E4M3), *_heads(v_cache, "v_cache", pool, _E4M3), pages, layers, rows)
    _check(_lib.dcoco_tree_append_quant(handle, batch, args, _scales(k_scale, v_scale, (layers, pages, blocks, hkv)),
                                        _dense(new_len, "new_len", one, i32), _stream(stream)),
           "dcoco_tree_append_quant")


def dcoco_tree_status(handle) -> int:
    return _lib.dcoco_tree_status(handle)


def dcoco_tree_launches(handle) -> int:
    return int(_lib.dcoco_tree_launches(handle))


def dcoco_tree_destroy(handle) -> None:
    _lib.dcoco_tree_destroy(handle)


# ------------------------------------------------------------------ a cache's pages
_POOL_STATE = struct.Struct("@PqPPP")
_PLANE = struct.Struct("@PqqqiI")
assert _POOL_STATE.size == C.sizeof(dcoco_pages_state) and _PLANE.size == C.sizeof(dcoco_page_plane)


class _PagesHandle(C.c_void_p):
    """A dcoco_pages_handle and the sizes it was made for."""
    sizes: tuple = ()


def dcoco_pages_create(num_pages: int, page_size: int, max_pages: int, max_rows: int) -> _PagesHandle:
    """Handle of the page calls for one pool; see include/dcoco.h."""
    cfg = dcoco_pages_config(num_pages, page_size, max_pages, max_rows)
    h = _PagesHandle()
    _check(_lib.dcoco_pages_create(C.byref(cfg), C.byref(h)), "dcoco_pages_create")
    h.sizes = (num_pages, max_pages, max_rows)
    return h


class page_planes:
    """The tensors whose pages are copied with the pool's: [layers, pages, ...] each, what one page has of a layer
    contiguous in any order of its axes.  Keeps the tensors; make it once for a cache."""

    def __init__(self, tensors):
        self.tensors, self.pages, packed = tuple(tensors), set(), []
        for t in self.tensors:
            if not t.is_cuda or t.dim() < 3:
                raise ValueError("a plane must be a CUDA tensor [layers, pages, ...]")
            inner, dense = sorted(zip(t.stride()[2:], t.shape[2:])), 1
            for stride, n in inner:
                if n > 1 and stride != dense:
                    raise ValueError("what a page has of a layer must be contiguous")
                dense *= n
            size = t.element_size()
            self.pages.add(t.shape[1])
            packed.append(_PLANE.pack(t.data_ptr(), t.stride(0) * size, t.stride(1) * size, dense * size, t.shape[0], 0))
        if len(self.pages) > 1:
            raise ValueError("the planes must have the same number of pages")
        self.count, self.packed = len(packed), b"".join(packed)


def _pool_state(handle, page_table, held, lens, refs) -> bytes:
    pages, max_pages, rows = handle.sizes
    i32 = torch.int32
    return _POOL_STATE.pack(*_page_table(page_table, rows, max_pages), _dense(held, "held", (rows,), i32),
                            _dense_or_none(lens, "lens", (rows,), i32), _dense(refs, "refs", (pages,), i32))


def _planes_for(handle, planes) -> tuple:
    if planes.count and planes.pages != {handle.sizes[0]}:
        raise ValueError(f"the planes must have {handle.sizes[0]} pages")
    return planes.count, planes.packed


def _row_list(rows, name: str) -> tuple:
    """The shape of a list of rows: one axis."""
    if rows.dim() != 1:
        raise ValueError(f"{name} must have one axis")
    return rows.shape


def dcoco_pages_reserve(handle, rows, tokens, page_table, held, refs, *, done=None, stream=None) -> None:
    """Give each listed row pages for so many tokens.  rows, tokens and done int32 [count]; the pool's state:
    page_table int32 [max_rows, >= max_pages], held int32 [max_rows], refs int32 [num_pages]."""
    n, i32 = _row_list(rows, "rows"), torch.int32
    _check(_lib.dcoco_pages_reserve(handle, _pool_state(handle, page_table, held, None, refs), n[0],
                                    _dense(rows, "rows", n, i32), _dense(tokens, "tokens", n, i32),
                                    _dense_or_none(done, "done", n, i32), _stream(stream)), "dcoco_pages_reserve")


def dcoco_pages_fork(handle, planes, src, dst, page_table, held, lens, refs, *, done=None, stream=None) -> None:
    """Rows dst become copies of rows src (int32 [count]): full pages shared, the partly filled one copied in all
    planes.  lens int32 [max_rows]: the rows' tokens."""
    n, i32 = _row_list(src, "src"), torch.int32
    _check(_lib.dcoco_pages_fork(handle, _pool_state(handle, page_table, held, lens, refs), *_planes_for(handle, planes),
                                 n[0], _dense(src, "src", n, i32), _dense(dst, "dst", n, i32),
                                 _dense_or_none(done, "done", n, i32), _stream(stream)), "dcoco_pages_fork")


def dcoco_pages_free(handle, rows, page_table, held, lens, refs, *, stream=None) -> None:
    """The listed rows (int32 [count]) hold nothing any more."""
    n = _row_list(rows, "rows")
    _check(_lib.dcoco_pages_free(handle, _pool_state(handle, page_table, held, lens, refs), n[0],
                                 _dense(rows, "rows", n, torch.int32), _stream(stream)), "dcoco_pages_free")


def dcoco_pages_compact(handle, planes, page_table, held, refs, *, live, page_table_out=None, refs_out=None,
                        stream=None) -> None:
    """Move the pages in use to the front.  live int32 [1]; page_table_out and refs_out: the state's own where None."""
    table_out, refs_to = page_table if page_table_out is None else page_table_out, refs if refs_out is None else refs_out
    pages, max_pages, rows = handle.sizes
    _check(_lib.dcoco_pages_compact(handle, _pool_state(handle, page_table, held, None, refs),
                                    *_planes_for(handle, planes), *_page_table(table_out, rows, max_pages),
                                    _dense(refs_to, "refs_out", (pages,), torch.int32),
                                    _dense(live, "live", (1,), torch.int32), _stream(stream)), "dcoco_pages_compact")


def dcoco_pages_status(handle) -> int:
    return _lib.dcoco_pages_status(handle)


def dcoco_pages_launches(handle) -> int:
    return int(_lib.dcoco_pages_launches(handle))


def dcoco_pages_destroy(handle) -> None:
    _lib.dcoco_pages_destroy(handle)


def _logit_rows(logits, name: str = "logits") -> tuple:
    """[rows, vocab] with dense rows: (rows, vocab, pointer, dtype code, row stride)."""
    dt, shape, st = logits.dtype, logits.shape, logits.stride()
    if len(shape) != 2 or not logits.is_cuda or (dt is not torch.bfloat16 and dt is not torch.float32) \
            or (st[1] != 1 and shape[1] > 1):
        raise ValueError(f"{name} must be a CUDA bf16 or fp32 [rows, vocab] tensor with dense rows")
    rows, vocab = shape
    # (one row's stride is never used: any that passes)
    return rows, vocab, logits.data_ptr(), _DTYPE[dt], st[0] if rows > 1 else (vocab + 7) // 8 * 8


def dcoco_sample(logits, u, tokens, *, temperature=None, top_k=None, top_p=None, min_p=None, logprob=None,
                 stream=None) -> None:
    """One token per row of logits [rows, vocab] (bf16 or fp32, row stride a multiple of 8), from uniforms u
    [rows]; temperature, top_p, min_p fp32 and top_k int32 [rows] or None; tokens int32, logprob fp32 [rows]."""
    rows, vocab, ptr, dt, stride = _logit_rows(logits)
    one, f32 = (rows,), torch.float32
    _check(_lib.dcoco_sample(rows, vocab, ptr, dt, stride, _dense_or_none(temperature, "temperature", one, f32),
                             _dense_or_none(top_k, "top_k", one, torch.int32), _dense_or_none(top_p, "top_p", one, f32),
                             _dense_or_none(min_p, "min_p", one, f32), _dense(u, "u", one, f32),
                             _dense(tokens, "tokens", one, torch.int32), _dense_or_none(logprob, "logprob", one, f32),
                             _stream(stream)), "dcoco_sample")


def _teacher(logits, teacher_ids, teacher_logits, teacher_lse, temperature):
    rows, vocab, ptr, dt, stride = _logit_rows(logits)
    if teacher_ids.dim() != 2:
        raise ValueError("teacher_ids must be [rows, topk]")
    k, f32 = teacher_ids.shape[1], torch.float32
    return (rows, vocab, ptr, dt, stride, k, _dense(teacher_ids, "teacher_ids", (rows, k), torch.int32),
            _dense(teacher_logits, "teacher_logits", (rows, k), f32),
            _dense_or_none(teacher_lse, "teacher_lse", (rows,), f32), float(temperature))


def _grad_rows(grad, logits):
    if grad.shape != logits.shape or grad.dtype is not logits.dtype:
        raise ValueError("grad must have the logits' shape and type")
    rows = _logit_rows(grad, "grad")
    return rows[2], rows[4]


def dcoco_distill_loss(logits, teacher_ids, teacher_logits, *, loss, lse, teacher_lse=None, temperature: float = 1.0,
                       stream=None) -> None:
    """Per-row distillation loss (and the log-sum-exp that the gradient needs) of logits [rows, vocab] against
    the teacher's top logits: teacher_ids int32, teacher_logits fp32 [rows, topk]; see include/dcoco.h."""
    t = _teacher(logits, teacher_ids, teacher_logits, teacher_lse, temperature)
    one = (t[0],)
    _check(_lib.dcoco_distill_loss(*t, _dense(loss, "loss", one, torch.float32), _dense(lse, "lse", one, torch.float32),
                                   _stream(stream)), "dcoco_distill_loss")


def dcoco_distill_grad(logits, teacher_ids, teacher_logits, lse, grad_loss, *, grad, teacher_lse=None,
                       temperature: float = 1.0, stream=None) -> None:
    """Gradient with respect to the logits, times grad_loss [rows], from the loss call's lse.  grad has the
    logits' shape and type and may be the logits themselves; hand it on with logits.backward(grad)."""
    t = _teacher(logits, teacher_ids, teacher_logits, teacher_lse, temperature)
    one = (t[0],)
    _check(_lib.dcoco_distill_grad(*t, _dense(lse, "lse", one, torch.float32),
                                   _dense(grad_loss, "grad_loss", one, torch.float32), *_grad_rows(grad, logits),
                                   _stream(stream)), "dcoco_distill_grad")


def dcoco_distill_step(logits, teacher_ids, teacher_logits, grad_loss, *, loss, lse, grad, teacher_lse=None,
                       temperature: float = 1.0, stream=None) -> None:
    """Loss and gradient in one pass over the logits (the rows' grad_loss known beforehand, e.g. 1 / rows)."""
    t = _teacher(logits, teacher_ids, teacher_logits, teacher_lse, temperature)
    one, f32 = (t[0],), torch.float32
    _check(_lib.dcoco_distill_step(*t, _dense(grad_loss, "grad_loss", one, f32), _dense(loss, "loss", one, f32),
                                   _dense(lse, "lse", one, f32), *_grad_rows(grad, logits), _stream(stream)),
           "dcoco_distill_step")


def tree_mask(parents) -> torch.Tensor:
    """Mask words of trees given by parents [batch, nodes] (-1: a root): node t sees its ancestors and itself."""
    n, t = parents.shape
    up = parents.long()
    words = (t + 31) // 32
    sees = torch.zeros(n, t, words * 32, dtype=torch.bool, device=parents.device)
    sees[:, :, :t] = torch.eye(t, dtype=torch.bool, device=parents.device)
    for i in range(1, t):  # a parent's row is complete before its children's
        row = sees.gather(1, up[:, i].clamp(min=0).view(n, 1, 1).expand(n, 1, words * 32))[:, 0]
        sees[:, i] |= row & (up[:, i] >= 0)[:, None]
    bits = (sees.view(n, t, words, 32).long() << torch.arange(32, device=parents.device)).sum(-1)
    return torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32)


class TreeVerifier:
    """Owns a tree handle; allocates output tensors per call.  One step of the target on a drafted tree:
    attention() in every layer, sample() on the nodes' logits, commit() for all layers at once.  max_batch is best
    near the batches that are run: the attention cuts requests for a full one (see include/dcoco.h)."""

    def __init__(self, q_heads: int, kv_heads: int, head_dim: int, page_size: int, max_pages: int, max_batch: int = 32,
                 max_tree: int = 64, dtype: torch.dtype = torch.bfloat16):
        self.handle = dcoco_tree_create(max_batch, max_tree, q_heads, kv_heads, head_dim, page_size, max_pages, dtype)

    def close(self):
        if getattr(self, "handle", None) is not None:
            dcoco_tree_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def attention(self, q, k_new, v_new, k_cache, v_cache, page_table, ctx_len, tree_mask=None, tree_len=None,
                  scale=None, stream=None):
        """-> (out [N, T, q_heads, D], lse [N, T, q_heads])"""
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
        dcoco_tree_attention(self.handle, q.shape[0], q, k_new, v_new, k_cache, v_cache, page_table, ctx_len, out=out,
                             tree_mask=tree_mask, tree_len=tree_len, lse=lse, scale=scale, stream=stream)
        return out, lse

    def sample(self, logits, u, temperature=None, top_k=None, top_p=None, min_p=None, stream=None):
        """logits [N, T, V] -> (tokens [N, T] int32, logprob [N, T]); u and the parameters [N, T] (or None)."""
        n, t, v = logits.shape
        flat = [None if x is None else x.reshape(n * t) for x in (temperature, top_k, top_p, min_p)]
        tokens = torch.empty(n, t, dtype=torch.int32, device=logits.device)
        logprob = torch.empty(n, t, dtype=torch.float32, device=logits.device)
        dcoco_sample(logits.view(n * t, v), u.reshape(n * t), tokens.view(n * t), temperature=flat[0], top_k=flat[1],
                     top_p=flat[2], min_p=flat[3], logprob=logprob.view(n * t), stream=stream)
        return tokens, logprob

    def commit(self, tokens, parents, sampled, k_new, v_new, k_cache, v_cache, page_table, ctx_len, tree_len=None,
               stream=None):
        """-> dict(path [N, T], accept_len [N], next_token [N], new_len [N]); the caches are written."""
        n, t = tokens.shape
        out = {"path": torch.empty(n, t, dtype=torch.int32, device=tokens.device)}
        for name in ("accept_len", "next_token", "new_len"):
            out[name] = torch.empty(n, dtype=torch.int32, device=tokens.device)
        dcoco_tree_commit(self.handle, n, tokens, parents, sampled, k_new, v_new, k_cache, v_cache, page_table, ctx_len,
                          tree_len=tree_len, stream=stream, **out)
        return out

    def status(self) -> int:
        return dcoco_tree_status(self.handle)


class QuantTreeVerifier(TreeVerifier):
    """A TreeVerifier on a cache in 8 bits: torch.float8_e4m3fn with an fp32 scale for each block of scale_tokens
    tokens and K/V head, [layers, pages, page_size / scale_tokens, kv_heads].  append() takes prompts."""

    def __init__(self, q_heads: int, kv_heads: int, head_dim: int, page_size: int, max_pages: int, max_batch: int = 32,
                 max_tree: int = 64, dtype: torch.dtype = torch.bfloat16, scale_tokens: int = 16):
        self.handle = dcoco_tree_create_quant(max_batch, max_tree, q_heads, kv_heads, head_dim, page_size, max_pages,
                                              scale_tokens, dtype)

    def attention(self, q, k_new, v_new, k_cache, v_cache, k_scale, v_scale, page_table, ctx_len, tree_mask=None,
                  tree_len=None, scale=None, stream=None):
        """-> (out [N, T, q_heads, D], lse [N, T, q_heads]); the cache and scales of one layer."""
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
        dcoco_tree_attention_quant(self.handle, q.shape[0], q, k_new, v_new, k_cache, v_cache, k_scale, v_scale,
                                   page_table, ctx_len, out=out, tree_mask=tree_mask, tree_len=tree_len, lse=lse,
                                   scale=scale, stream=stream)
        return out, lse

    def commit(self, tokens, parents, sampled, k_new, v_new, k_cache, v_cache, k_scale, v_scale, page_table, ctx_len,
               tree_len=None, stream=None):
        """-> dict(path [N, T], accept_len [N], next_token [N], new_len [N]); the caches and scales are written."""
        n, t = tokens.shape
        out = {"path": torch.empty(n, t, dtype=torch.int32, device=tokens.device)}
        for name in ("accept_len", "next_token", "new_len"):
            out[name] = torch.empty(n, dtype=torch.int32, device=tokens.device)
        dcoco_tree_commit_quant(self.handle, n, tokens, parents, sampled, k_new, v_new, k_cache, v_cache, k_scale,
                                v_scale, page_table, ctx_len, tree_len=tree_len, stream=stream, **out)
        return out

    def append(self, first, k_new, v_new, k_cache, v_cache, k_scale, v_scale, page_table, ctx_len, stream=None):
        """Rows first[n] .. first[n + 1] - 1 of k_new and v_new [layers, rows, kv_heads, D] onto request n. -> new_len [N]"""
        new_len = torch.empty_like(ctx_len)
        dcoco_tree_append_quant(self.handle, ctx_len.shape[0], first, k_new, v_new, k_cache, v_cache, k_scale, v_scale,
                                page_table, ctx_len, new_len=new_len, stream=stream)
        return new_len


class PagePool:
    """A pool of pages for max_rows sequences: owns a handle and the state (table [max_rows, max_pages], held, lens
    [max_rows], refs [num_pages], all int32), and copies the pages of `planes` (tensors [layers, pages, ...])."""

    def __init__(self, planes, page_size: int, max_pages: int, max_rows: int):
        self.planes = page_planes(planes)
        first = self.planes.tensors[0]
        i32 = dict(dtype=torch.int32, device=first.device)
        self.handle = dcoco_pages_create(first.shape[1], page_size, max_pages, max_rows)
        self.table = torch.zeros(max_rows, max_pages, **i32)
        self.held, self.lens = torch.zeros(max_rows, **i32), torch.zeros(max_rows, **i32)
        self.refs, self.live = torch.zeros(first.shape[1], **i32), torch.zeros(1, **i32)

    def close(self):
        if getattr(self, "handle", None) is not None:
            dcoco_pages_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def reserve(self, rows, tokens, stream=None):
        """-> done [count]: 1 where the row has pages for so many tokens."""
        done = torch.empty_like(rows)
        dcoco_pages_reserve(self.handle, rows, tokens, self.table, self.held, self.refs, done=done, stream=stream)
        return done

    def fork(self, src, dst, stream=None):
        """-> done [count]: 1 where row dst is a copy of row src."""
        done = torch.empty_like(src)
        dcoco_pages_fork(self.handle, self.planes, src, dst, self.table, self.held, self.lens, self.refs, done=done,
                         stream=stream)
        return done

    def free(self, rows, stream=None):
        dcoco_pages_free(self.handle, rows, self.table, self.held, self.lens, self.refs, stream=stream)

    def compact(self, stream=None):
        """-> live [1], the pages in use: 0 .. live - 1 from then on."""
        dcoco_pages_compact(self.handle, self.planes, self.table, self.held, self.refs, live=self.live, stream=stream)
        return self.live

    def status(self) -> int:
        return dcoco_pages_status(self.handle)


# ------------------------------------------------------------------ convenience wrapper
class Corrector:
    """Owns a handle + packed weights; allocates output tensors per call."""

    def __init__(self, weights: dict, vocab: int, hidden: int, slots: int = 16, topk: int = 16,
                 max_batch: int = 32, variant: int = 0, sigma: float = 1.0, ln_eps: float = 1e-5,
                 host_staging: bool = False, path_rule: int = 0, beam_width: int = 2, beam_topm: int = 0):
        self.vocab, self.hidden, self.slots, self.topk = vocab, hidden, slots, topk
        self.B = slots - 1
        self.max_batch = max_batch
        self.path_rule = path_rule
        self.handle = dcoco_create(vocab, hidden, slots, topk, max_batch, variant, sigma, ln_eps,
                                   host_staging=host_staging, path_rule=path_rule, beam_width=beam_width,
                                   beam_topm=beam_topm)
        try:
            self.weights = dcoco_weights_create(self.handle, weights)
        except Exception:
            dcoco_destroy(self.handle)
            raise

    def close(self):
        if getattr(self, "weights", None) is not None:
            dcoco_weights_destroy(self.weights)
            self.weights = None
        if getattr(self, "handle", None) is not None:
            dcoco_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def alloc_outputs(self, N: int, device="cuda", full: bool = True, features: bool = False):
        B, K = self.B, self.topk
        i32 = dict(dtype=torch.int32, device=device)
        f32 = dict(dtype=torch.float32, device=device)
        out = {"tokens": torch.empty(N, B, **i32), "accept_len": torch.empty(N, **i32)}
        if full:
            out.update(choice=torch.empty(N, B, **i32), scores=torch.empty(N, B - 1, K, K, **f32),
                       topk_ids=torch.empty(N, B, K, **i32), topk_val=torch.empty(N, B, K, **f32),
                       margin=torch.empty(N, B - 1, **f32))
        if features:
            out["cand_feat"] = torch.empty(N, B, K, 5, **f32)
        return out

    def correct(self, logits, hidden, cand_embed, target_tokens=None, out=None, full=True,
                logits_slot_stride=None, stream=None):
        N = logits.shape[0]
        out = out if out is not None else self.alloc_outputs(N, logits.device, full)
        kw = {k: v for k, v in out.items() if k != "accept_len"}
        dcoco_correct(self.handle, self.weights, N, logits, hidden, cand_embed, target_tokens,
                      accept_len=out.get("accept_len") if target_tokens is not None else None,
                      logits_slot_stride=logits_slot_stride, stream=stream, **kw)
        return out

    def verify_stochastic(self, target_logits, tokens, u_accept, u_draw, target_stride=None, stream=None):
        """-> dict(accept_len [N], next_token [N], q_accept [N, B]) on the tokens' device."""
        N = tokens.shape[0]
        dev = tokens.device
        out = {"accept_len": torch.empty(N, dtype=torch.int32, device=dev),
               "next_token": torch.empty(N, dtype=torch.int32, device=dev),
               "q_accept": torch.empty(N, self.B, dtype=torch.float32, device=dev)}
        dcoco_verify_stochastic(self.handle, N, target_logits, tokens, u_accept, u_draw, out["accept_len"],
                                out["next_token"], out["q_accept"], target_stride, stream)
        return out

    def status(self) -> int:
        return dcoco_get_device_status(self.handle)
