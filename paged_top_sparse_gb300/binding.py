"""Thin ctypes binding of libsps (``include/sparse_prefill.h``).

Argument marshalling only: every function takes torch tensors (device memory supplied by
the caller), derives pointers, pitches and strides from them, calls the C entry point of the
same name and raises ``SpsError`` on a non-OK status.  No computation happens here, and
there is no fallback: if the library is missing, ``lib()`` raises.
"""
from __future__ import annotations

import ctypes
import os
import re

from . import build as _build

BF16, FP16, E4M3, NVFP4 = 0, 1, 2, 3
DTYPE_CODES = {"bf16": BF16, "fp16": FP16, "e4m3": E4M3, "nvfp4": NVFP4}
STATUS = {0: "SPS_OK", 1: "SPS_EINVAL", 2: "SPS_EUNSUPPORTED", 3: "SPS_ENOSPACE",
          4: "SPS_ECUDA", 5: "SPS_EDEVICE"}
HEADER = os.path.join(os.path.dirname(_build.HERE), "include", "sparse_prefill.h")


class SpsError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


class Problem(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("q_lens", ctypes.POINTER(ctypes.c_int32)),
        ("ctx_lens", ctypes.POINTER(ctypes.c_int32)),
        ("num_q_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("max_pages_per_req", ctypes.c_int32),
        ("num_phys_pages", ctypes.c_int32),
        ("q_dtype", ctypes.c_int),
        ("kv_dtype", ctypes.c_int),
        ("idx_q_dtype", ctypes.c_int),
        ("idx_k_dtype", ctypes.c_int),
        ("softmax_scale", ctypes.c_float),
    ]


class PlanInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "num_tokens", "num_rows", "num_buckets", "max_entries", "indexer_tasks", "max_fwd_tasks",
        "workspace_bytes", "off_status", "off_tok_pos", "off_tok_req", "off_bucket_offsets",
        "off_entries", "off_fwd_task_count")]


class RopeArgs(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("rotary_dim", ctypes.c_int32), ("num_axes", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("pair_axis", ctypes.c_uint8 * 64)]


_lib = None


def header_functions() -> list[str]:
    """Names of the functions declared in include/sparse_prefill.h."""
    src = open(HEADER).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[A-Za-z_][\w\s\*]*?\b(\w+)\s*\(", src, re.M))
                  - {"if", "while"})


def lib(path: str | None = None):
    """Load libsps.so (built in-tree by ``build.build()``, or the file named by $SPS_LIB);
    raises if it is absent."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or os.environ.get("SPS_LIB") or _build.LIB
    if not os.path.exists(path):
        raise RuntimeError(f"libsps.so not built ({path}); run paged_top_sparse_gb300.build.build()")
    L = ctypes.CDLL(path)
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
    L.sparse_prefill_plan.argtypes = [ctypes.POINTER(Problem), ctypes.POINTER(vp),
                                      ctypes.POINTER(ctypes.c_size_t)]
    L.sps_plan_destroy.argtypes = [vp]
    L.sps_plan_destroy.restype = None
    L.sps_plan_get_info.argtypes = [vp, ctypes.POINTER(PlanInfo)]
    L.sps_plan_upload.argtypes = [vp, vp, ctypes.c_size_t, vp]
    L.indexer_scores.argtypes = [vp, vp, f32, vp, vp, f32, vp, vp, i64, vp, vp]
    L.topk_select.argtypes = [vp, vp, i64, vp, vp, vp]
    L.sparse_prefill_fwd.argtypes = [vp, vp, f32, vp, vp, vp, vp, vp, vp, vp, i64, vp, i64, vp, vp]
    L.partial_combine.argtypes = [i64, i32, i32, vp, i64, vp, i64, vp, i64, vp, vp, vp]
    L.sparse_prefill_fwd_bf16.argtypes = L.sparse_prefill_fwd.argtypes
    L.sparse_prefill_fwd_fp8qk.argtypes = L.sparse_prefill_fwd.argtypes
    L.sparse_prefill_fwd_f16.argtypes = L.sparse_prefill_fwd.argtypes
    L.sps_kv_append.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.sps_quantize_e4m3.argtypes = [vp, i64, f32, vp, vp]
    L.sps_absmax_bf16.argtypes = [vp, i64, vp, vp]
    rp = ctypes.POINTER(RopeArgs)
    L.sps_qk_norm_rope.argtypes = [vp, vp, i64, vp, i64, vp, vp, f32, rp, vp, i64, ctypes.c_int,
                                   f32, vp, i64, vp, vp]
    L.sps_kv_append_rope.argtypes = [vp, vp, i64, vp, i64, vp, f32, rp, vp, vp, vp, vp, vp, vp, vp]
    L.paged_attention_scratch.argtypes = [vp, ctypes.POINTER(ctypes.c_size_t)]
    L.paged_attention_fwd.argtypes = [vp, vp, i64, f32, vp, vp, vp, vp, vp, vp, i64, vp, vp,
                                      ctypes.c_size_t, vp, vp]
    L.partial_combine_bf16.argtypes = L.partial_combine.argtypes
    L.partial_combine_f16.argtypes = L.partial_combine.argtypes
    L.sparse_prefill_fwd_noalloc.argtypes = [vp, vp, f32, vp, vp, vp, vp, vp, vp, vp, i64, vp, i64,
                                             vp, vp]
    L.sps_read_device_status.argtypes = [vp, vp, ctypes.POINTER(i32)]
    L.sps_dequantize.argtypes = [ctypes.c_int, vp, vp, i64, vp, vp]
    L.sps_check_wait_timeout.argtypes = [i64, vp, vp]
    L.sps_check_barrier_timeout.argtypes = [i64, vp, vp, vp]
    L.sps_last_error.restype = ctypes.c_char_p
    for name in ("sparse_prefill_plan", "sps_plan_get_info", "sps_plan_upload", "indexer_scores",
                 "topk_select", "sparse_prefill_fwd", "partial_combine", "sps_read_device_status",
                 "sparse_prefill_fwd_noalloc", "sps_dequantize", "sps_check_wait_timeout",
                 "sps_check_barrier_timeout"):
        getattr(L, name).restype = ctypes.c_int
    _lib = L
    return L


def _check(st: int):
    if st != 0:
        raise SpsError(st, lib().sps_last_error().decode())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _find_stream():
    """The current stream's cudaStream_t.  The lookup goes past torch's stream objects where it can:
    making one costs more than a small kernel runs.  (Replaces itself on the first call.)"""
    global _current_stream
    import torch

    get, dev = (getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream",
                                                     "_cuda_getDevice"))
    _current_stream = ((lambda: get(dev())) if get and dev else
                       (lambda: torch.cuda.current_stream().cuda_stream))
    return _current_stream()


_current_stream = _find_stream


def _stream(stream):
    return _current_stream() if stream is None else stream.cuda_stream


class Plan:
    """Owns an sps_plan; ``workspace_bytes`` is the device workspace its calls need."""

    def __init__(self, q_lens, ctx_lens, num_q_heads, num_kv_heads, head_dim, top_k,
                 max_pages_per_req, num_phys_pages, q_dtype="bf16", kv_dtype="bf16",
                 idx_q_dtype=None, idx_k_dtype=None, softmax_scale=None, page_size=128):
        L = lib()
        n = len(q_lens)
        self._ql = (ctypes.c_int32 * n)(*[int(x) for x in q_lens])
        self._cl = (ctypes.c_int32 * n)(*[int(x) for x in ctx_lens])
        self.problem = Problem(
            n, self._ql, self._cl, num_q_heads, num_kv_heads, head_dim, page_size, top_k,
            max_pages_per_req, num_phys_pages, DTYPE_CODES[q_dtype], DTYPE_CODES[kv_dtype],
            DTYPE_CODES[idx_q_dtype or q_dtype], DTYPE_CODES[idx_k_dtype or kv_dtype],
            float(softmax_scale if softmax_scale is not None else head_dim ** -0.5))
        self.handle = ctypes.c_void_p()
        ws = ctypes.c_size_t()
        _check(L.sparse_prefill_plan(ctypes.byref(self.problem), ctypes.byref(self.handle),
                                     ctypes.byref(ws)))
        self.workspace_bytes = ws.value
        self.head_dim, self.top_k = head_dim, top_k
        self.num_tokens = sum(int(x) for x in q_lens)
        _load_types()
        self.table_shape, self.table_size = (n, max_pages_per_req), n * max_pages_per_req
        self.q_codes = self.problem.q_dtype == E4M3
        self.quant_kv = self.problem.kv_dtype == NVFP4
        # bytes of a cache (an NVFP4 one's scales: an eighth of them), and the types that may hold it
        elems = num_phys_pages * num_kv_heads * page_size * head_dim
        self.cache_bytes = elems // 2 if self.quant_kv else elems * 2
        self.cache_types = _CODES if self.quant_kv else _BITS16
        # shapes of a query, and of new keys or values
        self.q_shape = (self.num_tokens, num_q_heads, head_dim)
        self.kv_shape = (self.num_tokens, num_kv_heads, head_dim)

    def info(self) -> PlanInfo:
        inf = PlanInfo()
        _check(lib().sps_plan_get_info(self.handle, ctypes.byref(inf)))
        return inf

    def __del__(self):
        h = getattr(self, "handle", None)
        if h and _lib is not None:
            _lib.sps_plan_destroy(h)
            self.handle = None


def sparse_prefill_plan(*args, **kw) -> Plan:
    return Plan(*args, **kw)


def sps_plan_upload(plan: Plan, workspace, stream=None):
    _check(lib().sps_plan_upload(plan.handle, _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(stream)))


def indexer_scores(plan: Plan, q_idx, q_scale, k_idx_cache, k_idx_scales, k_scale, page_table,
                   scores, workspace, stream=None):
    _check(lib().indexer_scores(plan.handle, _ptr(q_idx), float(q_scale), _ptr(k_idx_cache),
                                _ptr(k_idx_scales), float(k_scale), _ptr(page_table), _ptr(scores),
                                scores.stride(0), _ptr(workspace), _stream(stream)))


def topk_select(plan: Plan, scores, idx, workspace, stream=None):
    _check(lib().topk_select(plan.handle, _ptr(scores), scores.stride(0), _ptr(idx),
                             _ptr(workspace), _stream(stream)))


def sparse_prefill_fwd(plan: Plan, q, q_scale, k_cache, v_cache, k_scales, v_scales, page_table,
                       idx, partial, lse, workspace, stream=None):
    """``partial`` is a [splits][rows][D] view (its stride(0) is the split stride); ``lse`` is
    [splits][rows] (stride(0) is the LSE split stride)."""
    _check(lib().sparse_prefill_fwd(plan.handle, _ptr(q), float(q_scale), _ptr(k_cache),
                                    _ptr(v_cache), _ptr(k_scales), _ptr(v_scales), _ptr(page_table),
                                    _ptr(idx), _ptr(partial), partial.stride(0), _ptr(lse),
                                    lse.stride(0), _ptr(workspace), _stream(stream)))


def sparse_prefill_fwd_bf16(plan: Plan, q, q_scale, k_cache, v_cache, k_scales, v_scales,
                            page_table, idx, partial, lse, workspace, stream=None):
    """As ``sparse_prefill_fwd`` with ``partial`` a BF16 [splits][rows][D] view."""
    _check(lib().sparse_prefill_fwd_bf16(plan.handle, _ptr(q), float(q_scale), _ptr(k_cache),
                                         _ptr(v_cache), _ptr(k_scales), _ptr(v_scales),
                                         _ptr(page_table), _ptr(idx), _ptr(partial),
                                         partial.stride(0), _ptr(lse), lse.stride(0),
                                         _ptr(workspace), _stream(stream)))


def sparse_prefill_fwd_f16(plan: Plan, q, q_scale, k_cache, v_cache, k_scales, v_scales,
                           page_table, idx, partial, lse, workspace, stream=None):
    """As ``sparse_prefill_fwd`` with ``partial`` an FP16 [splits][rows][D] view."""
    _check(lib().sparse_prefill_fwd_f16(plan.handle, _ptr(q), float(q_scale), _ptr(k_cache),
                                        _ptr(v_cache), _ptr(k_scales), _ptr(v_scales),
                                        _ptr(page_table), _ptr(idx), _ptr(partial),
                                        partial.stride(0), _ptr(lse), lse.stride(0),
                                        _ptr(workspace), _stream(stream)))


def sparse_prefill_fwd_fp8qk(plan: Plan, q, q_scale, k_cache, v_cache, k_scales, v_scales,
                             page_table, idx, partial, lse, workspace, stream=None):
    """As ``sparse_prefill_fwd``: E4M3 Q, NVFP4 K rounded to E4M3, FP8 Q K^T (the pages' route)."""
    _check(lib().sparse_prefill_fwd_fp8qk(plan.handle, _ptr(q), float(q_scale), _ptr(k_cache),
                                          _ptr(v_cache), _ptr(k_scales), _ptr(v_scales),
                                          _ptr(page_table), _ptr(idx), _ptr(partial),
                                          partial.stride(0), _ptr(lse), lse.stride(0),
                                          _ptr(workspace), _stream(stream)))


def sparse_prefill_fwd_noalloc(plan: Plan, q, q_scale, k_cache, v_cache, k_scales, v_scales,
                               page_table, idx, partial, lse, dev_status=None, stream=None):
    """sparse_prefill_fwd without a workspace: the library's own fixed scratch array is used
    (for callers that cannot allocate device memory; see the header for the rules)."""
    _check(lib().sparse_prefill_fwd_noalloc(
        plan.handle, _ptr(q), float(q_scale), _ptr(k_cache), _ptr(v_cache), _ptr(k_scales),
        _ptr(v_scales), _ptr(page_table), _ptr(idx), _ptr(partial), partial.stride(0), _ptr(lse),
        lse.stride(0), _ptr(dev_status), _stream(stream)))


def partial_combine(partial, lse, out, out_lse=None, dev_status=None, stream=None):
    """partial [splits][rows][D] FP32 (rows contiguous), lse [splits][rows], out [rows][D] BF16."""
    S, R, D = partial.shape
    _check(lib().partial_combine(R, S, D, _ptr(partial), partial.stride(0), _ptr(lse),
                                 lse.stride(0), _ptr(out), out.stride(0), _ptr(out_lse),
                                 _ptr(dev_status), _stream(stream)))


def partial_combine_bf16(partial, lse, out, out_lse=None, dev_status=None, stream=None):
    """As ``partial_combine`` with ``partial`` BF16 [splits][rows][D] (rows contiguous)."""
    S, R, D = partial.shape
    _check(lib().partial_combine_bf16(R, S, D, _ptr(partial), partial.stride(0), _ptr(lse),
                                      lse.stride(0), _ptr(out), out.stride(0), _ptr(out_lse),
                                      _ptr(dev_status), _stream(stream)))


def partial_combine_f16(partial, lse, out, out_lse=None, dev_status=None, stream=None):
    """As ``partial_combine`` with ``partial`` FP16 [splits][rows][D] (rows contiguous)."""
    S, R, D = partial.shape
    _check(lib().partial_combine_f16(R, S, D, _ptr(partial), partial.stride(0), _ptr(lse),
                                     lse.stride(0), _ptr(out), out.stride(0), _ptr(out_lse),
                                     _ptr(dev_status), _stream(stream)))


def sps_kv_append(plan: Plan, k_new, v_new, page_table, k_cache, v_cache, k_scales, v_scales,
                  workspace, stream=None):
    """New tokens' K/V [T][H_kv][D] BF16 into the paged cache (the plan's kv dtype)."""
    _check(lib().sps_kv_append(plan.handle, _ptr(k_new), _ptr(v_new), _ptr(page_table),
                               _ptr(k_cache), _ptr(v_cache), _ptr(k_scales), _ptr(v_scales),
                               _ptr(workspace), _stream(stream)))


class Rope:
    """A rotation by position (``sps_rope``): ``inv_freq`` FP32 [rotary_dim / 2] and, where the
    tokens have positions of their own, ``positions`` int32 [axes][T] (one axis: also [T]), both
    on the device and kept alive here; ``pair_axis``: the axis of each pair (default 0)."""

    def __init__(self, inv_freq, positions=None, pair_axis=None, interleaved=False):
        self.inv_freq, self.positions = inv_freq, positions
        n, axes = inv_freq.numel(), 1
        _load_types()
        _vector(inv_freq, _F32, n, "inv_freq")
        if n > 64:
            raise ValueError("at most 64 pairs (rotary_dim 128)")
        if positions is not None:
            _vector(positions, _I32, positions.numel(), "positions")
            axes = positions.shape[0] if positions.dim() == 2 else 1
        ax = [int(a) for a in pair_axis] if pair_axis is not None else [0] * n
        if len(ax) != n or any(not 0 <= a < 256 for a in ax):
            raise ValueError("pair_axis needs one axis per pair")
        self.args = RopeArgs(_ptr(inv_freq), _ptr(positions), 2 * n, axes, int(bool(interleaved)),
                             (ctypes.c_uint8 * 64)(*ax))
        self.ref = ctypes.pointer(self.args)


_F32 = _I32 = _BF16 = _BITS16 = _CODES = None


def _load_types():
    global _F32, _I32, _BF16, _BITS16, _CODES
    import torch

    _F32, _I32, _BF16 = torch.float32, torch.int32, torch.bfloat16
    _BITS16 = {torch.bfloat16, torch.int16, torch.uint16}
    _CODES = {torch.uint8, torch.int8, getattr(torch, "float4_e2m1fn_x2", torch.uint8)}


def _vector(t, dtype, numel, name):
    """A contiguous tensor of the type and size (or None)."""
    if t is not None and (t.dtype is not dtype or t.numel() != numel or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {numel} elements")


def _table(t, plan):
    """The page table's address: rows of max_pages_per_req entries, or those in one flat vector; rows
    behind the batch's are allowed."""
    if (t.dtype is not _I32 or not t.is_contiguous()
            or (t.shape != plan.table_shape
                and (t.numel() < plan.table_size or (t.dim() > 1 and t.shape[-1] != plan.table_shape[1])))):
        raise ValueError(f"page_table must be a contiguous int32 tensor of >= {plan.table_size} entries "
                         f"in rows of {plan.table_shape[1]}")
    return t.data_ptr()


def _caches(plan, k, v, k_scales, v_scales):
    """The addresses of the caches, and of an NVFP4 cache's scales: contiguous, of the plan's type (or
    raw elements of its size), with the plan's pages at least."""
    n, types = plan.cache_bytes, plan.cache_types
    if (k.nbytes < n or v.nbytes < n or k.dtype not in types or v.dtype not in types
            or not k.is_contiguous() or not v.is_contiguous()):
        for t, name in ((k, "k_cache"), (v, "v_cache")):
            if t.nbytes < n or t.dtype not in types or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous "
                                 f"{'NVFP4 codes' if plan.quant_kv else 'bfloat16'} of >= {n} bytes")
    if not plan.quant_kv:
        return k.data_ptr(), v.data_ptr(), None, None
    for t, name in ((k_scales, "k_scales"), (v_scales, "v_scales")):
        if (t is None or t.element_size() != 1 or t.nbytes < n // 8 or not t.is_contiguous()):
            raise ValueError(f"{name} must be contiguous bytes, >= {n // 8}")
    return k.data_ptr(), v.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr()


def _workspace(t, plan):
    if t.nbytes < plan.workspace_bytes:
        raise ValueError(f"workspace must hold >= {plan.workspace_bytes} bytes")
    return t.data_ptr()


def _rope(rope, plan):
    if rope.positions is not None and rope.positions.shape[-1] != plan.num_tokens:
        raise ValueError(f"positions must be [axes][{plan.num_tokens}]")
    return rope.ref


def _rows(t, shape, name, codes=False):
    """Elements between the tokens of a [T][heads][D] view of BF16, or of one-byte codes, whose rows
    are contiguous."""
    st = t.stride()
    if (t.shape != shape or st[2] != 1 or (st[1] != shape[2] and shape[1] > 1)
            or (t.element_size() != 1 if codes else t.dtype is not _BF16)):
        raise ValueError(f"{name} must be [{shape[0]}][{shape[1]}][{shape[2]}] "
                         f"{'codes' if codes else 'bfloat16'} with contiguous rows")
    return st[0] if shape[0] > 1 else shape[1] * shape[2]


def sps_qk_norm_rope(plan: Plan, q, k, q_weight, k_weight, eps, rope, q_out, q_scale, k_out,
                     workspace, stream=None):
    """Norm per head and rotation of q [T][H][D] and k [T][H_kv][D] (or None); token strides come
    from the tensors.  A one-byte ``q_out`` takes E4M3 codes of the result / ``q_scale``."""
    qs, ks = plan.q_shape, plan.kv_shape
    _vector(q_weight, _F32, plan.head_dim, "q_weight")
    _vector(k_weight, _F32, plan.head_dim, "k_weight")
    codes = q_out.element_size() == 1
    st = (_lib or lib()).sps_qk_norm_rope(
        plan.handle, q.data_ptr(), _rows(q, qs, "q"), _ptr(k),
        0 if k is None else _rows(k, ks, "k"), _ptr(q_weight), _ptr(k_weight), eps,
        None if rope is None else _rope(rope, plan), q_out.data_ptr(),
        _rows(q_out, qs, "q_out", codes), E4M3 if codes else BF16, q_scale,
        _ptr(k_out), 0 if k_out is None else _rows(k_out, ks, "k_out"),
        _workspace(workspace, plan), _stream(stream))
    if st:
        _check(st)


def sps_kv_append_rope(plan: Plan, k_new, v_new, k_weight, eps, rope, page_table, k_cache, v_cache,
                       k_scales, v_scales, workspace, stream=None):
    """``sps_kv_append`` with the key's norm and rotation on the way; k_new / v_new [T][H_kv][D]
    may be views with a token stride."""
    ks = plan.kv_shape
    _vector(k_weight, _F32, plan.head_dim, "k_weight")
    st = (_lib or lib()).sps_kv_append_rope(
        plan.handle, k_new.data_ptr(), _rows(k_new, ks, "k_new"), v_new.data_ptr(),
        _rows(v_new, ks, "v_new"), _ptr(k_weight), eps,
        None if rope is None else _rope(rope, plan), _table(page_table, plan),
        *_caches(plan, k_cache, v_cache, k_scales, v_scales),
        _workspace(workspace, plan), _stream(stream))
    if st:
        _check(st)


def paged_attention_scratch(plan: Plan) -> int:
    """Bytes of device scratch that ``paged_attention_fwd`` needs for this plan."""
    n = ctypes.c_size_t()
    _check(lib().paged_attention_scratch(plan.handle, ctypes.byref(n)))
    return n.value


def paged_attention_fwd(plan: Plan, q, q_scale, k_cache, v_cache, k_scales, v_scales, page_table,
                        out, out_lse, scratch, workspace, stream=None):
    """Full causal attention of q [T][H][D] over the paged cache into out [T][H][D] BF16 (both may
    have a token stride) and, unless None, out_lse [T][H] FP32."""
    qs = plan.q_shape
    _vector(out_lse, _F32, qs[0] * qs[1], "out_lse")
    st = (_lib or lib()).paged_attention_fwd(
        plan.handle, q.data_ptr(), _rows(q, qs, "q", plan.q_codes), q_scale,
        *_caches(plan, k_cache, v_cache, k_scales, v_scales),
        _table(page_table, plan), out.data_ptr(), _rows(out, qs, "out"), _ptr(out_lse),
        scratch.data_ptr(), scratch.nbytes, _workspace(workspace, plan), _stream(stream))
    if st:
        _check(st)


def sps_quantize_e4m3(x_bf16, scale: float, codes, stream=None):
    """E4M3 codes of ``x_bf16`` (any shape, n % 16 == 0) with a per-tensor scale."""
    _check(lib().sps_quantize_e4m3(_ptr(x_bf16), x_bf16.numel(), float(scale), _ptr(codes),
                                   _stream(stream)))


def sps_absmax_bf16(x_bf16, out_f32, stream=None):
    """out_f32[0] = max |x| over ``x_bf16`` (device)."""
    _check(lib().sps_absmax_bf16(_ptr(x_bf16), x_bf16.numel(), _ptr(out_f32), _stream(stream)))


def sps_dequantize(in_dtype: str, data, scales, n: int, out_f16, stream=None):
    """Exact E4M3 / NVFP4 -> FP16 of n elements into ``out_f16`` (see the header)."""
    _check(lib().sps_dequantize(DTYPE_CODES[in_dtype], _ptr(data), _ptr(scales), int(n),
                                _ptr(out_f16), _stream(stream)))


def sps_check_wait_timeout(limit_ns: int, dev_status, stream=None):
    """Launch the bounded-wait self-check; *dev_status becomes SPS_DEV_TIMEOUT (1)."""
    _check(lib().sps_check_wait_timeout(int(limit_ns), _ptr(dev_status), _stream(stream)))


def sps_check_barrier_timeout(limit_ns: int, dev_barrier, dev_status, stream=None):
    """Grid-barrier timeout self-check: dev_barrier is a zeroed device int32 tensor of 2."""
    _check(lib().sps_check_barrier_timeout(int(limit_ns), _ptr(dev_barrier), _ptr(dev_status),
                                           _stream(stream)))


def sps_read_device_status(plan: Plan, workspace) -> int:
    code = ctypes.c_int32()
    st = lib().sps_read_device_status(plan.handle, _ptr(workspace), ctypes.byref(code))
    if st not in (0, 5):
        _check(st)
    return code.value
