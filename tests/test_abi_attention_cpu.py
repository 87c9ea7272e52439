"""Refusals and work split of paged_attention_fwd that need no GPU: every call has real host buffers
of the size its arguments declare, and is rejected before any launch."""
import ctypes

import numpy as np
import pytest

from paged_top_sparse_gb300 import binding as B
from paged_top_sparse_gb300 import build

T, H, G, D = 3, 4, 2, 64


@pytest.fixture(scope="module")
def L():
    build.build()
    return B.lib()


def _aligned(n):
    raw = np.zeros(n + 256, np.uint8)
    off = -raw.ctypes.data % 256
    return raw[off:off + n]


def _ptr(a, off=0):
    return ctypes.c_void_p(a.ctypes.data + off)


def _call(L, quant=False, **kw):
    plan = B.Plan([T], [10], H, G, D, 1, 1, 2, q_dtype="e4m3" if quant else "bf16",
                  kv_dtype="nvfp4" if quant else "bf16")
    n = B.paged_attention_scratch(plan)
    ws, scratch = _aligned(plan.workspace_bytes), _aligned(n)
    buf = {k: _aligned(1 << 17) for k in ("q", "k", "v", "ks", "vs", "out", "lse")}
    pt = np.zeros(1, np.int32)
    a = dict(plan=plan.handle, q=_ptr(buf["q"]), qs=H * D, scale=1.0, k=_ptr(buf["k"]),
             v=_ptr(buf["v"]), ks=_ptr(buf["ks"]), vs=_ptr(buf["vs"]), pt=_ptr(pt),
             out=_ptr(buf["out"]), os=H * D, lse=_ptr(buf["lse"]), scratch=_ptr(scratch), n=n,
             ws=_ptr(ws))
    for name, v in kw.items():
        a[name] = v(buf, scratch, ws) if callable(v) else v
    if "n" in kw:
        a["n"] = n + kw["n"]
    return L.paged_attention_fwd(a["plan"], a["q"], a["qs"], a["scale"], a["k"], a["v"], a["ks"],
                                 a["vs"], a["pt"], a["out"], a["os"], a["lse"], a["scratch"], a["n"],
                                 a["ws"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(plan=None), 1), (dict(ws=None), 1), (dict(q=None), 1), (dict(out=None), 1),
    (dict(k=None), 1), (dict(v=None), 1), (dict(pt=None), 1), (dict(scratch=None), 1),
    (dict(qs=H * D - 8), 1), (dict(qs=H * D + 4), 1), (dict(os=H * D + 2), 1), (dict(os=0), 1),
    (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(n=-1), 3),
    (dict(q=lambda b, s, w: _ptr(b["q"], 8)), 1), (dict(out=lambda b, s, w: _ptr(b["out"], 8)), 1),
    (dict(k=lambda b, s, w: _ptr(b["k"], 8)), 1), (dict(v=lambda b, s, w: _ptr(b["v"], 2)), 1),
    (dict(lse=lambda b, s, w: _ptr(b["lse"], 2)), 1), (dict(ws=lambda b, s, w: _ptr(w, 16)), 1),
    (dict(scratch=lambda b, s, w: _ptr(s, 128)), 1),
    (dict(quant=True, ks=None), 1), (dict(quant=True, vs=None), 1),
    (dict(quant=True, qs=H * D + 8), 1), (dict(quant=True, ks=lambda b, s, w: _ptr(b["ks"], 4)), 1),
])
def test_refusals(L, kw, status):
    assert _call(L, **kw) == status
    assert L.sps_last_error()


def test_scratch_needs_a_plan(L):
    n = ctypes.c_size_t()
    assert L.paged_attention_scratch(None, ctypes.byref(n)) == 1


def test_tensor_map_limit_is_refused(L):
    plan = B.Plan([1], [0], 16, 16, D, 1, 1, 1 << 21)
    ws = _aligned(plan.workspace_bytes)
    n = B.paged_attention_scratch(plan)
    scratch, buf = _aligned(n), _aligned(1 << 16)
    pt = np.zeros(1, np.int32)
    assert L.paged_attention_fwd(plan.handle, _ptr(buf), 16 * D, 1.0, _ptr(buf), _ptr(buf), None,
                                 None, _ptr(pt), _ptr(buf), 16 * D, None, _ptr(scratch), n,
                                 _ptr(ws), None) == 2


def test_scratch_follows_the_rows_a_cut_tile_can_have(L):
    one = B.paged_attention_scratch(B.Plan([1], [1000], 32, 2, 128, 1, 8, 8))
    many = B.paged_attention_scratch(B.Plan([500], [1000], 32, 2, 128, 1, 12, 12))
    # 16 rows a tile against 256
    assert one * 16 == pytest.approx(many, rel=0.01)
    assert one % 256 == 0 and many % 256 == 0


def test_a_scale_that_leaves_fp32_is_refused(L):
    """softmax_scale x q_scale is one FP32 factor of the scores: rounded to zero it would turn masked
    scores into NaN (0 * infinity), rounded to infinity every equal one."""
    for scale, softmax, status in ((1e-40, 1e-10, 1), (3e38, 4.0, 1), (3e38, 1.0, 1)):
        plan = B.Plan([T], [10], H, G, D, 1, 1, 2, softmax_scale=softmax)
        n = B.paged_attention_scratch(plan)
        ws, scratch, buf = _aligned(plan.workspace_bytes), _aligned(n), _aligned(1 << 17)
        pt = np.zeros(1, np.int32)
        assert L.paged_attention_fwd(plan.handle, _ptr(buf), H * D, scale, _ptr(buf), _ptr(buf), None,
                                     None, _ptr(pt), _ptr(buf), H * D, None, _ptr(scratch), n,
                                     _ptr(ws), None) == status
        assert b"scale" in L.sps_last_error()
