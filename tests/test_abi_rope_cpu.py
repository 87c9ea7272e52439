"""Refusals of sps_qk_norm_rope and sps_kv_append_rope that need no GPU: every call has real host
buffers of the size its arguments declare, and is rejected before any launch."""
import ctypes

import numpy as np
import pytest

from paged_top_sparse_gb300 import binding as B
from paged_top_sparse_gb300 import build

T, H, G, D = 6, 4, 2, 128


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


class Env:
    def __init__(self, **kw):
        self.plan = B.Plan([T], [0], H, G, D, 1, 1, 1, **kw)
        self.ws = _aligned(self.plan.workspace_bytes)
        self.buf = {n: _aligned(1 << 16) for n in ("q", "k", "v", "qo", "ko", "kc", "vc", "ks", "vs")}
        self.f = np.ones(64, np.float32)
        self.w = np.ones(D, np.float32)
        self.pt = np.zeros(4, np.int32)

    def rope(self, **kw):
        a = dict(inv_freq=_ptr(self.f), positions=None, rotary_dim=128, num_axes=1, interleaved=0)
        axis = kw.pop("pair_axis", [0] * 64)
        a.update(kw)
        return B.RopeArgs(a["inv_freq"], a["positions"], a["rotary_dim"], a["num_axes"],
                          a["interleaved"], (ctypes.c_uint8 * 64)(*axis))

    def qk(self, L, rope=None, **kw):
        b = self.buf
        a = dict(plan=self.plan.handle, q=_ptr(b["q"]), qs=H * D, k=_ptr(b["k"]), ks=G * D,
                 qw=_ptr(self.w), kw=_ptr(self.w), eps=1e-6, qo=_ptr(b["qo"]), qos=H * D,
                 dt=B.BF16, scale=1.0, ko=_ptr(b["ko"]), kos=G * D, ws=_ptr(self.ws))
        a.update(kw)
        return L.sps_qk_norm_rope(a["plan"], a["q"], a["qs"], a["k"], a["ks"], a["qw"], a["kw"],
                                  a["eps"], ctypes.byref(rope) if rope else None, a["qo"],
                                  a["qos"], a["dt"], a["scale"], a["ko"], a["kos"], a["ws"], None)

    def kv(self, L, rope=None, **kw):
        b = self.buf
        a = dict(plan=self.plan.handle, k=_ptr(b["k"]), ks=G * D, v=_ptr(b["v"]), vs=G * D,
                 w=_ptr(self.w), eps=1e-6, pt=_ptr(self.pt), kc=_ptr(b["kc"]), vc=_ptr(b["vc"]),
                 kcs=_ptr(b["ks"]), vcs=_ptr(b["vs"]), ws=_ptr(self.ws))
        a.update(kw)
        return L.sps_kv_append_rope(a["plan"], a["k"], a["ks"], a["v"], a["vs"], a["w"], a["eps"],
                                    ctypes.byref(rope) if rope else None, a["pt"], a["kc"], a["vc"],
                                    a["kcs"], a["vcs"], a["ws"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(plan=None), 1), (dict(ws=None), 1), (dict(q=None), 1), (dict(qo=None), 1),
    (dict(k=None), 1), (dict(ko=None), 1), (dict(qs=H * D - 8), 1), (dict(qs=H * D + 4), 1),
    (dict(ks=G * D + 1), 1), (dict(qos=0), 1), (dict(kos=8), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(dt=B.FP16), 2),
    (dict(dt=B.E4M3, scale=0.0), 1), (dict(dt=B.E4M3, scale=float("nan")), 1),
    (dict(dt=B.E4M3, qos=H * D + 8), 1),
])
def test_qk_refusals(L, kw, status):
    e = Env()
    assert e.qk(L, **kw) == status
    assert L.sps_last_error()


def test_qk_refuses_misaligned_rows(L):
    e = Env()
    for n in ("q", "k", "qo", "ko"):
        assert e.qk(L, **{n: _ptr(e.buf[n], 8)}) == 1
    assert e.qk(L, qw=_ptr(e.w.view(np.uint8), 2)) == 1


def test_qk_refuses_an_output_that_lies_on_other_rows(L):
    e = Env()
    q, k = _ptr(e.buf["q"]), _ptr(e.buf["k"])
    assert e.qk(L, qo=q, dt=B.E4M3) == 1  # codes over the rows that they come from
    assert e.qk(L, qo=q, qos=H * D + 16) == 1
    assert e.qk(L, ko=k, kos=G * D + 8) == 1


@pytest.mark.parametrize("kw,status", [
    (dict(rotary_dim=-16), 1), (dict(rotary_dim=144), 1), (dict(rotary_dim=24), 2),
    (dict(num_axes=0), 1), (dict(num_axes=5), 1), (dict(inv_freq=None), 1),
    (dict(pair_axis=[0] * 63 + [1]), 1), (dict(num_axes=3, pair_axis=[3] + [0] * 63), 1),
])
def test_rope_refusals(L, kw, status):
    e = Env()
    assert e.qk(L, rope=e.rope(**kw)) == status
    assert e.kv(L, rope=e.rope(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(plan=None), 1), (dict(ws=None), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(pt=None), 1), (dict(kc=None), 1), (dict(vc=None), 1), (dict(ks=G * D - 8), 1),
    (dict(vs=G * D + 2), 1), (dict(eps=-0.5), 1),
])
def test_append_refusals(L, kw, status):
    e = Env()
    assert e.kv(L, **kw) == status
    assert L.sps_last_error()


def test_append_needs_scales_for_an_nvfp4_cache(L):
    e = Env(q_dtype="e4m3", kv_dtype="nvfp4")
    assert e.kv(L, kcs=None) == 1
    assert e.kv(L, vcs=None) == 1


def test_binding_checks_shapes():
    torch = pytest.importorskip("torch")
    f = torch.ones(64)
    with pytest.raises(ValueError):
        B.Rope(torch.ones(65))
    with pytest.raises(ValueError):
        B.Rope(f.double())
    with pytest.raises(ValueError):
        B.Rope(f, positions=torch.zeros(2, T, dtype=torch.int64))
    with pytest.raises(ValueError):
        B.Rope(f, pair_axis=[0] * 63)
    plan = B.Plan([T], [0], H, G, D, 1, 1, 1)
    q = torch.zeros(T, H, D, dtype=torch.bfloat16)
    for bad in (q[:, :2], q[:3], q.transpose(1, 2), q[..., ::2]):
        with pytest.raises(ValueError):
            B._rows(bad, plan.q_shape, "q")
    wide = torch.zeros(T, H + 3, D, dtype=torch.bfloat16)
    assert B._rows(wide[:, 1:1 + H], plan.q_shape, "q") == (H + 3) * D
    for bad, codes in ((q.half(), False), (q.float(), False), (q, True)):
        with pytest.raises(ValueError):
            B._rows(bad, plan.q_shape, "q", codes)
    with pytest.raises(ValueError):
        B.sps_qk_norm_rope(plan, q, None, torch.ones(D // 2), None, 1e-6, None, q, 1.0, None, q)
    with pytest.raises(ValueError):
        B.sps_kv_append_rope(plan, q[:, :G], q[:, G:], None, 1e-6, None,
                             torch.zeros(1, dtype=torch.int64), q, q, None, None, q)
    with pytest.raises(ValueError):
        B.paged_attention_fwd(plan, q, 1.0, q, q, None, None, torch.zeros(0, dtype=torch.int32), q,
                              None, q, q)
    assert B._rows(q, plan.q_shape, "q") == B._rows(q.to(torch.uint8), plan.q_shape, "q", True) == H * D
    with pytest.raises(ValueError):
        B._rope(B.Rope(f, positions=torch.zeros(T - 1, dtype=torch.int32)), plan)
