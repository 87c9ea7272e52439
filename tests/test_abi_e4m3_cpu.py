"""Plans of an E4M3 K/V cache, the refusals of the calls over it and of sps_page_tables, and what the binding
refuses before it calls the library; no GPU needed: every call has real host buffers of the size its
arguments declare, and is rejected before any launch."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from paged_top_sparse_gb300 import binding as B
from paged_top_sparse_gb300 import build

T, H, G, D, PAGES = 3, 4, 2, 64, 5


@pytest.fixture(scope="module", autouse=True)
def L():
    build.build()
    return B.lib()


def _aligned(n):
    raw = np.zeros(n + 256, np.uint8)
    off = -raw.ctypes.data % 256
    return raw[off:off + n]


def _ptr(a, off=0):
    return ctypes.c_void_p(a.ctypes.data + off)


@pytest.mark.parametrize("q,kv,ok", [("bf16", "e4m3", True), ("e4m3", "e4m3", True), ("fp16", "e4m3", False),
                                     ("nvfp4", "e4m3", False), ("bf16", "nvfp4", False)])
def test_plans_of_an_e4m3_cache(q, kv, ok):
    if ok:
        B.Plan([T], [10], H, G, D, 1, 1, 2, q_dtype=q, kv_dtype=kv)
        return
    with pytest.raises(B.SpsError) as e:
        B.Plan([T], [10], H, G, D, 1, 1, 2, q_dtype=q, kv_dtype=kv, idx_q_dtype="bf16", idx_k_dtype="bf16")
    assert e.value.status == 2


def test_plans_of_other_caches_keep_their_layout():
    """The append's list of pages is there for an E4M3 cache alone, in front of what the forward reads."""
    a = B.Plan([700, 1], [100, 300], H, G, D, 1, 8, 9).info()
    b = B.Plan([700, 1], [100, 300], H, G, D, 1, 8, 9, kv_dtype="e4m3").info()
    extra = b.off_status - a.off_status
    assert 0 < extra <= 256 * (1 + 32 * 8 // 256) + 256
    for n in ("off_tok_pos", "off_tok_req", "off_bucket_offsets", "off_entries", "workspace_bytes"):
        assert getattr(b, n) - getattr(a, n) == extra, n


def _buffers(q="bf16"):
    plan = B.Plan([T], [10], H, G, D, 1, 1, PAGES, q_dtype=q, kv_dtype="e4m3")
    n = B.paged_attention_scratch(plan)
    big = lambda: _aligned(1 << 17)
    return plan, dict(ws=_aligned(plan.workspace_bytes), scratch=_aligned(n), n=n, q=big(), k=big(), v=big(),
                      ks=big(), vs=big(), out=big(), pt=np.zeros(1, np.int32), idx=big(), partial=big(), lse=big())


@pytest.mark.parametrize("name,off,status", [("ks", None, 1), ("vs", None, 1), ("ks", 2, 1), ("vs", 1, 1),
                                             ("k", 8, 1), ("v", 4, 1), ("k", None, 1)])
def test_refusals_of_caches_and_scales(L, name, off, status):
    plan, b = _buffers()
    p = {k: _ptr(v) for k, v in b.items() if k != "n"}
    p[name] = None if off is None else _ptr(b[name], off)
    calls = [L.paged_attention_fwd(plan.handle, p["q"], H * D, 1.0, p["k"], p["v"], p["ks"], p["vs"], p["pt"],
                                   p["out"], H * D, None, p["scratch"], b["n"], p["ws"], None),
             L.sps_kv_append(plan.handle, p["q"], p["out"], p["pt"], p["k"], p["v"], p["ks"], p["vs"], p["ws"], None),
             L.sps_kv_append_rope(plan.handle, p["q"], G * D, p["out"], G * D, None, 1e-6, None, p["pt"], p["k"],
                                  p["v"], p["ks"], p["vs"], p["ws"], None)]
    for fwd in (L.sparse_prefill_fwd, L.sparse_prefill_fwd_f16, L.sparse_prefill_fwd_bf16):
        calls.append(fwd(plan.handle, p["q"], 1.0, p["k"], p["v"], p["ks"], p["vs"], p["pt"], p["idx"],
                         p["partial"], T * H * D, p["lse"], T * H, p["ws"], None))
    assert calls == [status] * len(calls)
    assert L.sps_last_error()


@pytest.mark.parametrize("q,stride,status", [("bf16", H * D + 4, 1), ("e4m3", H * D + 8, 1), ("bf16", H * D - 8, 1)])
def test_query_strides(L, q, stride, status):
    plan, b = _buffers(q)
    p = {k: _ptr(v) for k, v in b.items() if k != "n"}
    assert L.paged_attention_fwd(plan.handle, p["q"], stride, 1.0, p["k"], p["v"], p["ks"], p["vs"], p["pt"],
                                 p["out"], H * D, None, p["scratch"], b["n"], p["ws"], None) == status


def test_the_fp8_route_is_for_nvfp4(L):
    plan, b = _buffers("e4m3")
    p = {k: _ptr(v) for k, v in b.items() if k != "n"}
    assert L.sparse_prefill_fwd_fp8qk(plan.handle, p["q"], 1.0, p["k"], p["v"], p["ks"], p["vs"], p["pt"], p["idx"],
                                      p["partial"], T * H * D, p["lse"], T * H, p["ws"], None) == 2


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), 1), (dict(batch=-1), 1), (dict(batch=16385), 2), (dict(width=0), 1), (dict(width=131073), 1),
    (dict(room=-1), 1), (dict(room=1 << 31), 1), (dict(free_n=-1), 1), (dict(free_n=1 << 31), 1),
    (dict(q=None), 1), (dict(c=None), 1), (dict(free=None), 1), (dict(state=None), 1), (dict(table=None), 1),
    (dict(slots=4), 1), (dict(positions=2), 1), (dict(starts=1), 1), (dict(status=2), 1), (dict(q=2), 1),
    (dict(state=1), 1), (dict(table=2), 1),
])
def test_page_tables_refusals(L, kw, status):
    buf = {n: _aligned(1 << 10) for n in ("q", "c", "free", "state", "table", "slots", "positions", "starts", "status")}
    a = dict(batch=3, free_n=20, width=8, room=10)
    p = {n: _ptr(b) for n, b in buf.items()}
    for k, v in kw.items():
        if k in a:
            a[k] = v
        else:
            p[k] = None if v is None else _ptr(buf[k], v)
    assert L.sps_page_tables(a["batch"], p["q"], p["c"], p["free"], a["free_n"], p["state"], p["table"], a["width"],
                             p["slots"], p["positions"], a["room"], p["starts"], p["status"], None) == status
    assert L.sps_last_error()


class _Reached(Exception):
    """Raised behind every check, where the stream is looked up: nothing is launched here."""


class _Stream:
    @property
    def cuda_stream(self):
        raise _Reached


def test_binding_checks_of_an_e4m3_cache():
    plan = B.Plan([T], [200], H, G, D, 1, 2, PAGES, kv_dtype="e4m3")
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    a = dict(k_cache=u8(PAGES, G, 128, D), v_cache=u8(PAGES, G, 128, D), k_scales=torch.ones(PAGES, G),
             v_scales=torch.ones(PAGES, G))
    pt, ws, scratch = torch.zeros((1, 2), dtype=torch.int32), u8(plan.workspace_bytes), u8(B.paged_attention_scratch(plan))

    def attention(k_cache, v_cache, k_scales, v_scales):
        B.paged_attention_fwd(plan, bf(T, H, D), 1.0, k_cache, v_cache, k_scales, v_scales, pt, bf(T, H, D), None,
                              scratch, ws, _Stream())

    def append(k_cache, v_cache, k_scales, v_scales):
        B.sps_kv_append_rope(plan, bf(T, G, D), bf(T, G, D), None, 1e-6, None, pt, k_cache, v_cache, k_scales,
                             v_scales, ws, _Stream())

    for call in (attention, append):
        with pytest.raises(_Reached):
            call(**a)
        with pytest.raises(_Reached):  # more pages than the plan's, as FP8
            call(**dict(a, k_cache=torch.zeros((PAGES + 2, G, 128, D)).to(torch.float8_e4m3fn), k_scales=torch.ones(PAGES + 2, G)))
        for n in ("k_cache", "v_cache"):
            for bad in (a[n][:-1], bf(PAGES, G, 128, D), a[n].transpose(1, 2), a[n][..., ::2],
                        torch.zeros((PAGES, G, 128, D)).to(torch.float8_e5m2)):
                with pytest.raises(ValueError, match=n):
                    call(**dict(a, **{n: bad}))
        for n in ("k_scales", "v_scales"):
            for bad in (None, a[n][:-1], a[n].double(), a[n].bfloat16(), torch.ones(G, PAGES).T):
                with pytest.raises(ValueError, match=n):
                    call(**dict(a, **{n: bad}))


def test_binding_checks_of_page_tables():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    a = dict(q_lens=i32(3), ctx_lens=i32(3), free_pages=i32(9), free_state=i32(2), page_table=i32(4, 8),
             slots=torch.zeros(10, dtype=torch.int64), positions=i32(10), starts=i32(4), dev_status=i32(1))
    call = lambda **kw: B.sps_page_tables(**dict(a, **kw), stream=_Stream())
    for good in ({}, dict(slots=None), dict(positions=None), dict(starts=None, dev_status=None), dict(slots=None, positions=None)):
        with pytest.raises(_Reached):
            call(**good)
    for n, bad in (("q_lens", a["q_lens"].long()), ("ctx_lens", i32(2)), ("ctx_lens", i32(6)[::2]), ("free_state", i32(1)),
                   ("free_pages", i32(9).float()), ("page_table", i32(2, 8)), ("page_table", i32(4, 8).long()),
                   ("page_table", i32(8, 4).T), ("page_table", i32(32)), ("slots", i32(10)), ("positions", i32(9)),
                   ("starts", i32(3)), ("dev_status", i32(2))):
        with pytest.raises(ValueError, match=n):
            call(**{n: bad})
