"""What the binding of the norm, rotation, append and attention refuses before it calls the library."""
import pytest

torch = pytest.importorskip("torch")

from paged_top_sparse_gb300 import binding as B
from paged_top_sparse_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def test_page_table_rows_are_the_plans():
    """The kernels step max_pages_per_req entries from request to request: a table with wider rows
    would give request 1 the entries of request 0."""
    plan = B.Plan([1, 1, 1], [10, 300, 0], 4, 2, 64, 1, 3, 9)
    table = torch.zeros((8, 3), dtype=torch.int32)
    flat = torch.zeros(9, dtype=torch.int32)
    for good in (table[:3], table, flat, torch.zeros(20, dtype=torch.int32)):
        assert B._table(good, plan) == good.data_ptr()
    wide = torch.zeros((3, 4), dtype=torch.int32)
    for bad in (wide, torch.zeros((9, 2), dtype=torch.int32), wide[:, :3], table[:2], flat[:8],
                table.long(), torch.zeros((3, 1, 9), dtype=torch.int32)):
        with pytest.raises(ValueError, match="page_table"):
            B._table(bad, plan)


T, H, G, D, PAGES = 3, 4, 2, 64, 5


def _batch(kv):
    """A plan and tensors of the sizes it asks for; every case below spoils one of them."""
    quant = kv == "nvfp4"
    plan = B.Plan([T], [200], H, G, D, 1, 2, PAGES, q_dtype="e4m3" if quant else "bf16", kv_dtype=kv)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    cache = (PAGES, G, 128, D)
    a = dict(q=u8(T, H, D) if quant else bf(T, H, D), out=bf(T, H, D), k_new=bf(T, G, D), v_new=bf(T, G, D),
             k_cache=u8(*cache[:3], D // 2) if quant else bf(*cache),
             v_cache=u8(*cache[:3], D // 2) if quant else bf(*cache),
             k_scales=u8(*cache[:3], D // 16) if quant else None,
             v_scales=u8(*cache[:3], D // 16) if quant else None,
             page_table=torch.zeros((1, 2), dtype=torch.int32),
             scratch=u8(B.paged_attention_scratch(plan)), workspace=u8(plan.workspace_bytes))
    return plan, a


def _attention(plan, a):
    B.paged_attention_fwd(plan, a["q"], 1.0, a["k_cache"], a["v_cache"], a["k_scales"], a["v_scales"],
                          a["page_table"], a["out"], None, a["scratch"], a["workspace"], _Stream())


def _append(plan, a):
    B.sps_kv_append_rope(plan, a["k_new"], a["v_new"], None, 1e-6, None, a["page_table"], a["k_cache"],
                         a["v_cache"], a["k_scales"], a["v_scales"], a["workspace"], _Stream())


def _norm(plan, a):
    B.sps_qk_norm_rope(plan, a["out"], None, None, None, 1e-6, None, a["out"], 1.0, None,
                       a["workspace"], _Stream())


class _Reached(Exception):
    """Raised behind every check, where the stream is looked up: nothing is launched here."""


class _Stream:
    @property
    def cuda_stream(self):
        raise _Reached


SHORT = lambda t: t[:-1]
ROWS = lambda t: t[:, :, :, ::2]
CACHES = {
    "bf16": [lambda t: t.to(torch.uint8), lambda t: t.half(), lambda t: t.float(), SHORT, ROWS,
             lambda t: t.transpose(1, 2)],
    "nvfp4": [lambda t: t.to(torch.bfloat16), lambda t: t.int(), SHORT, ROWS, lambda t: t.transpose(1, 2)],
}


@pytest.mark.parametrize("kv", ["bf16", "nvfp4"])
@pytest.mark.parametrize("call", [_attention, _append])
def test_caches_and_scales_are_the_plans(call, kv):
    plan, a = _batch(kv)
    with pytest.raises(_Reached):
        call(plan, a)
    for name in ("k_cache", "v_cache"):
        for spoil in CACHES[kv]:
            with pytest.raises(ValueError, match=name):
                call(plan, dict(a, **{name: spoil(a[name])}))
        # more pages than the plan's, or raw bits of the elements, are no mistake
        more = torch.zeros((PAGES + 1, *a[name].shape[1:]), dtype=torch.uint8 if kv == "nvfp4" else torch.int16)
        with pytest.raises(_Reached):
            call(plan, dict(a, **{name: more}))
    if kv == "nvfp4":
        for name in ("k_scales", "v_scales"):
            for bad in (None, SHORT(a[name]), a[name].half(), a[name].transpose(1, 2)):
                with pytest.raises(ValueError, match=name):
                    call(plan, dict(a, **{name: bad}))


@pytest.mark.parametrize("call", [_attention, _append, _norm])
def test_a_short_workspace_is_refused(call):
    plan, a = _batch("bf16")
    with pytest.raises(_Reached):
        call(plan, a)
    with pytest.raises(ValueError, match="workspace"):
        call(plan, dict(a, workspace=a["workspace"][:-1]))
