"""What the binding refuses over an E4M3 K/V cache in the calls that take bare addresses for the other caches
(the plain append, the sparse forwards, the indexer); nothing is launched."""
import pytest

torch = pytest.importorskip("torch")

from paged_top_sparse_gb300 import binding as B
from paged_top_sparse_gb300 import build

T, H, G, D, PAGES, K = 3, 4, 2, 128, 5, 2


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


class _Reached(Exception):
    """Raised behind every check, where the stream is looked up."""


class _Stream:
    @property
    def cuda_stream(self):
        raise _Reached


u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
i32 = lambda *s: torch.zeros(s, dtype=torch.int32)


def _calls(plan, kc, vc, ks, vs):
    pt, ws, idx, q = i32(1, 2), u8(plan.workspace_bytes), i32(T, H, K), bf(T, H, D)
    lse = torch.zeros(K, T * H)
    yield lambda: B.sps_kv_append(plan, bf(T, G, D), bf(T, G, D), pt, kc, vc, ks, vs, ws, _Stream())
    for fwd, dt in ((B.sparse_prefill_fwd, torch.float32), (B.sparse_prefill_fwd_f16, torch.float16),
                    (B.sparse_prefill_fwd_bf16, torch.bfloat16), (B.sparse_prefill_fwd_fp8qk, torch.float32)):
        yield lambda f=fwd, d=dt: f(plan, q, 1.0, kc, vc, ks, vs, pt, idx, torch.zeros(K, T * H, D, dtype=d), lse,
                                    ws, _Stream())
    yield lambda: B.sparse_prefill_fwd_noalloc(plan, q, 1.0, kc, vc, ks, vs, pt, idx, torch.zeros(K, T * H, D), lse,
                                               None, _Stream())


def test_caches_and_scales_are_the_plans():
    plan = B.Plan([T], [200], H, G, D, K, 2, PAGES, kv_dtype="e4m3")
    good = dict(kc=u8(PAGES, G, 128, D), vc=u8(PAGES, G, 128, D), ks=torch.ones(PAGES, G), vs=torch.ones(PAGES, G))
    for call in _calls(plan, **good):
        with pytest.raises(_Reached):
            call()
    more = dict(kc=torch.zeros((PAGES + 2, G, 128, D)).to(torch.float8_e4m3fn), ks=torch.ones(PAGES + 2, G))
    for call in _calls(plan, **dict(good, **more)):  # more pages than the plan's, as FP8
        with pytest.raises(_Reached):
            call()
    for n, name in (("kc", "k_cache"), ("vc", "v_cache")):
        for bad in (good[n][:-1], bf(PAGES, G, 128, D), good[n].transpose(1, 2), good[n][..., ::2]):
            for call in _calls(plan, **dict(good, **{n: bad})):
                with pytest.raises(ValueError, match=name):
                    call()
    for n, name in (("ks", "k_scales"), ("vs", "v_scales")):
        for bad in (None, good[n][:-1], good[n].bfloat16(), good[n].double(), torch.ones(G, PAGES).T):
            for call in _calls(plan, **dict(good, **{n: bad})):
                with pytest.raises(ValueError, match=name):
                    call()


@pytest.mark.parametrize("iq,ik", [(None, None), ("e4m3", "e4m3"), ("e4m3", "nvfp4")])
def test_index_keys_are_a_cache_of_their_own(iq, ik):
    """The four steps of another cache's call, with the E4M3 cache as index keys, would read twice its bytes as
    BF16."""
    plan = B.Plan([T], [200], H, G, D, K, 2, PAGES, kv_dtype="e4m3", idx_q_dtype=iq, idx_k_dtype=ik)
    keys, scales = {None: (bf(PAGES, G, 128, D), None), "e4m3": (u8(PAGES, G, 128, D), None),
                    "nvfp4": (u8(PAGES, G, 128, D // 2), u8(PAGES, G, 128, D // 16))}[ik]

    def call(k, s=scales):
        B.indexer_scores(plan, bf(T, H, D), 1.0, k, s, 1.0, i32(1, 2), torch.zeros(T * H, 4), u8(plan.workspace_bytes),
                         _Stream())

    with pytest.raises(_Reached):
        call(keys)
    for bad in (keys[:-1], keys.float(), keys.transpose(1, 2), keys[..., ::2]):
        with pytest.raises(ValueError, match="k_idx_cache"):
            call(bad)
    if ik is None:
        with pytest.raises(ValueError, match="k_idx_cache"):
            call(u8(PAGES, G, 128, D))
    if ik == "nvfp4":
        for bad in (None, scales[:-1], scales.float()):
            with pytest.raises(ValueError, match="k_idx_scales"):
                call(keys, bad)


@pytest.mark.parametrize("kv", ["bf16", "nvfp4"])
def test_other_caches_pass_as_they_did(kv):
    plan = B.Plan([T], [200], H, G, D, K, 2, PAGES, q_dtype="e4m3" if kv == "nvfp4" else "bf16", kv_dtype=kv)
    for call in _calls(plan, u8(7), u8(7), u8(7), None):
        with pytest.raises(_Reached):
            call()
