"""The sparse forward over an E4M3 cache whose slots behind a request's last token were never written: every
byte of a pool may be a NaN code."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_top_sparse_gb300 import build

    build.build()


def _forward(c, k, sel, kind):
    B, R = c.B, c.T * c.H
    dt = {"f16": torch.float16, "bf16": torch.bfloat16}.get(kind, torch.float32)
    partial = torch.full((k, R, c.D), 7.0, dtype=dt, device=DEV)
    lse = torch.full((k, R), 7.0, device=DEV)
    args = (c.plan, c.q, c.q_scale, c.kc, c.vc, c.ks, c.vs, c.pt, sel, partial, lse)
    if kind == "noalloc":
        B.sparse_prefill_fwd_noalloc(*args)
    else:
        {"f32": B.sparse_prefill_fwd, "f16": B.sparse_prefill_fwd_f16,
         "bf16": B.sparse_prefill_fwd_bf16}[kind](*args, c.ws)
    combine = {"f16": B.partial_combine_f16, "bf16": B.partial_combine_bf16}.get(kind, B.partial_combine)
    combine(partial, lse, c.out.view(R, c.D), c.lse.view(R))
    torch.cuda.synchronize()
    assert B.sps_read_device_status(c.plan, c.ws) == 0
    return partial, lse


@pytest.mark.parametrize("q", ["bf16", "e4m3"])
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16", "noalloc"])
@pytest.mark.parametrize("q_lens,ctx,H,G,D,k", [([200, 1, 70, 1], [900, 0, 128, 127], 8, 2, 128, 4),
                                                ([130, 3, 128], [0, 2500, 0], 4, 1, 64, 16),
                                                ([1, 1, 1, 2], [5000, 127, 300, 126], 32, 2, 128, 20),
                                                ([2] * 40, [61 * i for i in range(40)], 4, 2, 64, 3)])
def test_unwritten_slots_count_for_nothing(q_lens, ctx, H, G, D, k, kind, q):
    """The same bits whether the slots behind the last token hold NaN codes or finite ones."""
    from tests.test_gpu_attention_e4m3 import Case, _selection

    sides = [Case(H + k, q_lens, ctx, H, G, D, q, top_k=k, nan_tail=nan) for nan in (False, True)]
    assert torch.equal(sides[0].q.view(torch.uint8), sides[1].q.view(torch.uint8))
    sel = _selection(sides[0], k, 3)
    clean, nan = (_forward(c, k, sel, kind) for c in sides)
    for x, y in zip(clean, nan):
        assert torch.equal(x, y)
    assert bool(torch.isfinite(sides[1].out.float()).all())
    assert torch.equal(sides[0].out, sides[1].out) and torch.equal(sides[0].lse, sides[1].lse)


@pytest.mark.parametrize("q", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
def test_append_and_sparse_forward_on_a_pool_never_written(D, q):
    """Pages that this append alone has touched: the sparse forward of every page is full attention."""
    from paged_top_sparse_gb300 import binding as B

    q_lens, H, G, k = [300, 1, 129], 8, 2, 4
    T, NP = sum(q_lens), 3 + 1 + 2
    g = torch.Generator(device=DEV)
    g.manual_seed(D)
    plan = B.Plan(q_lens, [0] * 3, H, G, D, k, 3, NP, q_dtype=q, kv_dtype="e4m3")
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device=DEV)
    B.sps_plan_upload(plan, ws)
    pt = torch.tensor([[4, 1, 5], [0, -1, -1], [2, 3, -1]], dtype=torch.int32, device=DEV)
    kc, vc = (torch.full((NP, G, 128, D), 0x7F, dtype=torch.uint8, device=DEV) for _ in "kv")
    ks, vs = (torch.full((NP, G), float("nan"), device=DEV) for _ in "kv")
    new = torch.randn((2, T, G, D), generator=g, device=DEV).bfloat16()
    B.sps_kv_append(plan, new[0], new[1], pt, kc, vc, ks, vs, ws)
    x = torch.randn((T, H, D), generator=g, device=DEV)
    qs = 0.0117 if q == "e4m3" else 1.0
    x = (x / qs).clamp(-448, 448).to(torch.float8_e4m3fn) if q == "e4m3" else x.bfloat16()
    pos = torch.cat([torch.arange(n, device=DEV) for n in q_lens])
    page = torch.arange(k, device=DEV)
    sel = torch.where(page <= (pos // 128)[:, None], page, -1).int()[:, None].expand(T, H, k).contiguous()
    partial, lse = torch.empty((k, T * H, D), device=DEV), torch.empty((k, T * H), device=DEV)
    out, full = (torch.empty((T, H, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    B.sparse_prefill_fwd(plan, x, qs, kc, vc, ks, vs, pt, sel, partial, lse, ws)
    B.partial_combine(partial, lse, out.view(T * H, D))
    scratch = torch.empty(B.paged_attention_scratch(plan), dtype=torch.uint8, device=DEV)
    B.paged_attention_fwd(plan, x, qs, kc, vc, ks, vs, pt, full, None, scratch, ws)
    torch.cuda.synchronize()
    assert B.sps_read_device_status(plan, ws) == 0
    # each within an FP16 P (2^-11 of the weighted values, which are below the largest value) and half a
    # BF16 step of the definition
    big = new[1].float().abs().amax()
    tol = 2 * ((2.0 ** -11 + 2.0 ** -13) * big + 2.0 ** -8 * full.float().abs())
    assert bool(((out.float() - full.float()).abs() <= tol).all())
