"""GPU checks of paged_attention_fwd over long runs of work: waits that outlast their limit while the
block's other work goes on."""
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


@pytest.mark.parametrize("kv", ["bf16", "nvfp4"])
@pytest.mark.parametrize("H,D,last_q", [(16, 128, 16), (2, 64, 1)])
def test_a_wait_beside_other_work_does_not_time_out(H, D, last_q, kv):
    """Blocks of 400 one-page pieces of which the last alone needs the second softmax warpgroup (16
    tokens of 16 heads: two row tiles) and has slots behind its last token: the roles that take part
    in that piece only wait for longer than their limit, while pieces come and go.

    The requests cost one page each and fill every block alike, so that the plan's runs are whole
    tiles in order, and no others would be shorter."""
    from paged_top_sparse_gb300 import binding as B

    ctas = min(torch.cuda.get_device_properties(0).multi_processor_count, 256)
    per, pages, limit_us = 400, 4, 200
    n = ctas * per
    q_lens = [last_q if i % per == per - 1 else 1 for i in range(n)]
    ctx = [100 if i % per == per - 1 else 127 for i in range(n)]
    T = sum(q_lens)
    g = torch.Generator(device=DEV)
    g.manual_seed(H)
    req = torch.repeat_interleave(torch.arange(n, device=DEV), torch.tensor(q_lens, device=DEV))
    pt = (torch.arange(n, dtype=torch.int32, device=DEV) % pages)[:, None].contiguous()
    quant = kv == "nvfp4"
    ks = vs = None
    if quant:  # any codes, scales of 1 / 4 (0x28)
        kc, vc = (torch.randint(0, 256, (pages, 1, 128, D // 2), generator=g, device=DEV,
                                dtype=torch.uint8) for _ in "kv")
        ks, vs = (torch.full((pages, 1, 128, D // 16), 0x28, dtype=torch.uint8, device=DEV)
                  for _ in "kv")
        kd, vd = (torch.empty((pages, 128, D), dtype=torch.float16, device=DEV) for _ in "kv")
        for c, s, o in ((kc, ks, kd), (vc, vs, vd)):
            B.sps_dequantize("nvfp4", c, s, o.numel(), o)
        q = torch.randn((T, H, D), generator=g, device=DEV).to(torch.float8_e4m3fn)
    else:
        kc, vc = (torch.randn((pages, 1, 128, D), generator=g, device=DEV).bfloat16() for _ in "kv")
        kd, vd = kc[:, 0], vc[:, 0]
        q = torch.randn((T, H, D), generator=g, device=DEV).bfloat16()
    plan = B.Plan(q_lens, ctx, H, 1, D, 1, 1, pages, q_dtype="e4m3" if quant else "bf16", kv_dtype=kv)
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device=DEV)
    B.sps_plan_upload(plan, ws)
    scratch = torch.empty(B.paged_attention_scratch(plan), dtype=torch.uint8, device=DEV)
    out = torch.empty((T, H, D), dtype=torch.bfloat16, device=DEV)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    B.lib().sps_internal_attention_wait(limit_us * 1000)
    try:
        torch.cuda.synchronize()
        a.record()
        B.paged_attention_fwd(plan, q, 1.0, kc, vc, ks, vs, pt, out, None, scratch, ws)
        b.record()
        torch.cuda.synchronize()
    finally:
        B.lib().sps_internal_attention_wait(0)
    assert B.sps_read_device_status(plan, ws) == 0
    assert a.elapsed_time(b) * 1000 > 2 * limit_us  # the waits did last longer than their limit
    # in FP64: P rounded by half a step of its type, the output by half a BF16 step
    p_half = 2.0 ** -11 if quant else 2.0 ** -8
    i0 = torch.cumsum(torch.tensor(q_lens, device=DEV), 0) - torch.tensor(q_lens, device=DEV)
    pos = torch.tensor(ctx, device=DEV)[req] + torch.arange(T, device=DEV) - i0[req]
    for page in range(pages):
        rows = (req % pages == page).nonzero()[:, 0]
        for r in rows.split(4096):
            s = q[r].double() @ kd[page].double().T * D ** -0.5
            s.masked_fill_(torch.arange(128, device=DEV) > pos[r][:, None, None], -float("inf"))
            p = torch.softmax(s, -1)
            ref, mag = p @ vd[page].double(), p @ vd[page].double().abs()
            tol = (p_half + 2.0 ** -14) * mag + 2.0 ** -8 * ref.abs()
            if quant:
                tol = tol + 128 * 2.0 ** -32 * 16
            assert bool(((out[r].double() - ref).abs() <= tol).all())
