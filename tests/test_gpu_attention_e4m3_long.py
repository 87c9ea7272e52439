"""GPU checks of paged_attention_fwd over long runs of work on an E4M3 cache: waits that outlast their limit
while the block's other work goes on, answers and scales that depend on single pages, and the relative error
of random data."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_top_sparse_gb300 import build

    build.build()


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("H,D,last_q", [(16, 128, 16), (64, 64, 4), (2, 64, 1)])
def test_a_wait_beside_other_work_does_not_time_out(H, D, last_q, quant):
    """Blocks of 400 one-page pieces of which the last alone needs the second softmax warpgroup (two row
    tiles): it waits for longer than its limit, while pieces come and go.  (The last form is of tiles of
    few rows, whose warps all take part in every piece.)"""
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
    kc, vc = ((torch.randn((pages, 1, 128, D), generator=g, device=DEV) * 100).to(F8) for _ in "kv")
    ks, vs = ((1 + torch.rand((pages, 1), generator=g, device=DEV)) / 128 for _ in "kv")
    kd, vd = ((c.double() * s.double()[:, :, None, None])[:, 0] for c, s in ((kc, ks), (vc, vs)))
    q = torch.randn((T, H, D), generator=g, device=DEV)
    q = q.to(F8) if quant else q.bfloat16()
    plan = B.Plan(q_lens, ctx, H, 1, D, 1, 1, pages, q_dtype="e4m3" if quant else "bf16", kv_dtype="e4m3")
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
    if H >= 16:
        assert a.elapsed_time(b) * 1000 > 2 * limit_us  # the waits did last longer than their limit
    i0 = torch.cumsum(torch.tensor(q_lens, device=DEV), 0) - torch.tensor(q_lens, device=DEV)
    pos = torch.tensor(ctx, device=DEV)[req] + torch.arange(T, device=DEV) - i0[req]
    for page in range(pages):
        rows = (req % pages == page).nonzero()[:, 0]
        for r in rows.split(2048):
            s = q[r].double() @ kd[page].T * D ** -0.5
            s.masked_fill_(torch.arange(128, device=DEV) > pos[r][:, None, None], -float("inf"))
            p = torch.softmax(s, -1)
            ref, mag = p @ vd[page], p @ vd[page].abs()
            # P to FP16, the output to BF16, the FP32 chain 2^-14; P below its normal range
            tol = (2.0 ** -11 + 2.0 ** -14) * mag + 2.0 ** -8 * ref.abs() + 128 * 2.0 ** -32 * 8
            err = (out[r].double() - ref).abs()
            # a draw beyond 464 is a NaN code: NaN in the rows that see it (0 x NaN in the others here)
            nan = ref.isnan() & (out[r].isnan() | (pos[r] < 127)[:, None, None])
            bad = (~((err <= tol) | nan)).nonzero()
            assert not len(bad), (len(bad), r[bad[:4, 0]].tolist(), bad[:4].tolist())


def _needles(quant, H, G, D, q_lens, ctx, seed):
    """A cache in which every page holds one key of +-1.5 in directions of its own, at a slot of its own,
    among keys of deviation 1 / 2 or less, under scales of its own, and queries 4 times such a direction:
    that key scores 6 sqrt(D) (48 at D 64, 68 at 128), every other at most about half as much.  A row's
    softmax is then that key's alone, to e^-18."""
    from paged_top_sparse_gb300 import binding as B

    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    pages = (ctx + q_lens - 1) // 128 + 1
    sign = torch.randint(0, 2, (pages, G, D), generator=g, device=DEV)
    slot = (torch.arange(pages, device=DEV) * 37 + 5) % 128
    slot[-1] %= (ctx % 128) + 1 if ctx // 128 == pages - 1 else 1
    page = torch.arange(pages, device=DEV)
    # powers of two from page to page: the needle's code is 1.5 / scale
    ks, vs = (torch.exp2(-torch.randint(0, 7, (pages, G), generator=g, device=DEV).float()) for _ in "kv")
    kc = (torch.randn((pages, G, 128, D), generator=g, device=DEV) * 0.25 / ks[:, :, None, None]).clamp(-448, 448).to(F8)
    vc = (torch.randn((pages, G, 128, D), generator=g, device=DEV) * 16).clamp(-448, 448).to(F8)
    kc.view(torch.uint8)[page, :, slot] = ((1.5 - 3.0 * sign) / ks[:, :, None]).to(F8).view(torch.uint8)
    want = vc.view(torch.uint8)[page, :, slot].view(F8).float() * vs[:, :, None]
    queries = 4.0 - 8.0 * sign.float()
    queries = queries.to(F8) if quant else queries.bfloat16()
    table = torch.randperm(pages, generator=g, device=DEV)

    def place(x):  # physical page table[i] holds what page i of the request is
        raw = x.view(torch.uint8) if x.dtype == F8 else x
        return torch.empty_like(raw).index_copy_(0, table, raw).view(x.dtype)

    kc, vc, ks, vs = (place(x) for x in (kc, vc, ks, vs))
    plan = B.Plan([q_lens], [ctx], H, G, D, 1, pages, pages, q_dtype="e4m3" if quant else "bf16", kv_dtype="e4m3")
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device=DEV)
    B.sps_plan_upload(plan, ws)
    scratch = torch.full((B.paged_attention_scratch(plan),), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.empty((q_lens, H, D), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((q_lens, H), device=DEV)
    pt = table.int()[None].contiguous()

    def ask(which):
        """which [tokens][H]: the page that each row's query points to."""
        group = torch.arange(H, device=DEV) // (H // G)
        q = queries.view(torch.uint8 if quant else torch.int16)[which, group].view(queries.dtype)
        B.paged_attention_fwd(plan, q, 1.0, kc, vc, ks, vs, pt, out, lse, scratch, ws)
        # the softmax is one key's: its value with P and the output rounded once each, its score
        w = want[which, group].double()
        assert bool(((out.double() - w).abs() <= (2.0 ** -8 + 2.0 ** -10) * w.abs() + 2.0 ** -16).all())
        assert bool(((lse.double() - 6.0 * D ** 0.5).abs() <= 2.0 ** -12).all())

    return ask, pages, lambda: B.sps_read_device_status(plan, ws)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("H,q", [(8, 1), (16, 1), (16, 3)])
def test_every_page_of_a_1m_context_is_read_where_it_lies(H, q, quant):
    """8192 pages in pieces of about 54 over the SMs, every one of them asked for, under its own scales."""
    ask, pages, status = _needles(quant, H, 1, 64, q, (1 << 20) - q, 11 * H + q)
    assert pages == 8192
    rows = q * H
    for i in range(0, pages, rows):
        ask(((i + torch.arange(rows, device=DEV)) % pages).view(q, H))
    assert status() == 0


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_every_page_of_a_chunk_is_read_where_it_lies(D, quant):
    """1200 tokens after 20,000, two row tiles a work tile: every row asks for a page of its own choice,
    every page is asked for by many rows of every tile."""
    H, G, T, ctx = 16, 2, 1200, 20000
    ask, pages, status = _needles(quant, H, G, D, T, ctx, D)
    r = torch.arange(T * H, device=DEV).view(T, H)
    for step in (1, 7, 41):
        ask(r * step % (ctx // 128))  # pages that every row sees
    assert status() == 0


@pytest.mark.parametrize("q", ["bf16", "e4m3"])
def test_relative_error_of_random_data(q):
    """Rounding a value of any significand to BF16 costs 1.66e-3 of it in the mean square; with P in FP16
    (an eighth of that) the output is off by 1.67e-3."""
    from tests.test_gpu_attention_e4m3 import Case

    c = Case(71, [300, 1, 1, 2], [900, 5000, 20000, 3000], 16, 2, 128, q)
    c.run()
    torch.cuda.synchronize()
    out = c.reference()[0]
    for t0, t1 in ((0, 300), (300, 301), (301, 302), (302, 304)):
        err = (c.out[t0:t1].double() - out[t0:t1]).norm() / out[t0:t1].norm()
        # (one row set of 16 x 128 elements: the mean square's own deviation is 2 %)
        assert float(err) <= 1.8e-3 * (1.06 if t1 - t0 < 3 else 1.0), float(err)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("q_lens,ctx", [([150, 1], [300, 0]), ([1, 2], [500, 700])])
def test_pages_whose_offsets_pass_32_bits(q_lens, ctx, quant):
    """The same append, attention and sparse forward in a small pool and in pages at the end of one of
    4.6 GB: the same bits."""
    from paged_top_sparse_gb300 import binding as B

    H, G, D, pool = 16, 2, 128, 140_000
    g = torch.Generator(device=DEV)
    g.manual_seed(len(q_lens) + ctx[0])
    total = [a + b for a, b in zip(q_lens, ctx)]
    pages = [(n + 127) // 128 for n in total]
    T, S = sum(q_lens), sum(total)
    k, v = (torch.randn((S, G, D), generator=g, device=DEV).bfloat16() for _ in "kv")
    q = torch.randn((T, H, D), generator=g, device=DEV) * 4
    q = q.to(F8) if quant else q.bfloat16()
    qt, width = "e4m3" if quant else "bf16", max(pages)
    sel = torch.full((T, H, 8), -1, dtype=torch.int32, device=DEV)
    pos = torch.cat([torch.arange(c, c + n, device=DEV) for n, c in zip(q_lens, ctx)])
    page = torch.arange(8, device=DEV, dtype=torch.int32).expand(T, H, 8)
    sel = torch.where(page <= (pos // 128)[:, None, None], page, sel)
    results = []
    for phys in (sum(pages), pool):
        table = torch.full((len(q_lens), width), -1, dtype=torch.int32, device=DEV)
        at = phys - 1
        for b, n in enumerate(pages):
            table[b, :n] = torch.arange(at, at - n, -1, device=DEV, dtype=torch.int32)
            at -= n
        used = torch.cat([table[b, :n] for b, n in enumerate(pages)]).long()
        kc, vc = (torch.empty((phys, G, 128, D), dtype=torch.uint8, device=DEV) for _ in "kv")
        ks, vs = (torch.zeros((phys, G), device=DEV) for _ in "kv")
        kc[used] = 0
        vc[used] = 0
        kc, vc = kc.view(F8), vc.view(F8)
        out, lse = torch.empty((T, H, D), dtype=torch.bfloat16, device=DEV), torch.empty((T, H), device=DEV)
        part, plse = torch.zeros((8, T * H, D), device=DEV), torch.empty((8, T * H), device=DEV)
        fill = B.Plan(total, [0] * len(total), H, G, D, 1, width, phys, q_dtype=qt, kv_dtype="e4m3")
        plan = B.Plan(q_lens, ctx, H, G, D, 8, width, phys, q_dtype=qt, kv_dtype="e4m3")
        for p in (fill, plan):
            ws = torch.zeros(p.workspace_bytes, dtype=torch.uint8, device=DEV)
            B.sps_plan_upload(p, ws)
            if p is fill:
                B.sps_kv_append(p, k, v, table, kc, vc, ks, vs, ws)
        scratch = torch.empty(B.paged_attention_scratch(plan), dtype=torch.uint8, device=DEV)
        B.paged_attention_fwd(plan, q, 0.5, kc, vc, ks, vs, table, out, lse, scratch, ws)
        B.sparse_prefill_fwd(plan, q, 0.5, kc, vc, ks, vs, table, sel, part, plse, ws)
        torch.cuda.synchronize()
        assert B.sps_read_device_status(plan, ws) == 0
        results.append([x.clone() for x in (kc.view(torch.uint8)[used], vc.view(torch.uint8)[used], ks[used],
                                            vs[used], out.view(torch.int16), lse, part, plse)])
    assert int(results[0][0].count_nonzero()) > 0 and bool(results[0][4].any())
    for a, b in zip(*results):
        assert torch.equal(a, b)
