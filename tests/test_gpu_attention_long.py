"""GPU checks of paged_attention_fwd over long runs of work: waits that outlast their limit while the
block's other work goes on, answers that depend on single pages, and long contexts against bounds that a
lost or wrong page breaks."""
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


def _needles(kv, H, G, D, q_lens, ctx, seed):
    """A cache in which every page holds one key of +-1.5 in directions of its own, at a slot of its
    own, among keys of deviation 1 or less, and queries 4 times such a direction: with `a` = 4 and
    `b` = 1.5 that key scores a b sqrt(D) (48 at D 64, 68 at 128), every other at most about 6 a b.
    A row's softmax is then that key's alone, to e^-18."""
    from paged_top_sparse_gb300 import binding as B

    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    pages = (ctx + q_lens - 1) // 128 + 1
    quant = kv == "nvfp4"
    sign = torch.randint(0, 2, (pages, G, D), generator=g, device=DEV, dtype=torch.uint8)
    slot = (torch.arange(pages, device=DEV) * 37 + 5) % 128
    slot[-1] %= (ctx % 128) + 1 if ctx // 128 == pages - 1 else 1
    page = torch.arange(pages, device=DEV)
    ks = vs = None
    if quant:
        codes = lambda: torch.randint(0, 256, (pages, G, 128, D // 2), generator=g, device=DEV,
                                      dtype=torch.uint8)
        kc, vc = codes(), codes()
        ks, vs = (torch.full((pages, G, 128, D // 16), 0x28, dtype=torch.uint8, device=DEV)
                  for _ in "kv")  # 1 / 4
        c = 3 + 8 * sign  # +-1.5
        kc[page, :, slot] = c[..., 0::2] | (c[..., 1::2] << 4)
        ks[page, :, slot] = 0x38  # 1
        want = torch.empty((pages, G, D), dtype=torch.float16, device=DEV)
        B.sps_dequantize("nvfp4", vc[page, :, slot].contiguous(), vs[page, :, slot].contiguous(),
                         want.numel(), want)
    else:
        kc, vc = (torch.randn((pages, G, 128, D), generator=g, device=DEV).bfloat16() for _ in "kv")
        kc[page, :, slot] = (1.5 - 3.0 * sign).bfloat16()
        want = vc[page, :, slot]
    queries = 4.0 - 8.0 * sign.float()
    queries = queries.to(torch.float8_e4m3fn) if quant else queries.bfloat16()
    table = torch.randperm(pages, generator=g, device=DEV)
    # physical page table[i] holds what page i of the request is
    place = lambda x: None if x is None else torch.empty_like(x).index_copy_(0, table, x)
    kc, vc, ks, vs = (place(x) for x in (kc, vc, ks, vs))
    plan = B.Plan([q_lens], [ctx], H, G, D, 1, pages, pages, q_dtype="e4m3" if quant else "bf16",
                  kv_dtype=kv)
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
        assert bool(((out.double() - w).abs() <= (2.0 ** -7 + 2.0 ** -14) * w.abs() + 2.0 ** -16).all())
        assert bool(((lse.double() - 6.0 * D ** 0.5).abs() <= 2.0 ** -12).all())

    return ask, pages, lambda: B.sps_read_device_status(plan, ws)


@pytest.mark.parametrize("kv", ["bf16", "nvfp4"])
@pytest.mark.parametrize("H,q", [(8, 1), (16, 1), (16, 3)])
def test_every_page_of_a_1m_context_is_read_where_it_lies(H, q, kv):
    """8192 pages in pieces of about 54 over the SMs, every one of them asked for: the first and last
    of each piece and those on both sides of a reload of page numbers among them."""
    ask, pages, status = _needles(kv, H, 1, 64, q, (1 << 20) - q, 11 * H + q)
    assert pages == 8192
    rows = q * H
    for i in range(0, pages, rows):
        ask(((i + torch.arange(rows, device=DEV)) % pages).view(q, H))
    assert status() == 0


@pytest.mark.parametrize("kv", ["bf16", "nvfp4"])
@pytest.mark.parametrize("D", [64, 128])
def test_every_page_of_a_chunk_is_read_where_it_lies(D, kv):
    """1200 tokens after 20,000, two row tiles a work tile in pieces of some 80 pages: every row asks
    for a page of its own choice, every page is asked for by many rows of every tile."""
    H, G, T, ctx = 16, 2, 1200, 20000
    ask, pages, status = _needles(kv, H, G, D, T, ctx, D)
    before = ctx // 128  # pages that every row sees
    r = torch.arange(T * H, device=DEV).view(T, H)
    for step in (1, 7, 41):
        ask(r * step % before)
    assert status() == 0


def _bounds(c, drop=None, swap=None):
    """FP64 results of a Case, and the tolerances of random data; `drop`, `swap`: mistakes planted in
    request 0, pages left out and pages whose values are read in reverse order."""
    T, H, G, D = c.T, c.H, c.G, c.D
    out = torch.zeros((T, H, D), dtype=torch.float64, device=DEV)
    lse = torch.zeros((T, H), dtype=torch.float64, device=DEV)
    tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    t0 = 0
    p_half = 2.0 ** -8 if c.kv == "bf16" else 2.0 ** -11
    for b, (ql, ctx) in enumerate(zip(c.q_lens, c.ctx)):
        ids = c.pt[b, :c.pages[b]].long()
        vids = ids.clone()
        if b == 0 and swap is not None:
            vids[swap] = vids[swap].flip(0)
        n = ctx + ql
        for g in range(G):
            k, v = c.kd[ids, g].reshape(-1, D)[:n], c.vd[vids, g].reshape(-1, D)[:n]
            h = slice(g * (H // G), (g + 1) * (H // G))
            s = (c.qd[t0:t0 + ql, h].reshape(-1, D) @ k.T * D ** -0.5).view(ql, H // G, n)
            pos = ctx + torch.arange(ql, device=DEV)
            s.masked_fill_(torch.arange(n, device=DEV) > pos[:, None, None], -float("inf"))
            if b == 0 and drop is not None:
                s[..., drop.start * 128:drop.stop * 128] = -float("inf")
            z = torch.logsumexp(s, -1, keepdim=True)
            p = torch.exp(s - z)
            out[t0:t0 + ql, h], lse[t0:t0 + ql, h] = p @ v, z[..., 0]
            # Roundings of P and errors of the FP32 chain in front of it (2^-14) are independent from
            # key to key: six deviations of a sum of terms that are each at most (half step) p |v|.
            # The output's half step, and 2^-18 of sum p |v| for sums that are cut off, not rounded.
            # FP16 P below its normal range: 2^-32 of the largest p, per key.
            t = 6 * (p_half + 2.0 ** -14) * ((p * p) @ (v * v)).sqrt()
            t += 2.0 ** -8 * out[t0:t0 + ql, h].abs() + 2.0 ** -18 * (p @ v.abs())
            if c.kv != "bf16":
                t += 6 * 2.0 ** -32 * n ** 0.5 * v.abs().max()
            tol[t0:t0 + ql, h] = t
            # a row's sum: at least four accumulators, each addition off by 2^-24 either way
            lse_tol[t0:t0 + ql, h] = 2.0 ** -13 + 6 * (n / 4) ** 0.5 * 2.0 ** -24 + z[..., 0].abs() * 2.0 ** -22
        t0 += ql
    return out, lse, tol, lse_tol


def _violations(c, **planted):
    out, lse, tol, lse_tol = _bounds(c, **planted)
    return (int(((c.out.double() - out).abs() > tol).sum()),
            int(((c.lse.double() - lse).abs() > lse_tol).sum()))


@pytest.mark.parametrize("kv", ["bf16", "nvfp4"])
@pytest.mark.parametrize("q_lens,ctx,H,G,D", [
    ([1], [(1 << 20) - 1], 8, 1, 64), ([1, 1], [30000, 9000], 16, 1, 128), ([40, 3], [20000, 700], 16, 2, 128),
])
def test_long_contexts_to_the_roundings_of_random_data(q_lens, ctx, H, G, D, kv):
    """Outputs of a long context are small (1 / sqrt(keys)), so a bound by sum p |v| would hide pages
    that are lost or read from elsewhere; the same mistakes planted in the oracle break this one."""
    from tests.test_gpu_attention import Case

    c = Case(sum(ctx) % 997, q_lens, ctx, H, G, D, kv)
    c.run()
    torch.cuda.synchronize()
    assert c.B.sps_read_device_status(c.plan, c.ws) == 0
    assert _violations(c) == (0, 0)
    n = c.pages[0]
    piece = slice(n // 3, n // 3 + max(2, n // 152))  # what one SM reads of the request, about
    lost = _violations(c, drop=piece)
    assert lost[0] > 0 and lost[1] > 0
    assert _violations(c, swap=slice(n // 3, n // 3 + max(2, n // 40)))[0] > 0


@pytest.mark.parametrize("kv,bound", [("bf16", 2.5e-3), ("nvfp4", 1.8e-3)])
def test_relative_error_of_random_data(kv, bound):
    """Rounding a value of any significand to BF16 costs 2^-8 / sqrt(3) sqrt(3 / (8 ln 2)) = 1.66e-3 of
    it in the mean square (2^-3 of that in FP16): once for P over a BF16 cache and once for the output
    they make 2.35e-3, with P in FP16 1.67e-3."""
    from tests.test_gpu_attention import Case

    c = Case(71, [300, 1, 1], [900, 5000, 20000], 16, 2, 128, kv)
    c.run()
    torch.cuda.synchronize()
    out = c.reference()[0]
    for t0, t1 in ((0, 300), (300, 301), (301, 302)):
        err = (c.out[t0:t1].double() - out[t0:t1]).norm() / out[t0:t1].norm()
        # (one row set of 16 x 128 elements: the mean square's own deviation is 2 %)
        assert float(err) <= bound * (1.06 if t1 - t0 == 1 else 1.0), float(err)
