"""GPU checks of full attention (paged_attention_fwd) and of the sparse forward over an E4M3 cache with a
scale for each page and KV head, against the definition in 64 bits: head layouts, ragged batches of
chunks and single tokens, page borders, long contexts, NaN in unwritten slots, growing scores, scales
that differ from page to page, strided views and graph replay."""
import numpy as np
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


class Case:
    """A batch with its caches, filled; every slot behind a request's last token holds a NaN code.
    ``k_gain`` / ``v_gain``: a factor on the scales of a request's page i."""

    def __init__(self, seed, q_lens, ctx, H, G, D, q="bf16", k_gain=None, v_gain=None, q_pad=0,
                 out_pad=0, top_k=1, max_pages=None, nan_tail=True, q_mag=None):
        from paged_top_sparse_gb300 import binding as B

        self.B = B
        self.q_lens, self.ctx, self.H, self.G, self.D, self.qt = q_lens, ctx, H, G, D, q
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        randn = lambda *s: torch.randn(s, generator=g, device=DEV)
        self.pages = pages = [(c + n - 1) // 128 + 1 if n else 0 for n, c in zip(q_lens, ctx)]
        NP, T = sum(pages), sum(q_lens)
        self.T, self.NP = T, NP
        perm = np.random.default_rng(seed).permutation(NP).astype(np.int32)
        pt = np.full((len(q_lens), max_pages or max(pages)), -1, np.int32)  # unused: out of range
        at = 0
        for b, n in enumerate(pages):
            pt[b, :n] = perm[at:at + n]
            at += n
        self.pt = torch.from_numpy(pt).to(DEV)
        # codes as quantised values are (most of them far below 448), scales of any FP32 value
        self.kc, self.vc = ((randn(NP, G, 128, D) * 100).clamp(-448, 448).to(F8) for _ in "kv")
        self.ks = (0.5 + torch.rand((NP, G), generator=g, device=DEV)) / 100
        self.vs = torch.exp2(4 * torch.rand((NP, G), generator=g, device=DEV) - 2) / 100
        for gain, s in ((k_gain, self.ks), (v_gain, self.vs)):
            if gain is not None:
                for b, n in enumerate(pages):
                    for i in range(n):
                        s[pt[b, i]] *= gain(i)
        self.kd, self.vd = (c.double() * s.double()[:, :, None, None]
                            for c, s in ((self.kc, self.ks), (self.vc, self.vs)))
        tail = torch.zeros((NP, 128), dtype=torch.bool, device=DEV)
        for b, n in enumerate(pages):
            if n:
                tail[pt[b, n - 1], (ctx[b] + q_lens[b] - 1) % 128 + 1:] = True
        if nan_tail:
            for c in (self.kc, self.vc):
                c.view(torch.uint8).transpose(1, 2)[tail] = 0x7F
        if q == "bf16":
            self.q_scale = 1.0
            x = randn(T, H + q_pad, D)
            if q_mag is not None:
                x = x * q_mag(T, H + q_pad, g)
            self.q = x.bfloat16()[:, :H]
            self.qd = self.q.double()
        else:
            self.q_scale = 0.0117
            self.q = (randn(T, H + q_pad, D) / self.q_scale).clamp(-448, 448).to(F8)[:, :H]
            self.qd = self.q.double() * self.q_scale
        self.plan = B.Plan(q_lens, ctx, H, G, D, top_k, pt.shape[1], NP, q_dtype=q, kv_dtype="e4m3")
        self.ws = torch.zeros(self.plan.workspace_bytes, dtype=torch.uint8, device=DEV)
        B.sps_plan_upload(self.plan, self.ws)
        self.scratch = torch.full((B.paged_attention_scratch(self.plan),), 0xFF, dtype=torch.uint8,
                                  device=DEV)  # FP32 NaN
        # two tokens behind the last one, which nothing may touch
        self.wide = torch.full((T + 2, H + out_pad, D), 7.0, dtype=torch.bfloat16, device=DEV)
        self.out = self.wide[:T, :H]
        self.lse = torch.full((T, H), float("nan"), device=DEV)

    def run(self, stream=None):
        self.B.paged_attention_fwd(self.plan, self.q, self.q_scale, self.kc, self.vc, self.ks,
                                   self.vs, self.pt, self.out, self.lse, self.scratch, self.ws,
                                   stream)

    def reference(self, ctx=None, sel=None):
        """(out, lse, sum of weight * |v|, largest |v| a code and scale of the head can stand for, keys
        of the row) in FP64; sel [T][H][k]: the pages that a row keeps."""
        T, H, G, D = self.T, self.H, self.G, self.D
        out = torch.zeros((T, H, D), dtype=torch.float64, device=DEV)
        mag, lse = torch.zeros_like(out), torch.zeros((T, H), dtype=torch.float64, device=DEV)
        top, keys = torch.zeros_like(lse), torch.zeros_like(lse)
        t0 = 0
        for b, (ql, c) in enumerate(zip(self.q_lens, ctx or self.ctx)):
            if not ql:
                continue
            n = c + ql
            ids = self.pt[b, :(n - 1) // 128 + 1].long()
            for g in range(G):
                k = self.kd[ids, g].reshape(-1, D)[:n]
                v = self.vd[ids, g].reshape(-1, D)[:n]
                h = slice(g * (H // G), (g + 1) * (H // G))
                q = self.qd[t0:t0 + ql, h].reshape(-1, D)
                s = (q @ k.T * D ** -0.5).view(ql, H // G, n)
                pos = c + torch.arange(ql, device=DEV)
                s.masked_fill_(torch.arange(n, device=DEV) > pos[:, None, None], -float("inf"))
                if sel is not None:
                    keep = torch.zeros((ql, H // G, len(ids) + 1), dtype=torch.bool, device=DEV)
                    x = sel[t0:t0 + ql, h].long()
                    keep.scatter_(-1, torch.where(x < 0, len(ids), x), True)
                    s.masked_fill_(~keep[..., torch.arange(n, device=DEV) // 128], -float("inf"))
                z = torch.logsumexp(s, -1, keepdim=True)
                p = torch.exp(s - z)
                out[t0:t0 + ql, h], mag[t0:t0 + ql, h] = p @ v, p @ v.abs()
                lse[t0:t0 + ql, h] = z[..., 0]
                keys[t0:t0 + ql, h] = (pos + 1)[:, None].double()
                # per page the weight of its heaviest key, times the largest value there
                w = torch.nn.functional.pad(p, (0, -n % 128)).view(ql, H // G, -1, 128).amax(-1)
                top[t0:t0 + ql, h] = (w * self.vs[ids, g].double() * 448).amax(-1)
            t0 += ql
        return out, lse, mag, top, keys

    def check(self, ctx=None, noise=2.0 ** -14):
        torch.cuda.synchronize()
        assert self.B.sps_read_device_status(self.plan, self.ws) == 0
        out, lse, mag, top, keys = self.reference(ctx)
        # P is rounded by at most half an FP16 step, the output by half a BF16 step; the FP32 chain in
        # front of P (scores of size 2^7 in log2 units, exp2, sums) stays below 2^-14.  FP16 P (times its
        # page's scale) below 2^-21 of the row's largest is subnormal: 2^-32 of it at most, per key.
        tol = (2.0 ** -11 + noise) * mag + 2.0 ** -8 * out.abs() + (keys * 2.0 ** -32 * top)[..., None]
        err = (self.out.double() - out).abs()
        bad = ~(err <= tol)
        assert not bool(bad.any()), (int(bad.sum()), float(err.max()), bad.nonzero()[:3].tolist())
        # the sum: scores as above, n / 4 additions of 2^-24 in a row
        lerr = (self.lse.double() - lse).abs()
        assert bool((lerr <= 2 * noise + keys * 2.0 ** -26 + lse.abs() * 2.0 ** -22).all()), float(lerr.max())
        assert bool((self.wide[:, self.H:] == 7.0).all()) and bool((self.wide[self.T:] == 7.0).all())


RAGGED = ([1, 0, 130, 7, 300, 1, 128, 1], [0, 5, 1000, 121, 0, 127, 128, 4000])


@pytest.mark.parametrize("q", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,G,D", [(4, 2, 64), (32, 2, 128), (2, 2, 128), (7, 1, 128), (6, 2, 64),
                                   (160, 1, 64), (128, 1, 128), (33, 3, 128)])
def test_ragged_batches(H, G, D, q):
    c = Case(H * 131 + D, *RAGGED, H, G, D, q)
    c.run()
    c.check()


@pytest.mark.parametrize("q", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_lens,ctx", [
    ([1], [0]), ([1], [126]), ([1], [127]), ([1], [128]), ([2], [127]), ([129], [0]), ([17], [111]),
    ([1] * 200, [(37 * i) % 700 for i in range(200)]), ([513], [77]), ([40, 1], [20000, 30000]),
])
def test_lengths_and_page_borders(q_lens, ctx, q):
    c = Case(len(q_lens) + sum(ctx) % 1000, q_lens, ctx, 16, 2, 128, q)
    c.run()
    c.check()


@pytest.mark.parametrize("q", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,G,D,n", [(16, 1, 128, 1), (16, 2, 64, 2), (2, 2, 128, 1), (2, 2, 64, 16),
                                     (5, 1, 128, 3), (28, 4, 64, 2), (34, 2, 128, 1),
                                     (8, 1, 128, 1), (3, 1, 128, 2), (8, 2, 64, 2), (7, 1, 64, 1)])
def test_tiles_of_few_rows(H, G, D, n, q):
    """Decode steps of up to 17 rows a tile, the last page from one key to full, requests without a token
    among them; scores that grow along the context."""
    q_lens = [n, 0, n, 1, n, n, n]
    ctx = [0, 3, 127, 128 * 3 - 1, 5000, 128 * 9 - n, 250]
    for gain in (None, lambda i: 0.3 + 0.7 * i):
        c = Case(H + n, q_lens, ctx, H, G, D, q, k_gain=gain, q_pad=1, out_pad=1)
        c.run()
        # growing scores reach about 2^9 in log2 units: an FP32 rounding of s c of 2^-14 there
        c.check(noise=2.0 ** -14 if gain is None else 2.0 ** -12)


@pytest.mark.parametrize("q", ["bf16", "e4m3"])
def test_single_token_after_a_1m_context(q):
    c = Case(5, [1], [(1 << 20) - 1], 8, 1, 64, q)
    c.run()
    c.check()


@pytest.mark.parametrize("q", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_lens,ctx,H,G", [([1, 1, 3], [3000, 6000, 900], 8, 2), ([400], [2000], 16, 2),
                                            ([40, 30], [3000, 900], 4, 2)])
def test_scores_that_grow_along_the_context(q_lens, ctx, H, G, q):
    """The running maximum grows, jumps and falls: O is rescaled many times, or never after a
    first page that holds the largest scores."""
    for gain in (lambda i: 0.2 + 1.5 * i, lambda i: 40.0 if i % 7 == 3 else 0.5, lambda i: 30.0 / (1 + i)):
        c = Case(17, q_lens, ctx, H, G, 128, q, k_gain=gain)
        c.run()
        # |s| log2 e up to 2^11: an FP32 rounding of s c of 2^-13 there, and two of them
        c.check(noise=2.0 ** -11)


@pytest.mark.parametrize("q", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_lens,ctx,H,G,D", [([1, 3], [3000, 900], 8, 2, 128), ([300, 1], [700, 50], 8, 2, 64),
                                              ([50], [2000], 4, 1, 128), ([1], [2000], 32, 1, 128)])
def test_value_scales_that_differ_from_page_to_page(q_lens, ctx, H, G, D, q):
    """Values of 2^-20 beside values of 2^20, in either order; of falling and of rising size; all tiny."""
    for gain in (lambda i: 2.0 ** (-20 if i % 2 else 20), lambda i: 2.0 ** (-20 if i % 3 else 12),
                 lambda i: 2.0 ** (20 - 2 * i), lambda i: 2.0 ** (2 * i - 20), lambda i: 2.0 ** -30):
        c = Case(19, q_lens, ctx, H, G, D, q, v_gain=lambda i: gain(min(i, 20)))
        c.run()
        c.check()


@pytest.mark.parametrize("q_lens,ctx,H", [([1, 2], [700, 90], 8), ([1], [500], 32), ([200], [300], 4)])
def test_queries_of_any_magnitude(q_lens, ctx, H):
    """BF16 rows far above and below FP16's range (the keys make up for it), and rows whose elements differ
    by 2^20."""
    for e, spread in ((60, 0), (-60, 0), (0, 20), (25, 10)):
        def mag(T, n, g):
            row = torch.exp2(torch.full((T, n, 1), float(e), device=DEV))
            return row * torch.exp2(-spread * torch.rand((T, n, 128), generator=g, device=DEV))

        c = Case(123 + e, q_lens, ctx, H, 2, 128, k_gain=lambda i: 2.0 ** -e, q_mag=mag)
        c.run()
        c.check()


@pytest.mark.parametrize("q", ["bf16", "e4m3"])
def test_keys_and_values_of_scale_zero(q):
    """A page of zeros may have any scale, zero among them: its keys still take part in the sum."""
    for q_lens, ctx, H in (([1], [400], 4), ([140], [300], 8), ([30], [300], 2)):
        c = Case(47, q_lens, ctx, H, 2, 128, q)
        for cache, scale, d in ((c.kc, c.ks, c.kd), (c.vc, c.vs, c.vd)):
            page = int(c.pt[0, 1])
            cache.view(torch.uint8)[page] = 0
            scale[page] = 0.0
            d[page] = 0.0
        c.run()
        c.check()


@pytest.mark.parametrize("q", ["bf16", "e4m3"])
def test_strided_views_without_lse_and_repeated_bits(q):
    c = Case(23, [200, 1, 64], [500, 70, 3], 6, 3, 128, q, q_pad=5, out_pad=2)
    c.run()
    c.check()
    first, lse = c.out.clone(), c.lse.clone()
    for _ in range(3):
        c.scratch.fill_(0xFF)
        c.out.zero_()
        c.run()
        torch.cuda.synchronize()
        assert torch.equal(c.out, first) and torch.equal(c.lse, lse)
    c.out.zero_()
    c.B.paged_attention_fwd(c.plan, c.q, c.q_scale, c.kc, c.vc, c.ks, c.vs, c.pt, c.out, None,
                            c.scratch, c.ws)
    torch.cuda.synchronize()
    assert torch.equal(c.out, first)


@pytest.mark.parametrize("q", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,D", [(6, 128), (40, 64)])
def test_outputs_that_are_16_byte_aligned_only(H, D, q):
    """Rows of the output 16 bytes off every 32-byte border, or every other row of them, between guards."""
    for pad, off in ((16, 8), (8, 0), (8, 8)):
        c = Case(29, [200, 1, 64], [500, 70, 3], H, 2, D, q)
        flat = torch.full((c.T + 1, H * D + pad), 7.0, dtype=torch.bfloat16, device=DEV)
        c.out = flat[:c.T, off:off + H * D].view(c.T, H, D)
        assert c.out.data_ptr() % 32 == 2 * off
        c.run()
        c.check()
        guards = flat.clone()
        guards[:c.T, off:off + H * D] = 7.0
        assert bool((guards == 7.0).all())


@pytest.mark.parametrize("q_lens,ctx,H", [([3, 130], [300, 0], 4), ([1, 1], [300, 0], 4), ([20, 20], [300, 0], 4)])
def test_bad_page_is_reported(q_lens, ctx, H):
    c = Case(29, q_lens, ctx, H, 2, 64)
    c.pt[0, 1] = sum(c.pages)
    c.run()
    torch.cuda.synchronize()
    assert c.B.sps_read_device_status(c.plan, c.ws) == 2  # SPS_DEV_BAD_PAGE


@pytest.mark.parametrize("q", ["bf16", "e4m3"])
def test_captured_decode_replays_over_growing_contexts(q):
    """One capture serves a decode loop: a plan with longer contexts is uploaded to the same
    workspace between replays."""
    ctx = [1000, 4000, 126]
    end = [c + 300 for c in ctx]
    full = Case(31, [1, 1, 1], end, 16, 2, 128, q)  # pages for the longest step
    B = full.B
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        full.run(s)
    for step in (0, 1, 2, 150, 300):
        now = [c + step for c in ctx]
        plan = B.Plan([1, 1, 1], now, 16, 2, 128, 1, full.pt.shape[1], sum(full.pages), q_dtype=q,
                      kv_dtype="e4m3")
        assert plan.workspace_bytes <= full.ws.numel()
        with torch.cuda.stream(s):
            B.sps_plan_upload(plan, full.ws, s)
            full.out.zero_()
            g.replay()
        torch.cuda.synchronize()
        full.check(now)


@pytest.mark.parametrize("q", ["bf16", "e4m3"])
def test_capture_of_whole_tiles_replays_over_cut_ones(q):
    """Captured while no tile is cut over blocks, replayed over contexts whose tiles are, and back."""
    for q_lens, end in (([1] * 6, [9000, 70, 300, 20000, 5, 1]), ([150, 150], [6000, 90])):
        full = Case(47, q_lens, end, 8, 2, 128, q)
        B = full.B
        short = [min(c, 20) for c in end]
        plans = [B.Plan(q_lens, c, 8, 2, 128, 1, full.pt.shape[1], sum(full.pages), q_dtype=q,
                        kv_dtype="e4m3") for c in (short, end)]
        assert all(p.workspace_bytes <= full.ws.numel() for p in plans)
        B.sps_plan_upload(plans[0], full.ws)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        full.plan = plans[0]
        with torch.cuda.graph(g, stream=s):
            full.run(s)
        for plan, now in ((plans[0], short), (plans[1], end), (plans[0], short)):
            with torch.cuda.stream(s):
                B.sps_plan_upload(plan, full.ws, s)
                full.out.zero_()
                full.scratch.fill_(0xFF)
                g.replay()
            torch.cuda.synchronize()
            full.check(now)


@pytest.mark.parametrize("q", ["bf16", "e4m3"])
@pytest.mark.parametrize("seed", range(8))
def test_mixed_batches(seed, q):
    """Single tokens, chunks and empty requests after contexts of every size: tiles kept whole, cut
    in two and cut over many blocks in one call."""
    rng = np.random.default_rng(100 + seed)
    n = int(rng.choice([3, 9, 40]))
    q_lens = [int(rng.choice([0, 1, 1, 1, 2, int(rng.integers(3, 40)), int(rng.integers(40, 600))]))
              for _ in range(n)]
    q_lens[0] = 1
    ctx = [int(rng.choice([0, int(rng.integers(1, 300)), int(rng.integers(300, 2500))])) for _ in q_lens]
    if seed % 2:
        ctx[int(rng.integers(n))] = 30000  # one long context beside the others
    G = int(rng.choice([1, 2]))
    c = Case(seed, q_lens, ctx, G * int(rng.choice([1, 3, 4, 8, 16])), G, int(rng.choice([64, 128])),
             q, out_pad=1)
    c.run()
    c.check()


def test_two_streams_with_their_own_buffers():
    a, b = Case(37, [300], [1000], 8, 2, 128), Case(41, [1, 1], [9000, 50], 8, 2, 128, "e4m3")
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for st in (sa, sb):
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        a.run(sa)
        b.run(sb)
    a.check()
    b.check()


# ------------------------------------------------------------------ the sparse forward

def _selection(c, k, seed):
    """Pages of every row as topk_select leaves them: the own one and others, ascending, -1 behind."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    pos = torch.cat([torch.arange(a, a + n, device=DEV) for a, n in zip(c.ctx, c.q_lens)])
    own = (pos // 128)[:, None, None]
    n = c.pt.shape[1]
    page = torch.arange(n, device=DEV)
    score = torch.rand((c.T, c.H, n), generator=g, device=DEV)
    score = torch.where(page == own, 2.0, score).masked_fill_(page > own, -1.0)
    val, at = score.topk(min(k, n), -1)
    at = torch.where(val < 0, n, at).sort(-1).values
    sel = torch.full((c.T, c.H, k), -1, dtype=torch.int32, device=DEV)
    sel[..., :at.shape[-1]] = torch.where(at == n, -1, at).int()
    return sel


@pytest.mark.parametrize("q", ["bf16", "e4m3"])
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16", "noalloc"])
@pytest.mark.parametrize("q_lens,ctx,H,G,D,k", [([200, 1, 70], [900, 0, 128], 8, 2, 128, 4),
                                                ([130, 3], [0, 2500], 4, 1, 64, 16),
                                                ([1, 1, 1], [5000, 127, 300], 32, 2, 128, 20)])
def test_sparse_forward(q_lens, ctx, H, G, D, k, kind, q):
    # (the sparse path wants finite codes behind the last token)
    c = Case(H + k, q_lens, ctx, H, G, D, q, top_k=k, nan_tail=False)
    B, R = c.B, c.T * H
    sel = _selection(c, k, 3)
    dt = {"f16": torch.float16, "bf16": torch.bfloat16}.get(kind, torch.float32)
    partial = torch.full((k, R, D), float("nan"), dtype=dt, device=DEV)
    lse = torch.full((k, R), float("nan"), device=DEV)
    out_lse = torch.empty((R,), device=DEV)
    args = (c.plan, c.q.contiguous(), c.q_scale, c.kc, c.vc, c.ks, c.vs, c.pt, sel, partial, lse)
    if kind == "noalloc":
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        B.sparse_prefill_fwd_noalloc(*args, status)
        torch.cuda.synchronize()
        assert int(status) == 0
    else:
        {"f32": B.sparse_prefill_fwd, "f16": B.sparse_prefill_fwd_f16,
         "bf16": B.sparse_prefill_fwd_bf16}[kind](*args, c.ws)
    combine = {"f16": B.partial_combine_f16, "bf16": B.partial_combine_bf16}.get(kind, B.partial_combine)
    combine(partial, lse, c.out.view(R, D), out_lse)
    torch.cuda.synchronize()
    assert B.sps_read_device_status(c.plan, c.ws) == 0
    out, rlse, mag, top, keys = c.reference(sel=sel)
    # P to FP16, the partials to their type, the output to BF16; the FP32 chains below 2^-13
    half = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}.get(kind, 0.0)
    tol = (2.0 ** -11 + half + 2.0 ** -13) * mag + 2.0 ** -8 * out.abs() + (keys * 2.0 ** -24 * top)[..., None]
    err = (c.out.double() - out).abs()
    assert bool((err <= tol).all()), float((err - tol).max())
    assert bool(((out_lse.view(c.T, H).double() - rlse).abs() <= 2.0 ** -12 + rlse.abs() * 2.0 ** -22).all())


def test_sparse_forward_of_all_pages_is_full_attention():
    c = Case(43, [200, 70], [900, 128], 8, 2, 128, top_k=16, nan_tail=False)
    B, R = c.B, c.T * 8
    partial, lse = torch.empty((16, R, 128), device=DEV), torch.empty((16, R), device=DEV)
    out = torch.empty((R, 128), dtype=torch.bfloat16, device=DEV)
    B.sparse_prefill_fwd(c.plan, c.q, 1.0, c.kc, c.vc, c.ks, c.vs, c.pt, _selection(c, 16, 1), partial,
                         lse, c.ws)
    B.partial_combine(partial, lse, out)
    c.run()
    c.check()
    ref, _, mag, _, _ = c.reference()
    # both within an FP16 P and the output's rounding of the definition
    tol = (2.0 ** -10 + 2.0 ** -12) * mag + 2.0 ** -7 * ref.abs()
    assert bool(((out.view(c.T, 8, 128).double() - c.out.double()).abs() <= tol).all())


def test_sparse_step_with_index_keys_of_its_own():
    """Indexer over BF16 index keys, selection, forward over the E4M3 cache and combine."""
    from paged_top_sparse_gb300 import binding as B

    H, G, D, k = 8, 2, 128, 4
    c = Case(61, [200, 1, 70], [1300, 700, 128], H, G, D, top_k=k, nan_tail=False)
    R = c.T * H
    index_keys = torch.where(torch.isfinite(c.kd), c.kd, 0.0).bfloat16()
    n = c.pt.shape[1]
    scores = torch.full((R, (n + 3) // 4 * 4), float("nan"), device=DEV)
    idx = torch.empty((R, k), dtype=torch.int32, device=DEV)
    partial, lse = torch.empty((k, R, D), device=DEV), torch.empty((k, R), device=DEV)
    out_lse = torch.empty((R,), device=DEV)
    B.indexer_scores(c.plan, c.q, 1.0, index_keys, None, 1.0, c.pt, scores, c.ws)
    B.topk_select(c.plan, scores, idx, c.ws)
    B.sparse_prefill_fwd(c.plan, c.q, 1.0, c.kc, c.vc, c.ks, c.vs, c.pt, idx, partial, lse, c.ws)
    B.partial_combine(partial, lse, c.out.view(R, D), out_lse)
    torch.cuda.synchronize()
    assert B.sps_read_device_status(c.plan, c.ws) == 0
    sel = idx.view(c.T, H, k)
    pos = torch.cat([torch.arange(a, a + m, device=DEV) for a, m in zip(c.ctx, c.q_lens)])
    assert bool(((sel == (pos // 128)[:, None, None]).sum(-1) == 1).all())  # the own page is there
    out, rlse, mag, top, keys = c.reference(sel=sel)
    tol = (2.0 ** -11 + 2.0 ** -13) * mag + 2.0 ** -8 * out.abs() + (keys * 2.0 ** -24 * top)[..., None]
    assert bool(((c.out.double() - out).abs() <= tol).all())
    assert bool(((out_lse.view(c.T, H).double() - rlse).abs() <= 2.0 ** -12 + rlse.abs() * 2.0 ** -22).all())


@pytest.mark.parametrize("q", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,G,D,q_lens,ctx", [(16, 1, 128, [300, 9, 140] * 60, [0, 500, 90] * 60),
                                              (8, 2, 64, [70] * 150, [33 * i for i in range(150)]),
                                              (32, 2, 128, [3] * 200, [0, 120, 127, 1000] * 50)])
def test_blocks_of_many_pieces(H, G, D, q_lens, ctx, q):
    """More work tiles than blocks: a block goes through pieces of one and two row tiles, of one and many
    pages, in turn, and does so alike each time."""
    c = Case(len(q_lens), q_lens, ctx, H, G, D, q)
    c.run()
    c.check()
    first = c.out.clone()
    for _ in range(20):
        c.run()
    torch.cuda.synchronize()
    assert torch.equal(c.out, first)


def test_fp8qk_wants_an_nvfp4_cache():
    from paged_top_sparse_gb300 import binding as B

    c = Case(3, [4], [10], 4, 2, 128, "e4m3", top_k=2)
    sel = _selection(c, 2, 1)
    partial, lse = torch.empty((2, 16, 128), device=DEV), torch.empty((2, 16), device=DEV)
    with pytest.raises(B.SpsError) as e:
        B.sparse_prefill_fwd_fp8qk(c.plan, c.q, 1.0, c.kc, c.vc, c.ks, c.vs, c.pt, sel, partial, lse, c.ws)
    assert e.value.status == 2
