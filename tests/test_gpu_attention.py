"""GPU checks of paged_attention_fwd through the C ABI against the definition in 64 bits: head
layouts, ragged batches of chunks and single tokens, page borders, long contexts, NaN in unwritten
slots, growing scores, strided views, graph replay, and a whole step with the operators around it."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from paged_top_sparse_gb300 import synth

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_top_sparse_gb300 import build

    build.build()


class Case:
    """A batch with its caches, filled; every slot behind a request's last token holds `junk`."""

    def __init__(self, seed, q_lens, ctx, H, G, D, kv="bf16", junk="nan", k_gain=None, q_pad=0,
                 out_pad=0, top_k=1, max_pages=None):
        from paged_top_sparse_gb300 import binding as B

        self.B = B
        self.q_lens, self.ctx, self.H, self.G, self.D, self.kv = q_lens, ctx, H, G, D, kv
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        randn = lambda *s: torch.randn(s, generator=g, device=DEV)
        self.pages = pages = [(c + q - 1) // 128 + 1 if q else 0 for q, c in zip(q_lens, ctx)]
        NP, T = sum(pages), sum(q_lens)
        self.T = T
        rng = np.random.default_rng(seed)
        perm = rng.permutation(NP).astype(np.int32)
        pt = np.full((len(q_lens), max_pages or max(pages)), -1, np.int32)  # unused: out of range
        at = 0
        for b, n in enumerate(pages):
            pt[b, :n] = perm[at:at + n]
            at += n
        self.pt = torch.from_numpy(pt).to(DEV)
        k, v = randn(NP, G, 128, D), randn(NP, G, 128, D)
        if k_gain is not None:  # keys whose scores change with the position
            for b, n in enumerate(pages):
                for i in range(n):
                    k[pt[b, i]] *= k_gain(i)
        tail = torch.zeros((NP, 128), dtype=torch.bool, device=DEV)
        for b, n in enumerate(pages):
            if n:
                tail[pt[b, n - 1], (ctx[b] + q_lens[b] - 1) % 128 + 1:] = True
        self.ks = self.vs = None
        if kv == "bf16":
            self.q_scale = 1.0
            self.kc, self.vc = k.bfloat16(), v.bfloat16()
            self.kd, self.vd = self.kc.double(), self.vc.double()
            fill = float("nan") if junk == "nan" else float("inf")
            for c in (self.kc, self.vc):
                c.transpose(1, 2)[tail] = fill
            qv = randn(T, H + q_pad, D).bfloat16()
            self.q = qv[:, :H]
            self.qd = self.q.double()
        else:
            self.q_scale = 0.0117
            (self.kc, self.ks, self.kd), (self.vc, self.vs, self.vd) = (self._nvfp4(x) for x in (k, v))
            for s_ in (self.ks, self.vs):
                s_.transpose(1, 2)[tail] = 0x7F  # a NaN scale
            qv = (randn(T, H + q_pad, D) / self.q_scale).clamp(-448, 448).to(torch.float8_e4m3fn)
            self.q = qv[:, :H]
            self.qd = self.q.double() * self.q_scale
        self.plan = B.Plan(q_lens, ctx, H, G, D, top_k, pt.shape[1], NP,
                           q_dtype="bf16" if kv == "bf16" else "e4m3", kv_dtype=kv)
        self.ws = torch.zeros(self.plan.workspace_bytes, dtype=torch.uint8, device=DEV)
        B.sps_plan_upload(self.plan, self.ws)
        self.scratch = torch.full((B.paged_attention_scratch(self.plan),), 0xFF, dtype=torch.uint8,
                                  device=DEV)  # FP32 NaN
        # two tokens behind the last one, which nothing may touch
        self.wide = torch.full((T + 2, H + out_pad, D), 7.0, dtype=torch.bfloat16, device=DEV)
        self.out = self.wide[:T, :H]
        self.lse = torch.full((T, H), float("nan"), device=DEV)

    @staticmethod
    def _nvfp4(x):
        codes, scales = synth.quantize_nvfp4(x.cpu().numpy())
        mag = synth._E2M1_MAGS
        c = np.stack((codes & 15, codes >> 4), -1).reshape(x.shape)
        val = np.where(c & 8, -1.0, 1.0) * mag[c & 7]
        s = torch.from_numpy(scales).view(torch.float8_e4m3fn).double().numpy()
        d = (val.reshape(*s.shape, 16) * s[..., None]).reshape(x.shape)
        return torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), torch.from_numpy(d).to(DEV)

    def run(self, stream=None):
        self.B.paged_attention_fwd(self.plan, self.q, self.q_scale, self.kc, self.vc, self.ks,
                                   self.vs, self.pt, self.out, self.lse, self.scratch, self.ws,
                                   stream)

    def reference(self, ctx=None):
        """(out, lse, sum of weight * |v|, keys of the row) in FP64."""
        T, H, G, D = self.T, self.H, self.G, self.D
        out = torch.zeros((T, H, D), dtype=torch.float64, device=DEV)
        mag, lse = torch.zeros_like(out), torch.zeros((T, H), dtype=torch.float64, device=DEV)
        keys = torch.zeros((T, H), dtype=torch.float64, device=DEV)
        t0 = 0
        for b, (ql, c) in enumerate(zip(self.q_lens, ctx or self.ctx)):
            if not ql:
                continue
            ids = self.pt[b, :self.pages[b]].long()
            n = c + ql
            for g in range(G):
                k = self.kd[ids, g].reshape(-1, D)[:n]
                v = self.vd[ids, g].reshape(-1, D)[:n]
                h = slice(g * (H // G), (g + 1) * (H // G))
                q = self.qd[t0:t0 + ql, h].reshape(-1, D)
                s = (q @ k.T * D ** -0.5).view(ql, H // G, n)
                pos = c + torch.arange(ql, device=DEV)
                s.masked_fill_(torch.arange(n, device=DEV) > pos[:, None, None], -float("inf"))
                z = torch.logsumexp(s, -1, keepdim=True)
                p = torch.exp(s - z)
                out[t0:t0 + ql, h], mag[t0:t0 + ql, h] = p @ v, p @ v.abs()
                lse[t0:t0 + ql, h] = z[..., 0]
                keys[t0:t0 + ql, h] = (pos + 1)[:, None].double()
            t0 += ql
        return out, lse, mag, keys

    def check(self, ctx=None):
        torch.cuda.synchronize()
        assert self.B.sps_read_device_status(self.plan, self.ws) == 0
        out, lse, mag, keys = self.reference(ctx)
        # P is rounded by at most half a step of its type, the output by half a BF16 step; the FP32
        # chain in front of P (scores of size 2^7 in log2 units, exp2, sums) stays below 2^-14.
        # FP16 P below 2^-21 of the reference is subnormal: 2^-32 of it at most, per key.
        p_half = 2.0 ** -8 if self.kv == "bf16" else 2.0 ** -11
        tol = (p_half + 2.0 ** -14) * mag + 2.0 ** -8 * out.abs()
        if self.kv != "bf16":
            tol = tol + keys[..., None] * 2.0 ** -32 * 16
        err = (self.out.double() - out).abs()
        bad = ~(err <= tol)
        assert not bool(bad.any()), (int(bad.sum()), float(err.max()), bad.nonzero()[:3].tolist())
        # the sum: scores as above, n / 4 additions of 2^-24 in a row
        lerr = (self.lse.double() - lse).abs()
        assert bool((lerr <= 2.0 ** -13 + keys * 2.0 ** -26 + lse.abs() * 2.0 ** -22).all()), float(lerr.max())
        assert bool((self.wide[:, self.H:] == 7.0).all()) and bool((self.wide[self.T:] == 7.0).all())


RAGGED = ([1, 0, 130, 7, 300, 1, 128, 1], [0, 5, 1000, 121, 0, 127, 128, 4000])


@pytest.mark.parametrize("kv", ["bf16", "nvfp4"])
@pytest.mark.parametrize("H,G,D", [(4, 2, 64), (32, 2, 128), (2, 2, 128), (7, 1, 128), (6, 2, 64),
                                   (160, 1, 64), (128, 1, 128), (33, 3, 128)])
def test_ragged_batches(H, G, D, kv):
    c = Case(H * 131 + D, *RAGGED, H, G, D, kv)
    c.run()
    c.check()


@pytest.mark.parametrize("kv", ["bf16", "nvfp4"])
@pytest.mark.parametrize("q_lens,ctx", [
    ([1], [0]), ([1], [126]), ([1], [127]), ([1], [128]), ([2], [127]), ([129], [0]), ([17], [111]),
    ([1] * 200, [(37 * i) % 700 for i in range(200)]), ([513], [77]), ([40, 1], [20000, 30000]),
])
def test_lengths_and_page_borders(q_lens, ctx, kv):
    c = Case(len(q_lens) + sum(ctx) % 1000, q_lens, ctx, 16, 2, 128, kv, junk="inf")
    c.run()
    c.check()


@pytest.mark.parametrize("kv", ["bf16", "nvfp4"])
@pytest.mark.parametrize("H,G,D,q", [(16, 1, 128, 1), (16, 2, 64, 2), (2, 2, 128, 1), (2, 2, 64, 16),
                                     (5, 1, 128, 3), (28, 4, 64, 2), (34, 2, 128, 1),
                                     (8, 1, 128, 1), (3, 1, 128, 2), (8, 2, 64, 2), (7, 1, 64, 1)])
def test_tiles_of_few_rows(H, G, D, q, kv):
    """Decode steps of up to 16 rows a tile (one case of 17), the last page from one key to full,
    requests without a token among them."""
    q_lens = [q, 0, q, 1, q, q, q]
    ctx = [0, 3, 127, 128 * 3 - 1, 5000, 128 * 9 - q, 250]
    for gain in (None, lambda i: 0.3 + 0.7 * i):
        c = Case(H + q, q_lens, ctx, H, G, D, kv, k_gain=gain, q_pad=1, out_pad=1)
        c.run()
        if gain is None:
            c.check()
            continue
        torch.cuda.synchronize()
        assert c.B.sps_read_device_status(c.plan, c.ws) == 0
        # scores grow to about 2^9 in log2 units: an FP32 rounding of s c of 2^-14 there
        out, lse, mag, keys = c.reference()
        p_half = 2.0 ** -8 if kv == "bf16" else 2.0 ** -11
        tol = (p_half + 2.0 ** -12) * mag * 2 + 2.0 ** -8 * out.abs() + 2.0 ** -20
        assert bool(((c.out.double() - out).abs() <= tol).all())
        assert bool(((c.lse.double() - lse).abs() <= 2.0 ** -12 + lse.abs() * 2.0 ** -21).all())


@pytest.mark.parametrize("kv", ["bf16", "nvfp4"])
def test_single_token_after_a_1m_context(kv):
    c = Case(5, [1], [(1 << 20) - 1], 8, 1, 64, kv)
    c.run()
    c.check()


@pytest.mark.parametrize("kv", ["bf16", "nvfp4"])
@pytest.mark.parametrize("q_lens,ctx,H,G", [([1, 1, 3], [3000, 6000, 900], 8, 2), ([400], [2000], 16, 2)])
def test_scores_that_grow_along_the_context(q_lens, ctx, H, G, kv):
    """The running maximum grows, jumps and falls: O is rescaled many times, or never after a
    first page that holds the largest scores."""
    for gain in (lambda i: 0.2 + 1.5 * i, lambda i: 40.0 if i % 7 == 3 else 0.5,
                 lambda i: 30.0 / (1 + i)):
        c = Case(17, q_lens, ctx, H, G, 128, kv, k_gain=gain)
        # large scores: the FP32 rounding of s * c grows with them, so the bound is on a score
        # scale that keeps |s c| below 2^10
        c.run()
        torch.cuda.synchronize()
        out, lse, mag, keys = c.reference()
        smax = 2.0 ** 11  # |s| log2 e at most (gain 40, |q||k| of 5 sigma)
        noise = smax * 2.0 ** -22
        p_half = 2.0 ** -8 if kv == "bf16" else 2.0 ** -11
        tol = (p_half + noise) * mag * 2 + 2.0 ** -8 * out.abs() + 2.0 ** -20
        assert bool(((c.out.double() - out).abs() <= tol).all())
        assert bool(((c.lse.double() - lse).abs() <= 2 * noise + lse.abs() * 2.0 ** -22).all())


@pytest.mark.parametrize("kv", ["bf16", "nvfp4"])
def test_strided_views_without_lse_and_repeated_bits(kv):
    c = Case(23, [200, 1, 64], [500, 70, 3], 6, 3, 128, kv, q_pad=5, out_pad=2)
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


def test_bad_page_is_reported():
    c = Case(29, [3, 130], [300, 0], 4, 2, 64)
    c.pt[1, 1] = sum(c.pages)
    c.run()
    torch.cuda.synchronize()
    assert c.B.sps_read_device_status(c.plan, c.ws) == 2  # SPS_DEV_BAD_PAGE


@pytest.mark.parametrize("kv", ["bf16", "nvfp4"])
def test_captured_decode_replays_over_growing_contexts(kv):
    """One capture serves a decode loop: a plan with longer contexts is uploaded to the same
    workspace between replays."""
    ctx = [1000, 4000, 126]
    end = [c + 300 for c in ctx]
    full = Case(31, [1, 1, 1], end, 16, 2, 128, kv)  # pages for the longest step
    B = full.B
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        full.run(s)
    for step in (0, 1, 2, 150, 300):
        now = [c + step for c in ctx]
        plan = B.Plan([1, 1, 1], now, 16, 2, 128, 1, full.pt.shape[1], sum(full.pages),
                      q_dtype="bf16" if kv == "bf16" else "e4m3", kv_dtype=kv)
        assert plan.workspace_bytes <= full.ws.numel()
        with torch.cuda.stream(s):
            B.sps_plan_upload(plan, full.ws, s)
            full.out.zero_()
            g.replay()
        torch.cuda.synchronize()
        full.check(now)


@pytest.mark.parametrize("kv", ["bf16", "nvfp4"])
def test_capture_of_whole_tiles_replays_over_cut_ones(kv):
    """Captured while no tile is cut over blocks (an eager call needs no merge then), replayed over
    contexts whose tiles are, and back."""
    H, G = 8, 2
    for q_lens, end in (([1] * 6, [9000, 70, 300, 20000, 5, 1]), ([150, 150], [6000, 90])):
        full = Case(47, q_lens, end, H, G, 128, kv)
        B = full.B
        short = [min(c, 20) for c in end]
        plans = [B.Plan(q_lens, c, H, G, 128, 1, full.pt.shape[1], sum(full.pages),
                        q_dtype="bf16" if kv == "bf16" else "e4m3", kv_dtype=kv)
                 for c in (short, end)]
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


@pytest.mark.parametrize("kv", ["bf16", "nvfp4"])
@pytest.mark.parametrize("seed", range(8))
def test_mixed_batches(seed, kv):
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
             kv, out_pad=1)
    c.run()
    c.check()


def test_two_streams_with_their_own_buffers():
    a, b = Case(37, [300], [1000], 8, 2, 128), Case(41, [1, 1], [9000, 50], 8, 2, 128)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for st in (sa, sb):
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        a.run(sa)
        b.run(sb)
    a.check()
    b.check()


def test_equals_the_sparse_path_when_every_page_is_selected():
    """top_k pages at least as many as a row sees: the four sparse steps compute the same rows."""
    c = Case(43, [200, 70], [900, 128], 8, 2, 128, top_k=16, junk="inf")
    for x in (c.kc, c.vc):  # the sparse path wants finite values behind the last token
        x[~torch.isfinite(x)] = 0.0
    B, R = c.B, c.T * 8
    scores = torch.empty((R, 16), device=DEV)
    idx = torch.empty((R, 16), dtype=torch.int32, device=DEV)
    partial = torch.empty((16, R, 128), device=DEV)
    lse = torch.empty((16, R), device=DEV)
    out = torch.empty((R, 128), dtype=torch.bfloat16, device=DEV)
    out_lse = torch.empty((R,), device=DEV)
    B.indexer_scores(c.plan, c.q, 1.0, c.kc, None, 1.0, c.pt, scores, c.ws)
    B.topk_select(c.plan, scores, idx, c.ws)
    B.sparse_prefill_fwd(c.plan, c.q, 1.0, c.kc, c.vc, None, None, c.pt, idx, partial, lse, c.ws)
    B.partial_combine(partial, lse, out, out_lse)
    c.run()
    c.check()
    ref, rlse, mag, _ = c.reference()
    # both sides within their own roundings of the definition: BF16 P here, FP16 P there
    tol = (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -13) * mag + 2.0 ** -7 * ref.abs()
    assert bool(((out.view(c.T, 8, 128).double() - c.out.double()).abs() <= tol).all())
    assert bool(((out_lse.view(c.T, 8) - c.lse).abs() <= 2.0 ** -12).all())


@pytest.mark.parametrize("kv", ["bf16", "nvfp4"])
def test_step_of_norm_rotation_append_and_attention(kv):
    """A prompt in two chunks, then three single tokens, through sps_qk_norm_rope,
    sps_kv_append_rope and paged_attention_fwd, against attention over the whole sequence."""
    from paged_top_sparse_gb300 import binding as B

    H, G, D, N = 8, 2, 128, 333
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    qkv = torch.randn((N, H + 2 * G, D), generator=g, device=DEV).bfloat16()
    qw, kw = (1 + 0.2 * torch.randn(D, generator=g, device=DEV) for _ in range(2))
    f = (1e4 ** (-torch.arange(D // 2, device=DEV, dtype=torch.float64) * 2 / D)).float()
    rope = B.Rope(f)
    pages = 3
    pt = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=DEV)
    if kv == "bf16":
        kc, vc = (torch.full((pages, G, 128, D), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in "kv")
        ks = vs = None
        q_scale = 1.0
    else:
        kc, vc = (torch.full((pages, G, 128, D // 2), 0xFF, dtype=torch.uint8, device=DEV) for _ in "kv")
        ks, vs = (torch.full((pages, G, 128, D // 16), 0x7F, dtype=torch.uint8, device=DEV) for _ in "kv")
        q_scale = 0.02
    got = torch.empty((N, H, D), dtype=torch.bfloat16, device=DEV)
    queries = torch.empty((N, H, D), dtype=torch.float64, device=DEV)
    at = 0
    for n in (200, 130, 1, 1, 1):
        plan = B.Plan([n], [at], H, G, D, 1, pages, pages, q_dtype="bf16" if kv == "bf16" else "e4m3",
                      kv_dtype=kv)
        ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device=DEV)
        B.sps_plan_upload(plan, ws)
        x = qkv[at:at + n]
        q = torch.empty((n, H, D), dtype=torch.bfloat16 if kv == "bf16" else torch.uint8, device=DEV)
        B.sps_qk_norm_rope(plan, x[:, :H], None, qw, None, 1e-6, rope, q, q_scale, None, ws)
        B.sps_kv_append_rope(plan, x[:, H:H + G], x[:, H + G:], kw, 1e-6, rope, pt, kc, vc, ks, vs, ws)
        scratch = torch.empty(B.paged_attention_scratch(plan), dtype=torch.uint8, device=DEV)
        B.paged_attention_fwd(plan, q, q_scale, kc, vc, ks, vs, pt, got[at:at + n], None, scratch, ws)
        torch.cuda.synchronize()
        assert B.sps_read_device_status(plan, ws) == 0
        queries[at:at + n] = q.double() if kv == "bf16" else q.view(torch.float8_e4m3fn).double() * q_scale
        at += n
    # attention in FP64 over what the cache and the queries hold
    if kv == "bf16":
        k, v = kc.double(), vc.double()
    else:
        val = []
        for c_, s_ in ((kc, ks), (vc, vs)):
            o = torch.empty((pages, G, 128, D), dtype=torch.float16, device=DEV)
            B.sps_dequantize("nvfp4", c_, s_, o.numel(), o)
            val.append(o.double())
        k, v = val
    k, v = (x[pt[0].long()].transpose(0, 1).reshape(G, -1, D)[:, :N] for x in (k, v))
    s = torch.einsum("tghd,gkd->ghtk", queries.view(N, G, H // G, D), k) * D ** -0.5
    s = s.masked_fill(torch.ones(N, N, device=DEV).triu(1).bool(), -float("inf"))
    p = torch.softmax(s, -1)
    ref = torch.einsum("ghtk,gkd->tghd", p, v).reshape(N, H, D)
    mag = torch.einsum("ghtk,gkd->tghd", p, v.abs()).reshape(N, H, D)
    tol = (2.0 ** -8 + 2.0 ** -14) * mag + 2.0 ** -8 * ref.abs()
    assert bool(((got.double() - ref).abs() <= tol).all())
    # and the cached keys are the normalised, rotated ones (checked in full in test_gpu_rope.py)
    xk = qkv[:, H:H + G].double()
    n_ = xk / torch.sqrt((xk * xk).mean(-1, keepdim=True) + 1e-6) * kw.double()
    a = torch.arange(N, device=DEV, dtype=torch.float64)[:, None] * f.double()
    c_, s_ = a.cos()[:, None], a.sin()[:, None]
    y = torch.cat((n_[..., :64] * c_ - n_[..., 64:] * s_, n_[..., 64:] * c_ + n_[..., :64] * s_), -1)
    rel = float((k - y.transpose(0, 1)).norm() / y.norm())
    assert rel <= (2.0 ** -8 if kv == "bf16" else 0.25)


@pytest.mark.parametrize("kv", ["bf16", "nvfp4"])
@pytest.mark.parametrize("H,G,D", [(16, 1, 128), (8, 2, 64)])
def test_captured_decode_step_equals_the_eager_calls(H, G, D, kv):
    """One graph of norm and rotation, append and attention, replayed while the contexts grow over
    page borders: the same bits as eager calls on a cache of their own."""
    from paged_top_sparse_gb300 import binding as B

    ctx, steps, pages = [126, 500, 0], 4, 5
    n = len(ctx)
    g = torch.Generator(device=DEV)
    g.manual_seed(H + D)
    pt = torch.arange(n * pages, dtype=torch.int32, device=DEV).flip(0).reshape(n, pages)
    rope = B.Rope((1e4 ** (-torch.arange(D // 2, device=DEV, dtype=torch.float64) * 2 / D)).float())
    w = 1 + 0.1 * torch.randn(D, generator=g, device=DEV)
    quant = kv == "nvfp4"

    class Side:
        def __init__(self):
            shape = (n * pages, G, 128, D // 2 if quant else D)
            dt = torch.uint8 if quant else torch.bfloat16
            self.kc, self.vc = (torch.zeros(shape, dtype=dt, device=DEV) for _ in "kv")
            self.ks = self.vs = None
            if quant:
                self.ks, self.vs = (torch.zeros((n * pages, G, 128, D // 16), dtype=torch.uint8, device=DEV)
                                    for _ in "kv")
            self.x = torch.zeros((n, H + 2 * G, D), dtype=torch.bfloat16, device=DEV)
            self.q = torch.zeros((n, H, D), dtype=torch.uint8 if quant else torch.bfloat16, device=DEV)
            self.out = torch.zeros((n, H, D), dtype=torch.bfloat16, device=DEV)
            self.ws = torch.zeros(max(p.workspace_bytes for p in plans), dtype=torch.uint8, device=DEV)
            self.scratch = torch.zeros(B.paged_attention_scratch(plans[0]), dtype=torch.uint8, device=DEV)

        def step(self, plan, stream=None):
            x, s = self.x, 0.02 if quant else 1.0
            B.sps_qk_norm_rope(plan, x[:, :H], None, w, None, 1e-6, rope, self.q, s, None, self.ws, stream)
            B.sps_kv_append_rope(plan, x[:, H:H + G], x[:, H + G:], w, 1e-6, rope, pt, self.kc, self.vc,
                                 self.ks, self.vs, self.ws, stream)
            B.paged_attention_fwd(plan, self.q, s, self.kc, self.vc, self.ks, self.vs, pt, self.out, None,
                                  self.scratch, self.ws, stream)

    plans = [B.Plan([1] * n, [c + i for c in ctx], H, G, D, 1, pages, n * pages,
                    q_dtype="e4m3" if quant else "bf16", kv_dtype=kv) for i in range(steps)]
    a, b = Side(), Side()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    B.sps_plan_upload(plans[0], a.ws, s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        a.step(plans[0], s)
    for i, plan in enumerate(plans):
        x = torch.randn((n, H + 2 * G, D), generator=g, device=DEV).bfloat16()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            a.x.copy_(x)
            B.sps_plan_upload(plan, a.ws, s)
            graph.replay()
        b.x.copy_(x)
        B.sps_plan_upload(plan, b.ws)
        b.step(plan)
        torch.cuda.synchronize()
        assert B.sps_read_device_status(plan, a.ws) == 0
        assert torch.equal(a.q, b.q) and torch.equal(a.kc, b.kc) and torch.equal(a.vc, b.vc)
        assert torch.equal(a.out, b.out) and bool(torch.isfinite(a.out.float()).all())
        assert not bool((a.out == 0).all())
