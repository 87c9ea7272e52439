"""GPU checks of the append into an E4M3 cache with a scale for each page and KV head: sps_kv_append
byte by byte against the rule, sps_kv_append_rope against the rule on rows rotated in 64 bits, pages that
hold earlier tokens, graph replay, and a decode loop with the page tables, the rotation and the
attention around it."""
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


def to_e4m3(x):
    """Codes of FP64 x: nearest even, saturating; NaN stays one."""
    return x.clamp(-448, 448).float().to(F8)


def pow2_scale(a):
    """The smallest power of two s with a / s <= 448, within 2^-40 .. 2^40, by trying every one."""
    s = torch.exp2(torch.arange(-40, 41, dtype=torch.float64, device=DEV))
    fits = a[..., None] / s <= 448
    first = torch.where(fits.any(-1), fits.int().argmax(-1), 80)
    return s[first]


def append_rule(rows, t0s, ctx, pt, codes, scales):
    """The rule in 64 bits, on copies: rows [T][G][D] FP64."""
    codes, scales = codes.clone(), scales.clone()
    t = 0
    for b, (n, c) in enumerate(zip(t0s, ctx)):
        i = 0
        while i < n:
            pos = c + i
            m = min(n - i, 128 - pos % 128)
            phys, s0 = int(pt[b, pos // 128]), pos % 128
            x = rows[t + i:t + i + m].transpose(0, 1)  # [G][m][D]
            a = torch.where(torch.isnan(x), torch.zeros_like(x), x).abs().amax((1, 2))
            s = pow2_scale(a)
            if s0:
                old = scales[phys].double()
                s = torch.maximum(s, old)
                f = (scales[phys] / s.float())[:, None, None]  # FP32, as the rule says
                kept = codes[phys, :, :s0].float() * f
                grown = (s > old)[:, None, None]
                codes[phys, :, :s0] = torch.where(grown, to_e4m3(kept.double()).float(),
                                                  codes[phys, :, :s0].float()).to(F8)
            scales[phys] = s.float()
            q = (x.float() / s.float()[:, None, None]).double()
            codes[phys, :, s0:s0 + m] = to_e4m3(q)
            i += m
        t += n
    return codes, scales


class Batch:
    def __init__(self, q_lens, ctx, G, D, seed, kv_pad=0, H=None):
        from paged_top_sparse_gb300 import binding as B

        self.B, self.q_lens, self.ctx, self.G, self.D = B, q_lens, ctx, G, D
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.g = g
        pages = [(c + n - 1) // 128 + 1 if n else 0 for n, c in zip(q_lens, ctx)]
        NP, T = sum(pages) + 2, sum(q_lens)
        pt = np.full((len(q_lens), max(pages)), -1, np.int32)
        perm = np.random.default_rng(seed).permutation(NP).astype(np.int32)
        at = 0
        for b, n in enumerate(pages):
            pt[b, :n] = perm[at:at + n]
            at += n
        self.pt = torch.from_numpy(pt).to(DEV)
        raw = lambda: torch.randint(0, 256, (NP, G, 128, D), generator=g, device=DEV, dtype=torch.uint8)
        # any code but NaN
        self.kc, self.vc = (torch.where((x & 0x7F) == 0x7F, x & 0x80, x).view(F8) for x in (raw(), raw()))
        self.ks, self.vs = (torch.exp2(torch.randint(-12, 1, (NP, G), generator=g, device=DEV).float())
                            for _ in "kv")
        self.new = torch.randn((T, (2 + kv_pad) * G, D), generator=g, device=DEV).bfloat16()
        self.k, self.v = self.new[:, :G], self.new[:, G:2 * G]
        self.plan = B.Plan(q_lens, ctx, H or G, G, D, 1, pt.shape[1], NP, kv_dtype="e4m3")
        self.ws = torch.zeros(self.plan.workspace_bytes, dtype=torch.uint8, device=DEV)
        B.sps_plan_upload(self.plan, self.ws)

    def status(self):
        return self.B.sps_read_device_status(self.plan, self.ws)


BATCHES = [([200, 64, 131, 1], [1000, 2900, 555, 127]), ([1, 1, 1, 0, 2], [0, 127, 128, 40, 255]),
           ([1] * 70, [(37 * i) % 300 for i in range(70)]), ([700], [0])]


def edges(x, scale):
    """Rows and whole tokens that decide the rounding: zeros of both signs, tiny and huge values, the
    border of a scale (448 2^k, and the next BF16 value above it), infinities and NaN."""
    x = x.clone()
    n = x.shape[0]
    for i in range(0, n, 7):
        x[i] = 0.0
        x[i, :, ::2] = -0.0
    x[1::11] *= 1e-20
    x[2::13] = x[2::13] * 1e4
    x[3::17, 0, 0] = 448.0 * scale
    x[5::19, 0, 1] = 450.0 * scale
    if n > 140:
        x[140, 0, 3] = float("inf")
        x[100, -1, 5] = float("nan")
    return x


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 3])
@pytest.mark.parametrize("q_lens,ctx", BATCHES)
def test_append_bytes_match_the_rule(q_lens, ctx, G, D):
    b = Batch(q_lens, ctx, G, D, seed=len(q_lens) + D)
    k, v = edges(b.k, 2.0 ** -6).contiguous(), edges(b.v.float() * 100, 2.0).bfloat16().contiguous()
    want = [append_rule(x.double(), q_lens, ctx, b.pt, c, s) for x, c, s in ((k, b.kc, b.ks), (v, b.vc, b.vs))]
    b.B.sps_kv_append(b.plan, k, v, b.pt, b.kc, b.vc, b.ks, b.vs, b.ws)
    torch.cuda.synchronize()
    assert b.status() == 0
    for (codes, scales), c, s in zip(want, (b.kc, b.vc), (b.ks, b.vs)):
        assert torch.equal(scales, s)
        bad = codes.view(torch.uint8) != c.view(torch.uint8)
        assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4].tolist())


def test_earlier_tokens_under_a_scale_of_any_value():
    """A page written by others may have a scale that is no power of two: it is kept while it holds the new
    rows, and left for a power of two when it does not."""
    q_lens, ctx = [3, 3, 5], [50, 100, 126]
    b = Batch(q_lens, ctx, 2, 128, 7)
    b.ks[:] = 0.37
    b.vs[:] = 3.3e-4
    want = [append_rule(x.double(), q_lens, ctx, b.pt, c, s)
            for x, c, s in ((b.k, b.kc, b.ks), (b.v, b.vc, b.vs))]
    b.B.sps_kv_append(b.plan, b.k.contiguous(), b.v.contiguous(), b.pt, b.kc, b.vc, b.ks, b.vs, b.ws)
    torch.cuda.synchronize()
    for (codes, scales), c, s in zip(want, (b.kc, b.vc), (b.ks, b.vs)):
        assert torch.equal(scales, s)
        assert torch.equal(codes.view(torch.uint8), c.view(torch.uint8))


def rotated(x, pos, inv_freq, w, eps, interleaved):
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    a = pos.double()[:, None] * inv_freq.double()
    c, s = a.cos()[:, None], a.sin()[:, None]
    R = 2 * inv_freq.numel()
    r = x[..., :R]
    if interleaved:
        p, q = r[..., 0::2], r[..., 1::2]
        r = torch.stack((p * c - q * s, q * c + p * s), -1).flatten(-2)
    else:
        p, q = r[..., :R // 2], r[..., R // 2:]
        r = torch.cat((p * c - q * s, q * c + p * s), -1)
    return torch.cat((r, x[..., R:]), -1)


@pytest.mark.parametrize("D,R,interleaved,norm", [(128, 128, False, True), (128, 64, True, True),
                                                  (64, 64, False, False), (64, 32, True, True),
                                                  (128, 0, False, True)])
@pytest.mark.parametrize("q_lens,ctx", BATCHES)
def test_append_with_rotation(q_lens, ctx, D, R, interleaved, norm):
    b = Batch(q_lens, ctx, 2, D, seed=R + len(q_lens), kv_pad=1)
    f = (1e4 ** (-torch.arange(max(R // 2, 1), device=DEV, dtype=torch.float64) * 2 / max(R, 1))).float()
    rope = b.B.Rope(f, interleaved=interleaved) if R else None
    w = 1 + 0.2 * torch.randn(D, generator=b.g, device=DEV) if norm else None
    pos = torch.cat([torch.arange(c, c + n, device=DEV) for c, n in zip(ctx, q_lens)])
    rows = rotated(b.k, pos, f[:R // 2], w, 1e-6, interleaved)
    old_k, old_v = (b.kc.clone(), b.ks.clone()), (b.vc.clone(), b.vs.clone())
    b.B.sps_kv_append_rope(b.plan, b.k, b.v, w, 1e-6, rope, b.pt, b.kc, b.vc, b.ks, b.vs, b.ws)
    torch.cuda.synchronize()
    assert b.status() == 0
    codes, scales = append_rule(b.v.double(), q_lens, ctx, b.pt, *old_v)
    assert torch.equal(scales, b.vs) and torch.equal(codes.view(torch.uint8), b.vc.view(torch.uint8))
    codes, scales = append_rule(rows, q_lens, ctx, b.pt, *old_k)
    # the FP32 row is within 2^-19 of the row's size of the definition (the angle's 2^-24 turns, the norm,
    # two products): a scale could go the other way only for a maximum that near its border
    assert torch.equal(scales, b.ks)
    got, t = torch.zeros_like(rows), 0
    for i, (n, c) in enumerate(zip(q_lens, ctx)):
        for j in range(n):
            phys, slot = int(b.pt[i, (c + j) // 128]), (c + j) % 128
            got[t] = b.kc[phys, :, slot].double() * b.ks[phys].double()[:, None]
            t += 1
    size = rows.abs().amax(-1, keepdim=True)
    step = torch.stack([b.ks[int(b.pt[i, (c + j) // 128])] for i, (n, c) in enumerate(zip(q_lens, ctx))
                        for j in range(n)]).double()[..., None]
    # half an E4M3 step: 2^-4 relative, 2^-10 of the scale below 2^-6 of it
    tol = torch.maximum(2.0 ** -4 * rows.abs(), 2.0 ** -10 * step) + 2.0 ** -18 * size
    assert bool(((got - rows).abs() <= tol).all())
    # what the call does not write stays, and earlier rows move with the scale alone
    written = torch.zeros(b.kc.shape[:3], dtype=torch.bool, device=DEV)
    for i, (n, c) in enumerate(zip(q_lens, ctx)):
        for j in range(n):
            written[int(b.pt[i, (c + j) // 128]), :, (c + j) % 128] = True
    same = codes.view(torch.uint8) == b.kc.view(torch.uint8)
    assert bool(same[~written].all())


@pytest.mark.parametrize("D", [64, 128])
def test_many_heads_share_a_block(D):
    """Enough (page, head) tiles that a block takes several heads of a page, one behind the other; rows of
    a fused projection; new tokens behind earlier ones."""
    q_lens, ctx, G = [1500, 700, 130], [77, 0, 1000], 40
    b = Batch(q_lens, ctx, G, D, seed=D, kv_pad=1)
    f = (1e4 ** (-torch.arange(D // 2, device=DEV, dtype=torch.float64) * 2 / D)).float()
    pos = torch.cat([torch.arange(c, c + n, device=DEV) for c, n in zip(ctx, q_lens)])
    w = 1 + 0.2 * torch.randn(D, generator=b.g, device=DEV)
    want_v = append_rule(b.v.double(), q_lens, ctx, b.pt, b.vc, b.vs)
    want_k = append_rule(rotated(b.k, pos, f, w, 1e-6, False), q_lens, ctx, b.pt, b.kc, b.ks)
    b.B.sps_kv_append_rope(b.plan, b.k, b.v, w, 1e-6, b.B.Rope(f), b.pt, b.kc, b.vc, b.ks, b.vs, b.ws)
    torch.cuda.synchronize()
    assert b.status() == 0
    assert torch.equal(want_v[1], b.vs) and torch.equal(want_v[0].view(torch.uint8), b.vc.view(torch.uint8))
    assert torch.equal(want_k[1], b.ks)
    # a key next to a code's border may go either way: by a step at most, and few of them (the FP32 row is
    # off by 2^-19 of its size, a step is 2^-4 of a code at least: less than one in a thousand)
    x, y = want_k[0].double(), b.kc.double()
    step = torch.maximum(x.abs(), y.abs()).clamp(min=2.0 ** -6) * 2.0 ** -3
    assert bool(((x - y).abs() <= step).all()) and float((x != y).double().mean()) < 1e-3


def test_positions_of_their_own_axes():
    """Rotation by positions on three axes, as sps_rope gives them, into the E4M3 cache."""
    q_lens, ctx, G, D, R = [140, 3], [100, 127], 2, 128, 64
    b = Batch(q_lens, ctx, G, D, 9)
    T = sum(q_lens)
    f = (1e4 ** (-torch.arange(R // 2, device=DEV, dtype=torch.float64) * 2 / R)).float()
    pos = torch.randint(-500, 70000, (3, T), generator=b.g, device=DEV, dtype=torch.int32)
    axis = [j * 3 // (R // 2) for j in range(R // 2)]
    for inter in (False, True):
        rope = b.B.Rope(f, positions=pos, pair_axis=axis, interleaved=inter)
        x = b.k.double()
        a = pos[torch.tensor(axis, device=DEV)].T.double() * f.double()
        c, s = a.cos()[:, None], a.sin()[:, None]
        u, v = (x[..., 0:R:2], x[..., 1:R:2]) if inter else (x[..., :R // 2], x[..., R // 2:R])
        r = (torch.stack((u * c - v * s, v * c + u * s), -1).flatten(-2) if inter
             else torch.cat((u * c - v * s, v * c + u * s), -1))
        rows = torch.cat((r, x[..., R:]), -1)
        codes, scales = append_rule(rows, q_lens, ctx, b.pt, b.kc, b.ks)
        b.B.sps_kv_append_rope(b.plan, b.k, b.v, None, 0.0, rope, b.pt, b.kc, b.vc, b.ks, b.vs, b.ws)
        torch.cuda.synchronize()
        assert torch.equal(scales, b.ks)
        y, z = codes.double(), b.kc.double()
        step = torch.maximum(y.abs(), z.abs()).clamp(min=2.0 ** -6) * 2.0 ** -3
        assert bool(((y - z).abs() <= step).all()) and float((y != z).double().mean()) < 1e-3


def test_token_by_token_reaches_the_values_of_one_append():
    """300 tokens at once, and one at a time: the same scales, and the same values but where a code fell
    below 2^-6 of its scale on the way (rounded twice)."""
    from paged_top_sparse_gb300 import binding as B

    N, G, D = 300, 2, 64
    one = Batch([N], [0], G, D, 11)
    x = (one.new.float() * torch.exp2(torch.arange(N, device=DEV) / 40)[:, None, None]).bfloat16()
    k, v = x[:, :G].contiguous(), x[:, G:].contiguous()
    B.sps_kv_append(one.plan, k, v, one.pt, one.kc, one.vc, one.ks, one.vs, one.ws)
    two = Batch([N], [0], G, D, 11)
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device=DEV)
    for t in range(N):
        plan = B.Plan([1], [t], G, G, D, 1, two.pt.shape[1], two.kc.shape[0], kv_dtype="e4m3")
        assert plan.workspace_bytes <= ws.numel()
        B.sps_plan_upload(plan, ws)
        B.sps_kv_append(plan, k[t:t + 1], v[t:t + 1], two.pt, two.kc, two.vc, two.ks, two.vs, ws)
    torch.cuda.synchronize()
    for a, b, s, u in ((one.kc, two.kc, one.ks, two.ks), (one.vc, two.vc, one.vs, two.vs)):
        assert torch.equal(s, u)
        for p in range(3):
            phys, n = int(one.pt[0, p]), min(128, N - 128 * p)
            x, y = a[phys, :, :n].double(), b[phys, :, :n].double()
            near = (x.abs() < 2.0 ** -5) & ((x - y).abs() <= 2.0 ** -9)
            assert bool(((x == y) | near).all())


def test_bad_page_is_reported_and_skipped():
    b = Batch([3, 5], [10, 300], 2, 64, 5)
    before = b.kc.clone(), b.ks.clone()
    b.pt[1, 2] = b.kc.shape[0]
    b.B.sps_kv_append(b.plan, b.k.contiguous(), b.v.contiguous(), b.pt, b.kc, b.vc, b.ks, b.vs, b.ws)
    torch.cuda.synchronize()
    assert b.status() == 2  # SPS_DEV_BAD_PAGE
    page = int(b.pt[0, 0])
    others = torch.arange(b.kc.shape[0], device=DEV) != page
    assert torch.equal(b.kc.view(torch.uint8)[others], before[0].view(torch.uint8)[others])
    assert torch.equal(b.ks[others], before[1][others])


@pytest.mark.parametrize("q", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,G,D", [(16, 1, 128), (8, 2, 64)])
def test_captured_step_of_tables_rotation_append_and_attention(H, G, D, q):
    """Prompts, then single tokens through one graph of page tables, norm and rotation, append and
    attention, replayed while the contexts grow over page borders: the same bits as eager calls on a cache
    of their own, and the attention of the whole sequences within its bounds."""
    from paged_top_sparse_gb300 import binding as B

    n, rows, steps = 3, 5, 4
    prompt = [126, 500, 1]
    quant = q == "e4m3"
    g = torch.Generator(device=DEV)
    g.manual_seed(H + D)
    rope = B.Rope((1e4 ** (-torch.arange(D // 2, device=DEV, dtype=torch.float64) * 2 / D)).float())
    w = 1 + 0.1 * torch.randn(D, generator=g, device=DEV)
    mk = lambda q_lens, ctx: B.Plan(q_lens, ctx, H, G, D, 1, rows, n * rows, q_dtype=q, kv_dtype="e4m3")
    fill = mk(prompt, [0] * n)
    plans = [mk([1] * n, [c + i for c in prompt]) for i in range(steps)]
    free = torch.randperm(n * rows, generator=g, device=DEV).int()
    qs = 0.02 if quant else 1.0

    class Side:
        def __init__(self):
            self.kc, self.vc = (torch.full((n * rows, G, 128, D), 0x7F, dtype=torch.uint8, device=DEV) for _ in "kv")
            self.ks, self.vs = (torch.full((n * rows, G), float("nan"), device=DEV) for _ in "kv")
            self.pt = torch.full((n, rows), -1, dtype=torch.int32, device=DEV)
            self.state = torch.zeros(2, dtype=torch.int32, device=DEV)
            self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
            self.q_lens = torch.zeros(n, dtype=torch.int32, device=DEV)
            self.ctx = torch.zeros(n, dtype=torch.int32, device=DEV)
            self.slots = torch.zeros(n, dtype=torch.int64, device=DEV)
            self.ws = torch.zeros(max(p.workspace_bytes for p in plans + [fill]), dtype=torch.uint8, device=DEV)
            size = max(B.paged_attention_scratch(p) for p in plans + [fill])
            self.scratch = torch.zeros(size, dtype=torch.uint8, device=DEV)
            self.x = torch.zeros((n, H + 2 * G, D), dtype=torch.bfloat16, device=DEV)
            self.out = torch.zeros((n, H, D), dtype=torch.bfloat16, device=DEV)
            self.q = torch.zeros((n, H, D), dtype=torch.uint8 if quant else torch.bfloat16, device=DEV)

        def step(self, plan, x, qr, out, slots, stream=None):
            B.sps_page_tables(self.q_lens, self.ctx, free, self.state, self.pt, slots, None, None, self.status, stream)
            B.sps_qk_norm_rope(plan, x[:, :H], None, w, None, 1e-6, rope, qr, qs, None, self.ws, stream)
            B.sps_kv_append_rope(plan, x[:, H:H + G], x[:, H + G:], w, 1e-6, rope, self.pt, self.kc, self.vc,
                                 self.ks, self.vs, self.ws, stream)
            B.paged_attention_fwd(plan, qr, qs, self.kc, self.vc, self.ks, self.vs, self.pt, out, None,
                                  self.scratch, self.ws, stream)

        def lengths(self, q_lens, ctx):
            self.q_lens.copy_(torch.tensor(q_lens, dtype=torch.int32))
            self.ctx.copy_(torch.tensor(ctx, dtype=torch.int32))

    a, b = Side(), Side()
    T = sum(prompt)
    px = torch.randn((T, H + 2 * G, D), generator=g, device=DEV).bfloat16()
    for side in (a, b):
        side.lengths(prompt, [0] * n)
        B.sps_plan_upload(fill, side.ws)
        side.step(fill, px, torch.empty((T, H, D), dtype=side.q.dtype, device=DEV),
                  torch.empty((T, H, D), dtype=torch.bfloat16, device=DEV),
                  torch.zeros(T, dtype=torch.int64, device=DEV))
        torch.cuda.synchronize()
        assert int(side.status) == 0 and B.sps_read_device_status(fill, side.ws) == 0
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    a.lengths([1] * n, prompt)
    B.sps_plan_upload(plans[0], a.ws, s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        a.step(plans[0], a.x, a.q, a.out, a.slots, s)
    queries = []
    for i, plan in enumerate(plans):
        x = torch.randn((n, H + 2 * G, D), generator=g, device=DEV).bfloat16()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            a.x.copy_(x)
            a.lengths([1] * n, [c + i for c in prompt])
            B.sps_plan_upload(plan, a.ws, s)
            graph.replay()
        b.x.copy_(x)
        b.lengths([1] * n, [c + i for c in prompt])
        B.sps_plan_upload(plan, b.ws)
        b.step(plan, b.x, b.q, b.out, b.slots)
        torch.cuda.synchronize()
        assert int(a.status) == 0 and B.sps_read_device_status(plan, a.ws) == 0
        for u, v in ((a.q, b.q), (a.kc, b.kc), (a.vc, b.vc), (a.pt, b.pt), (a.slots, b.slots), (a.out, b.out)):
            assert torch.equal(u, v)
        queries.append(a.q.clone())
        # attention in FP64 over what the cache and the queries hold
        for r in range(n):
            N = prompt[r] + i + 1
            ids = a.pt[r, :(N - 1) // 128 + 1].long()
            assert int(a.slots[r]) == int(ids[-1]) * 128 + (N - 1) % 128
            k, v = ((c.view(F8)[ids].double() * sc[ids].double()[:, :, None, None]).transpose(0, 1)
                    .reshape(G, -1, D)[:, :N] for c, sc in ((a.kc, a.ks), (a.vc, a.vs)))
            qd = (a.q[r].view(F8).double() * qs if quant else a.q[r].double()).view(G, H // G, D)
            p = torch.softmax(torch.einsum("ghd,gkd->ghk", qd, k) * D ** -0.5, -1)
            ref = torch.einsum("ghk,gkd->ghd", p, v).reshape(H, D)
            mag = torch.einsum("ghk,gkd->ghd", p, v.abs()).reshape(H, D)
            top = (p.amax(-1) * v.abs().amax((1, 2))[:, None]).reshape(H, 1)
            tol = (2.0 ** -11 + 2.0 ** -14) * mag + 2.0 ** -8 * ref.abs() + N * 2.0 ** -31 * top
            assert bool(((a.out[r].double() - ref).abs() <= tol).all())
