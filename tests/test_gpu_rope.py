"""GPU checks of sps_qk_norm_rope and sps_kv_append_rope through the C ABI against the formulas in
64 bits: head dims, rotated dims, both pair layouts, several axes, far and negative positions,
strided views, in place, E4M3 and NVFP4 outputs, and a batch with an empty request."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from paged_top_sparse_gb300 import synth

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
EPS = 1e-6
# FP32 arithmetic in front of the one rounding, relative to the two elements of a pair: the sum of
# squares takes 13 roundings of 2^-24 (halved by the root), the root and two products 6 more, the
# cosine and sine 2^-21 in all, the rotation two more: under 2^-19 together; twice that is allowed
NOISE = 2.0 ** -18
BF16_HALF, E4M3_HALF = 2.0 ** -8, 2.0 ** -4


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_top_sparse_gb300 import build

    build.build()


def _plan(q_lens, ctx, H, G, D, **kw):
    from paged_top_sparse_gb300 import binding as B

    pages = [(c + q - 1) // 128 + 1 if q else 0 for q, c in zip(q_lens, ctx)]
    plan = B.Plan(q_lens, ctx, H, G, D, 1, max(pages), sum(pages), **kw)
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device=DEV)
    B.sps_plan_upload(plan, ws)
    pos = np.concatenate([c + np.arange(q) for q, c in zip(q_lens, ctx)])
    return plan, ws, pos, pages


def _inv_freq(rot):
    return torch.from_numpy((1e6 ** (-np.arange(rot // 2) * 2.0 / max(rot, 1))).astype(np.float32))


def _reference(x, w, rot, angle, interleaved):
    """x [T, heads, D] FP64 -> (result, |n_a| + |n_b| per element)."""
    n = x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + EPS) * w
    y, mag = n.copy(), np.abs(n)
    h = rot // 2
    ia = np.arange(h) * 2 if interleaved else np.arange(h)
    ib = ia + 1 if interleaved else ia + h
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    a, b = n[..., ia], n[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = np.abs(a) + np.abs(b)
    return y, mag


def _f64(t):
    return t.detach().cpu().float().numpy().astype(np.float64)


def _angle(inv_freq, pos, axis=None):
    """[T, pairs]; pos [axes, T]."""
    f = inv_freq.cpu().numpy().astype(np.float64)
    axis = [0] * len(f) if axis is None else axis
    return pos[axis].T.astype(np.float64) * f if len(f) else np.zeros((pos.shape[1], 0))


def _close(got, ref, mag, half):
    bad = np.abs(_f64(got) - ref) > half * np.abs(ref) + NOISE * mag
    assert not bad.any(), (int(bad.sum()), np.abs(_f64(got) - ref).max())


def _weights(rng, D, norm):
    return torch.from_numpy((1 + 0.3 * rng.standard_normal(D)).astype(np.float32)).to(DEV) if norm else None


def _np(w):
    return None if w is None else w.cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("D,rot,inter,H,G,qn,kn", [
    (128, 128, False, 32, 2, True, True),
    (128, 128, True, 5, 5, True, False),
    (128, 64, False, 7, 1, False, True),
    (128, 96, False, 4, 2, True, True),
    (128, 48, True, 3, 3, False, False),
    (128, 0, False, 3, 1, True, True),
    (64, 64, False, 6, 2, True, True),
    (64, 16, False, 1, 1, True, True),
    (64, 32, True, 9, 3, True, True),
])
def test_qk_norm_rope_matches_the_formula(D, rot, inter, H, G, qn, kn):
    from paged_top_sparse_gb300 import binding as B

    rng = np.random.default_rng(D + rot + H)
    q_lens, ctx = [1, 0, 133, 70], [5, 9, (1 << 20) - 133, 127]
    plan, ws, pos, _ = _plan(q_lens, ctx, H, G, D)
    T = len(pos)
    qkv = torch.from_numpy(rng.standard_normal((T, H + 2 * G, D)).astype(np.float32)).to(DEV).bfloat16()
    qkv[3] *= 1e-18  # squares below FP32's range: eps carries the norm
    qkv[4] *= 1e15
    q, k = qkv[:, :H], qkv[:, H:H + G]
    keep = qkv.clone()
    qw, kw = _weights(rng, D, qn), _weights(rng, D, kn)
    f = _inv_freq(rot).to(DEV)
    rope = B.Rope(f, interleaved=inter) if rot else None
    q_out = torch.full((T, H, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    k_out = torch.full((T, G, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    B.sps_qk_norm_rope(plan, q, k, qw, kw, EPS, rope, q_out, 1.0, k_out, ws)
    torch.cuda.synchronize()
    assert torch.equal(qkv, keep)
    ang = _angle(f, pos[None])
    for x, w, got in ((q, qw, q_out), (k, kw, k_out)):
        _close(got, *_reference(_f64(x), _np(w), rot, ang, inter), BF16_HALF)
    # queries alone, and in place in the projection's output: the same bits
    only = torch.empty_like(q_out)
    B.sps_qk_norm_rope(plan, q, None, qw, None, EPS, rope, only, 1.0, None, ws)
    B.sps_qk_norm_rope(plan, q, k, qw, kw, EPS, rope, q, 1.0, k, ws)
    torch.cuda.synchronize()
    assert torch.equal(only, q_out)
    assert torch.equal(q, q_out) and torch.equal(k, k_out)
    assert torch.equal(qkv[:, H + G:], keep[:, H + G:])


@pytest.mark.parametrize("D,inter,axes", [(128, False, 3), (64, True, 2), (128, True, 4)])
def test_several_axes_far_and_negative_positions(D, inter, axes):
    from paged_top_sparse_gb300 import binding as B

    rng = np.random.default_rng(7 * D + axes)
    plan, ws, pos, _ = _plan([97], [0], 4, 2, D)
    T = 97
    p = rng.integers(-(1 << 31), 1 << 31, (axes, T)).astype(np.int32)
    p[:, :4] = np.array([0, 1, -(1 << 31), (1 << 31) - 1])
    p[1:, 50:] = rng.integers(0, 64, (axes - 1, T - 50))
    n = D // 2
    axis = [j % axes for j in range(n)]
    # frequencies of every size, zero, negative and above one among them
    f = torch.from_numpy((np.exp(rng.uniform(-30, 0, n)) * np.where(rng.random(n) < 0.2, -1, 1)).astype(np.float32))
    f[0], f[1], f[2], f[3] = 1.0, 0.0, 3.5, 1e-40
    f = f.to(DEV)
    q = torch.from_numpy(rng.standard_normal((T, 4, D)).astype(np.float32)).to(DEV).bfloat16()
    out = torch.empty_like(q)
    rope = B.Rope(f, positions=torch.from_numpy(p).to(DEV), pair_axis=axis, interleaved=inter)
    B.sps_qk_norm_rope(plan, q, None, None, None, EPS, rope, out, 1.0, None, ws)
    torch.cuda.synchronize()
    # a product has at most 55 bits: 64-bit rounding is below 2^-20 radians, and cos and sin reduce
    # it in full
    _close(out, *_reference(_f64(q), None, D, _angle(f, p, axis), inter), BF16_HALF)


@pytest.mark.parametrize("D,inter", [(128, False), (64, True)])
def test_e4m3_queries(D, inter):
    from paged_top_sparse_gb300 import binding as B

    rng = np.random.default_rng(D)
    plan, ws, pos, _ = _plan([65, 3], [300, 0], 4, 2, D)
    T = 68
    q = torch.from_numpy(rng.standard_normal((T, 4, D)).astype(np.float32)).to(DEV).bfloat16()
    q[0] *= 1000.0  # without a norm these saturate
    k = torch.from_numpy(rng.standard_normal((T, 2, D)).astype(np.float32)).to(DEV).bfloat16()
    wide = torch.full((T, 5, D), 0x55, dtype=torch.uint8, device=DEV)
    k_out = torch.empty_like(k)
    f, scale = _inv_freq(D).to(DEV), 0.0131
    B.sps_qk_norm_rope(plan, q, k, None, None, EPS, B.Rope(f, interleaved=inter), wide[:, :4],
                       scale, k_out, ws)
    torch.cuda.synchronize()
    ang = _angle(f, pos[None])
    ref, mag = _reference(_f64(q), None, D, ang, inter)
    got = wide[:, :4].contiguous().view(torch.float8_e4m3fn).float().cpu().numpy().astype(np.float64)
    want = np.clip(ref / scale, -448, 448)
    # half a step of E4M3, or of its subnormals (2^-9)
    tol = np.maximum(E4M3_HALF * np.abs(want), 2.0 ** -10) + NOISE * mag / scale
    assert (np.abs(got - want) <= tol).all()
    assert bool((wide[:, 4] == 0x55).all())
    _close(k_out, *_reference(_f64(k), None, D, ang, inter), BF16_HALF)


def _cache(rng, NP, G, D, kv):
    if kv == "bf16":
        mk = lambda: rng.integers(0, 1 << 16, (NP, G, 128, D), dtype=np.uint16)
        return [mk(), mk(), None, None]
    mk = lambda d: rng.integers(0, 256, (NP, G, 128, d), dtype=np.uint8)
    return [mk(D // 2), mk(D // 2), mk(D // 16), mk(D // 16)]


def _dev(a):
    return None if a is None else torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).to(DEV)


@pytest.mark.parametrize("kv,D,rot,inter,norm,G", [
    ("bf16", 128, 128, False, True, 2), ("bf16", 64, 32, True, False, 1),
    ("bf16", 128, 64, False, True, 3), ("nvfp4", 128, 128, False, True, 2),
    ("nvfp4", 64, 64, False, True, 5), ("nvfp4", 128, 96, False, False, 1),
    ("nvfp4", 128, 0, False, False, 2),
])
def test_kv_append_rope(kv, D, rot, inter, norm, G):
    from paged_top_sparse_gb300 import binding as B

    rng = np.random.default_rng(11 * D + rot + G)
    q_lens, ctx = [200, 0, 1, 1, 129], [1000, 40, 127, 128, 65500]
    plan, ws, pos, pages = _plan(q_lens, ctx, 2 * G, G, D, q_dtype="bf16" if kv == "bf16" else "e4m3",
                                 kv_dtype=kv)
    T, NP = len(pos), sum(pages)
    pt = np.full((len(q_lens), max(pages)), -1, np.int32)
    perm, at = rng.permutation(NP).astype(np.int32), 0
    for b, n in enumerate(pages):
        pt[b, :n] = perm[at:at + n]
        at += n
    kv_new = rng.standard_normal((T, 2 * G + 1, D)).astype(np.float32)
    kv_new[0::5, :, 16:32] = 0.0
    kv_new[1::5] *= 1e-6
    kv_new[2::5] *= 3e3
    new = torch.from_numpy(kv_new).to(DEV).bfloat16()
    k, v = new[:, :G], new[:, G + 1:]
    w = _weights(rng, D, norm)
    f = _inv_freq(rot).to(DEV)
    host = _cache(rng, NP, G, D, kv)
    kc, vc, ks, vs = [_dev(a) for a in host]
    B.sps_kv_append_rope(plan, k, v, w, EPS, B.Rope(f, interleaved=inter) if rot else None,
                         torch.from_numpy(pt).to(DEV), kc, vc, ks, vs, ws)
    torch.cuda.synchronize()
    assert B.sps_read_device_status(plan, ws) == 0
    ref, mag = _reference(_f64(k), _np(w), rot, _angle(f, pos[None]), inter)
    req = np.concatenate([np.full(q, b) for b, q in enumerate(q_lens)]).astype(int)
    page, slot = pt[req, pos // 128], pos % 128
    new_bits = [_f64(k), v.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)]
    untouched = np.ones((NP, 128), bool)
    untouched[page, slot] = False
    for i, (before, after) in enumerate(zip(host, (kc, vc, ks, vs))):
        if before is None:
            continue
        after = after.cpu().numpy().view(before.dtype)
        hold = untouched[:, None, :, None] & np.ones_like(before, bool)
        assert np.array_equal(after[hold], before[hold]), i
    got_k = kc.cpu().numpy()[page, :, slot]
    got_v = vc.cpu().numpy()[page, :, slot]
    if kv == "bf16":
        assert np.array_equal(got_v.view(np.uint16), new_bits[1])
        _close(torch.from_numpy(got_k.view(np.int16)).view(torch.bfloat16), ref, mag, BF16_HALF)
        return
    want_codes, want_scales = synth.quantize_nvfp4(_f64(v).astype(np.float32))
    # the fixture encoder drops the sign of a zero code, the append keeps it (its bits are held to
    # sps_kv_append's in test_append_with_nothing_to_do_equals_the_plain_append)
    unsigned0 = lambda c: np.stack([np.where(n == 8, 0, n) for n in (c & 15, c >> 4)])
    assert np.array_equal(unsigned0(got_v), unsigned0(want_codes))
    assert np.array_equal(vs.cpu().numpy()[page, :, slot], want_scales)
    # keys: a scale or code next to a border may fall either way within the FP32 noise
    sc = ks.cpu().numpy()[page, :, slot]
    noise = NOISE * mag.reshape(T, G, D // 16, 16)
    y = ref.reshape(T, G, D // 16, 16)
    lo = synth.f32_to_e4m3_bits((np.abs(y) - noise).clip(0).max(-1) / 6.0)
    hi = synth.f32_to_e4m3_bits((np.abs(y) + noise).max(-1) / 6.0)
    assert ((sc == lo) | (sc == hi)).all()
    s = torch.from_numpy(sc).view(torch.float8_e4m3fn).double().numpy()[..., None]
    codes = np.stack((got_k & 15, got_k >> 4), -1).reshape(y.shape)
    val = np.where(codes & 8, -1.0, 1.0) * synth._E2M1_MAGS[codes & 7]
    safe = np.where(s > 0, s, 1.0)
    bound = []
    for z in (y - noise, y + noise):
        c = synth._e2m1_code(z / safe)
        bound.append(np.where(c & 8, -1.0, 1.0) * synth._E2M1_MAGS[c & 7])
    inside = (val >= bound[0]) & (val <= bound[1])
    assert (inside | (s == 0)).all()
    assert (val[np.broadcast_to(s == 0, val.shape)] == 0).all()


def test_append_reports_a_bad_page_and_skips_its_rows():
    from paged_top_sparse_gb300 import binding as B

    plan, ws, pos, pages = _plan([3, 2], [126, 0], 2, 1, 64)
    NP = sum(pages)
    pt = torch.tensor([[0, NP], [2, -1]], dtype=torch.int32, device=DEV)
    k = torch.ones((5, 1, 64), dtype=torch.bfloat16, device=DEV)
    kc = torch.zeros((NP, 1, 128, 64), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    B.sps_kv_append_rope(plan, k, k, None, EPS, None, pt, kc, vc, None, None, ws)
    torch.cuda.synchronize()
    assert B.sps_read_device_status(plan, ws) == 2  # SPS_DEV_BAD_PAGE
    want = torch.zeros_like(kc)
    want[0, 0, 126:] = 1
    want[2, 0, :2] = 1
    assert torch.equal(kc, want) and torch.equal(vc, want)


def test_append_with_nothing_to_do_equals_the_plain_append():
    """No norm and no rotation: the bytes sps_kv_append writes, for both cache types."""
    from paged_top_sparse_gb300 import binding as B

    rng = np.random.default_rng(3)
    for kv in ("bf16", "nvfp4"):
        plan, ws, pos, pages = _plan([150, 9], [77, 3000], 4, 2, 128, kv_dtype=kv,
                                     q_dtype="bf16" if kv == "bf16" else "e4m3")
        NP = sum(pages)
        pt = torch.full((2, max(pages)), -1, dtype=torch.int32)
        pt[0, :pages[0]] = torch.arange(pages[0], dtype=torch.int32)
        pt[1, :pages[1]] = torch.arange(pages[0], NP, dtype=torch.int32)
        pt = pt.to(DEV)
        k, v = (torch.from_numpy(rng.standard_normal((159, 2, 128)).astype(np.float32)).to(DEV).bfloat16()
                for _ in range(2))
        host = _cache(rng, NP, 2, 128, kv)
        a, b = [_dev(x) for x in host], [_dev(x) for x in host]
        B.sps_kv_append(plan, k, v, pt, *a, ws)
        B.sps_kv_append_rope(plan, k, v, None, 0.0, None, pt, *b, ws)
        torch.cuda.synchronize()
        for x, y in zip(a, b):
            assert x is None or torch.equal(x, y)


def test_replay_in_a_graph_on_another_stream():
    from paged_top_sparse_gb300 import binding as B

    rng = np.random.default_rng(5)
    plan, ws, pos, pages = _plan([1, 1, 1], [500, 30, 0], 8, 2, 128)
    f = _inv_freq(128).to(DEV)
    rope = B.Rope(f)
    q = torch.from_numpy(rng.standard_normal((3, 8, 128)).astype(np.float32)).to(DEV).bfloat16()
    out, eager = torch.empty_like(q), torch.empty_like(q)
    w = _weights(rng, 128, True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        B.sps_qk_norm_rope(plan, q, None, w, None, EPS, rope, out, 1.0, None, ws)
    q.mul_(-2.0)
    out.zero_()
    g.replay()
    B.sps_qk_norm_rope(plan, q, None, w, None, EPS, rope, eager, 1.0, None, ws)
    torch.cuda.synchronize()
    assert torch.equal(out, eager) and bool(out.any())


@pytest.mark.parametrize("D", [128, 64])
def test_e4m3_queries_with_nothing_to_do_are_the_quantisers_codes(D):
    """No norm and no rotation: sps_quantize_e4m3's codes, for every BF16 value but NaN.  With some of
    these scales (6.5, 7 / 512) a product with 1 / q_scale in place of the division would move codes
    next to a border; a significand one unit off a short one, all ones, the smallest and the largest
    scales are where a corrected product could go wrong."""
    from paged_top_sparse_gb300 import binding as B

    bits = torch.arange(1 << 16, device=DEV).to(torch.int32)
    bits[(bits & 0x7FFF) > 0x7F80] = 0
    x = bits.to(torch.int16).view(torch.bfloat16).view(-1, 4, D).contiguous()
    T = x.shape[0]
    plan, ws, pos, _ = _plan([T], [0], 4, 2, D)
    ulp = 2.0 ** -23
    scales = [0.3, 0.7, 0.75, 1.5, 6.5, 0.013671875, 0.02, 3e-3, 1 + ulp, 1.125 - ulp, 1.25 + 3 * ulp,
              2 - ulp, 0.875 * (1 - ulp), 1e-38, 3e-39, 1e-30, 2.0 ** -90, 2.0 ** 90, 1e30, 1e38]
    scales += list(np.exp(np.random.default_rng(D).uniform(-8, 3, 30)))
    for scale in scales:
        scale = float(np.float32(scale))
        got, want = (torch.zeros((T, 4, D), dtype=torch.uint8, device=DEV) for _ in range(2))
        B.sps_qk_norm_rope(plan, x, None, None, None, EPS, None, got, scale, None, ws)
        B.sps_quantize_e4m3(x, scale, want)
        torch.cuda.synchronize()
        assert torch.equal(got, want), (scale, int((got != want).sum()))


def test_e4m3_codes_are_of_the_bf16_forms_quotient():
    """A weight without a rotation, on rows whose norm is 1: FP32 results of 24 significant bits.  Their
    codes equal those of the quotient in FP32, for scales of every kind of significand."""
    from paged_top_sparse_gb300 import binding as B

    T, D = 64, 128
    rng = np.random.default_rng(9)
    plan, ws, pos, _ = _plan([T], [0], 4, 2, D)
    # elements of +-1 have the mean square 1: with eps 0 the result is +-w, bit for bit, if 1 / sqrt(1)
    # is 1
    q = torch.from_numpy(np.where(rng.random((T, 4, D)) < 0.5, -1.0, 1.0).astype(np.float32)).to(DEV).bfloat16()
    out = torch.zeros((T, 4, D), dtype=torch.uint8, device=DEV)
    ulp = 2.0 ** -23
    for scale in (1 + ulp, 1.125 + ulp, 1.375 - 2 * ulp, 1.75 + 4 * ulp, 2 - ulp, 1.5, 0.0131, 4.5 / 448):
        scale = np.float32(scale)
        # weights within a few units of scale x border, and anything
        m = (np.arange(16, 32) + 0.5) / 16 * np.exp2(rng.integers(-6, 8, (4, 16)))
        near = (m.ravel()[:64].astype(np.float32) * scale)
        near = (near.view(np.int32) + rng.integers(-2, 3, 64)).astype(np.int32).view(np.float32)
        w = np.concatenate((near, (rng.standard_normal(64) * 200 * scale).astype(np.float32)))
        B.sps_qk_norm_rope(plan, q, None, torch.from_numpy(w).to(DEV), None, 0.0, None, out, float(scale),
                           None, ws)
        torch.cuda.synchronize()
        quot = (_f64(q).astype(np.float32) * w / scale).clip(-448, 448)
        want = torch.from_numpy(quot).to(torch.float8_e4m3fn).view(torch.uint8)
        assert torch.equal(out.cpu(), want), (scale, int((out.cpu() != want).sum()))


def _turns(bits):
    """2^bits / (2 pi) as an integer, from pi = 16 atan(1/5) - 4 atan(1/239) (Machin)."""
    one = 1 << (2 * bits)

    def atan_inv(n):
        total, term, k = 0, one // n, 0
        while term:
            total += (-1) ** k * (term // (2 * k + 1))
            term //= n * n
            k += 1
        return total

    pi = 16 * atan_inv(5) - 4 * atan_inv(239)
    return (1 << (3 * bits)) // (2 * pi)


def test_angles_of_large_frequencies_keep_the_stated_bound():
    """(|f| + 1) |position| 2^-64 + 2^-25 turns, against angles from whole numbers of 300 bits."""
    from paged_top_sparse_gb300 import binding as B

    bits, D, T = 300, 128, 64
    inv2pi = _turns(bits)
    assert abs(inv2pi / 2 ** bits - 0.5 / np.pi) < 1e-16
    rng = np.random.default_rng(77)
    f = np.exp(rng.uniform(-3, np.log(1e9), D // 2)).astype(np.float32)
    f[:6] = [1.0, 3.5, 1e6, 2.0 ** 20, 2.0 ** 24 + 2, 1.5e9]
    f[10:20] *= -1
    p = rng.integers(-(1 << 31), 1 << 31, T).astype(np.int32)
    p[:5] = [0, 1, -1, -(1 << 31), (1 << 31) - 1]
    p[20:40] = rng.integers(-5000, 5000, 20)
    plan, ws, _, _ = _plan([T], [0], 1, 1, D)
    # pairs (1, 0): the results are the cosine and the sine themselves
    q = torch.zeros((T, 1, D), device=DEV)
    q[..., 0::2] = 1.0
    out = torch.empty((T, 1, D), dtype=torch.bfloat16, device=DEV)
    B.sps_qk_norm_rope(plan, q.bfloat16(), None, None, None, EPS,
                       B.Rope(torch.from_numpy(f).to(DEV), positions=torch.from_numpy(p).to(DEV),
                              interleaved=True), out, 1.0, None, ws)
    torch.cuda.synchronize()
    got = _f64(out)[:, 0]
    mask = (1 << bits) - 1
    for j in range(D // 2):
        m, e = np.frexp(np.float64(f[j]))
        mi, e = int(m * 2 ** 24), int(e) - 24  # f = mi 2^e, whole
        for t in range(T):
            x = int(p[t]) * mi * inv2pi
            x = (x << e if e >= 0 else x >> -e) & mask
            a = 2 * np.pi * (x / 2 ** bits)
            off = 2 * np.pi * ((abs(float(f[j])) + 1) * abs(int(p[t])) * 2.0 ** -64 + 2.0 ** -25)
            for d, ref in ((0, np.cos(a)), (1, np.sin(a))):
                assert abs(got[t, 2 * j + d] - ref) <= BF16_HALF * abs(ref) + NOISE + off, (j, t, d)
