"""Full attention of rows that have no finite answer: a query row that holds a NaN gives NaN, whatever blocks
and warps its pages were cut over, and no other row notices."""
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


SHAPES = [([1, 1, 2], [9000, 60, 300], 16, 2, 128), ([1, 2], [700, 3000], 8, 1, 64),
          ([150, 1, 3], [700, 40, 5000], 8, 2, 128), ([20, 9], [4000, 0], 4, 2, 64),
          ([400], [3000], 32, 2, 128)]


def _rows(c):
    """A few (token, head) in different tiles, and their mask."""
    hit = torch.zeros((c.T, c.H), dtype=torch.bool, device=DEV)
    for i, t in enumerate(sorted({0, c.T // 2, c.T - 1})):
        hit[t, (3 * i + 1) % c.H] = True
    return hit


def _check_e4m3(q_lens, ctx, H, G, D, q, value):
    from tests.test_gpu_attention_e4m3 import Case

    c = Case(71, q_lens, ctx, H, G, D, q)
    out, lse, mag, top, keys = c.reference()
    hit = _rows(c)
    c.q[..., 5][hit] = torch.tensor(float(value), device=DEV).to(c.q.dtype)
    c.run()
    torch.cuda.synchronize()
    assert c.B.sps_read_device_status(c.plan, c.ws) == 0
    assert bool(torch.isnan(c.out[hit].float()).all()) and bool(torch.isnan(c.lse[hit]).all())
    # P to FP16, the output to BF16, the FP32 chain in front of P below 2^-14; subnormal P
    tol = (2.0 ** -11 + 2.0 ** -14) * mag + 2.0 ** -8 * out.abs() + (keys * 2.0 ** -32 * top)[..., None]
    assert bool(((c.out.double() - out).abs() <= tol)[~hit].all())
    assert bool(((c.lse.double() - lse).abs() <= 2.0 ** -13 + keys * 2.0 ** -26 + lse.abs() * 2.0 ** -22)[~hit].all())


@pytest.mark.parametrize("q", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_lens,ctx,H,G,D", SHAPES)
def test_rows_over_an_e4m3_cache(q_lens, ctx, H, G, D, q):
    _check_e4m3(q_lens, ctx, H, G, D, q, "nan")


@pytest.mark.parametrize("value", ["inf", "-inf"])
@pytest.mark.parametrize("q_lens,ctx,H,G,D", SHAPES)
def test_an_infinite_query_over_an_e4m3_cache(q_lens, ctx, H, G, D, value):
    """Its scores are infinite or NaN: so is their softmax."""
    _check_e4m3(q_lens, ctx, H, G, D, "bf16", value)


@pytest.mark.parametrize("kv", ["bf16", "nvfp4"])
@pytest.mark.parametrize("q_lens,ctx,H,G,D", SHAPES)
def test_rows_over_the_other_caches(q_lens, ctx, H, G, D, kv):
    from paged_top_sparse_gb300 import binding as B

    g = torch.Generator(device=DEV)
    g.manual_seed(H + D)
    quant, T = kv == "nvfp4", sum(q_lens)
    pages = [(n + x - 1) // 128 + 1 for n, x in zip(q_lens, ctx)]
    NP, at = sum(pages), 0
    pt = torch.zeros((len(q_lens), max(pages)), dtype=torch.int32)
    for b, n in enumerate(pages):
        pt[b, :n] = torch.arange(at, at + n)
        at += n
    pt = pt.to(DEV)
    plan = B.Plan(q_lens, ctx, H, G, D, 1, pt.shape[1], NP, q_dtype="e4m3" if quant else "bf16", kv_dtype=kv)
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device=DEV)
    B.sps_plan_upload(plan, ws)
    scratch = torch.empty(B.paged_attention_scratch(plan), dtype=torch.uint8, device=DEV)
    randn = lambda *s: torch.randn(s, generator=g, device=DEV)
    if quant:
        kc, vc = (torch.randint(0, 256, (NP, G, 128, D // 2), generator=g, device=DEV, dtype=torch.uint8) for _ in "kv")
        ks, vs = (torch.full((NP, G, 128, D // 16), 0x38, dtype=torch.uint8, device=DEV) for _ in "kv")
    else:
        kc, vc, ks, vs = randn(NP, G, 128, D).bfloat16(), randn(NP, G, 128, D).bfloat16(), None, None
    q = randn(T, H, D).to(torch.float8_e4m3fn if quant else torch.bfloat16)
    outs = []
    hit = torch.zeros((T, H), dtype=torch.bool, device=DEV)
    for spoil in (False, True):
        if spoil:
            for i, t in enumerate(sorted({0, T // 2, T - 1})):
                hit[t, (3 * i + 1) % H] = True
            q[..., 5][hit] = torch.tensor(float("nan"), device=DEV).to(q.dtype)
        out, lse = torch.empty((T, H, D), dtype=torch.bfloat16, device=DEV), torch.empty((T, H), device=DEV)
        B.paged_attention_fwd(plan, q, 1.0, kc, vc, ks, vs, pt, out, lse, scratch, ws)
        torch.cuda.synchronize()
        assert B.sps_read_device_status(plan, ws) == 0
        outs.append((out, lse))
    assert bool(torch.isnan(outs[1][0][hit].float()).all()) and bool(torch.isnan(outs[1][1][hit]).all())
    # the other rows: P in 16 bits (2^-9 of the weighted values, which are below the largest), and the
    # output, twice; a reference raised for a neighbour's sake changes no more than that
    big = 4.0 * 6 if quant else float(vc.float().abs().amax())
    tol = 2 * (2.0 ** -9 * big + 2.0 ** -8 * outs[0][0].float().abs())
    assert bool(((outs[1][0].float() - outs[0][0].float()).abs() <= tol)[~hit].all())
    assert bool(((outs[1][1] - outs[0][1]).abs() <= 2.0 ** -10 + outs[0][1].abs() * 2.0 ** -20)[~hit].all())
