"""Cases and plain forms of the operators around a paged K/V cache: the norm and rotation of
queries and keys (``sps_qk_norm_rope``), the append with that rotation
(``sps_kv_append_rope``) and full attention of a batch of new tokens over the cache
(``paged_attention_fwd``).

``run`` computes an operator in elementary torch operations, or, where ``own`` is true, with
the library's calls.  Cases are dicts of plain values; ``op`` names the operator and ``lens``
seeds the lengths of the batch's requests.
"""
import math
import random

import torch

own = False
DEV = "cuda"
PAGE = 128
EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases

def _qk(name, batch, q, ctx, heads, kv_heads, dim, rot, axes=1, interleaved=False, out="bf16",
        lens=1):
    return dict(name=name, op="qk", batch=batch, q_lo=q[0], q_hi=q[1], c_lo=ctx[0], c_hi=ctx[1],
                heads=heads, kv_heads=kv_heads, dim=dim, rot=rot, axes=axes,
                interleaved=interleaved, out=out, lens=lens)


def _append(name, batch, q, ctx, kv_heads, dim, rot, cache="bf16", interleaved=False, norm=True,
            lens=1):
    return dict(name=name, op="append", batch=batch, q_lo=q[0], q_hi=q[1], c_lo=ctx[0],
                c_hi=ctx[1], heads=kv_heads, kv_heads=kv_heads, dim=dim, rot=rot, axes=1,
                interleaved=interleaved, cache=cache, norm=norm, lens=lens)


def _attn(name, batch, q, ctx, heads, kv_heads, dim, cache="bf16", lens=1):
    return dict(name=name, op="attn", batch=batch, q_lo=q[0], q_hi=q[1], c_lo=ctx[0], c_hi=ctx[1],
                heads=heads, kv_heads=kv_heads, dim=dim, cache=cache, lens=lens)


def listed():
    return [
        # one decode step of 64 requests: latency of the smallest launch
        _qk("qk_decode64", 64, (1, 1), (24576, 40960), 32, 2, 128, 128),
        # an 8K prompt, the headline prefill's shape
        _qk("qk_prefill8k", 1, (8192, 8192), (0, 0), 32, 2, 128, 128),
        # an image-and-text prompt: time/height/width positions, half the head rotated, E4M3 query
        _qk("qk_axes_e4m3", 3, (1001, 2777), (0, 900), 28, 4, 128, 64, axes=3, out="e4m3"),
        # the append of that decode step
        _append("append_decode64", 64, (1, 1), (24576, 40960), 2, 128, 128),
        # chunked prefill, 8 x 512 new tokens, into an NVFP4 cache (read back as values)
        _append("append_chunk_nvfp4", 8, (512, 512), (24576, 40960), 2, 128, 128, cache="nvfp4"),
        # a small ragged batch with one-token requests among it: latency of the attention
        _attn("attn_ragged_d64", 5, (1, 300), (0, 1000), 4, 2, 64),
        # one user at the end of a 128K context
        _attn("attn_decode1_128k", 1, (1, 1), (131071, 131071), 32, 2, 128),
        # a decode step of 64 requests at ~32K each
        _attn("attn_decode64", 64, (1, 1), (24576, 40960), 32, 2, 128),
        # the same from an NVFP4 cache with an E4M3 query
        _attn("attn_decode64_nvfp4", 64, (1, 1), (24576, 40960), 32, 2, 128, cache="nvfp4"),
        # an 8K prompt in full attention, the headline prefill's shape
        _attn("attn_prefill8k", 1, (8192, 8192), (0, 0), 32, 2, 128),
        # chunked prefill, 8 x 512 new tokens over ~32K cached
        _attn("attn_chunk32k", 8, (512, 512), (24576, 40960), 32, 2, 128),
        # chunked prefill over a quantised cache
        _attn("attn_chunk_nvfp4", 4, (200, 700), (2000, 9000), 32, 4, 128, cache="nvfp4"),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk", "append", "attn", "attn"])
    heads, kv_heads = rng.choice([(32, 2), (4, 2), (28, 4), (8, 8), (32, 8), (6, 1), (16, 4)])
    dim = rng.choice([64, 128, 128])
    rot = rng.choice([r for r in (32, 64, 96, 128) if r <= dim])
    lens = rng.randrange(1 << 20)
    if op == "attn":
        cache = rng.choice(["bf16", "bf16", "nvfp4"])
        batch = _logint(rng, 1, 64)
        q_hi = 1 if rng.random() < 0.4 else _logint(rng, 2, 4096)
        c_hi = _logint(rng, 16, 65536)
        # at most the work of the largest listed cases
        while batch * heads * q_hi * (c_hi + q_hi) > 5.0e9 or \
                batch * kv_heads * dim * (c_hi + q_hi) > 5.0e8:
            if c_hi > 4 * q_hi and c_hi > 64:
                c_hi //= 2
            elif q_hi > 64:
                q_hi //= 2
            else:
                batch = max(1, batch // 2)
        return _attn("attn", batch, (max(1, q_hi // 2), q_hi),
                     (0 if rng.random() < 0.3 else c_hi // 2, c_hi), heads, kv_heads, dim, cache,
                     lens)
    batch = _logint(rng, 1, 32)
    q_hi = 1 if rng.random() < 0.3 else _logint(rng, 2, 8192 // batch)
    c_hi = _logint(rng, 16, 65536)
    q, ctx = (max(1, q_hi // 2), q_hi), (0 if rng.random() < 0.3 else c_hi // 2, c_hi)
    if op == "qk":
        return _qk("qk", batch, q, ctx, heads, kv_heads, dim, rot, rng.choice([1, 1, 2, 3]),
                   rng.random() < 0.5, rng.choice(["bf16", "bf16", "e4m3"]), lens)
    return _append("append", batch, q, ctx, kv_heads, dim, rot, rng.choice(["bf16", "nvfp4"]),
                   rng.random() < 0.5, rng.random() < 0.7, lens)


def _lens(case):
    r = random.Random(case["lens"])
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["batch"])]
    c = [r.randint(case["c_lo"], case["c_hi"]) for _ in range(case["batch"])]
    return q, c


def work(case):
    q, c = _lens(case)
    T, G, D, H = sum(q), case["kv_heads"], case["dim"], case["heads"]
    if case["op"] == "qk":
        bytes_ = T * (H + G) * D * 2 + T * G * D * 2 + T * H * D * (2 if case["out"] == "bf16" else 1)
        return {"bytes": bytes_, "flops": 8 * T * (H + G) * D}
    per_el = 2 if case["cache"] == "bf16" else 9 / 16
    if case["op"] == "append":
        return {"bytes": 2 * T * G * D * (2 + per_el), "flops": 8 * T * G * D}
    kv = sum(a + b for a, b in zip(q, c))
    seen = sum(a * b + a * (a + 1) // 2 for a, b in zip(q, c))
    return {"bytes": 2 * kv * G * D * per_el + T * H * D * (2 if case["cache"] == "bf16" else 1)
            + T * H * (2 * D + 4), "flops": 4 * D * H * seen}


# ------------------------------------------------------------------ inputs

def _e2m1_code(y):
    """Nearest E2M1 magnitude code of |y| (ties to the even code), 6 the largest."""
    up = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=y.dtype, device=y.device)
    a = y.abs()
    # 0.75, 1.75 and 3.5 lie between an odd code below and an even one above: they round up
    hi = torch.bucketize(a, up)               # counts thresholds below a
    hi_tie = torch.bucketize(a, up, right=True)  # counts thresholds at or below a
    return torch.where(hi_tie % 2 == 0, hi_tie, hi)


def _nvfp4(x):
    """x [..., D] -> packed codes [..., D/2] and E4M3 scale bytes [..., D/16]."""
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    sc = (b.abs().amax(-1).float() / 6).clamp(max=448).to(torch.float8_e4m3fn)
    s = sc.to(x.dtype)[..., None]
    y = torch.where(s > 0, b / torch.where(s > 0, s, 1), 0)
    code = _e2m1_code(y) | (torch.signbit(y).long() << 3)
    code = torch.where(s > 0, code, 0).to(torch.uint8).reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), sc.view(torch.uint8)


def _values(codes, scales):
    """What packed codes and scale bytes stand for, FP32 [..., D]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = torch.stack((table[(codes & 15).long()], table[(codes >> 4).long()]), -1).flatten(-2)
    s = scales.view(torch.float8_e4m3fn).float()
    return (v.view(*v.shape[:-1], -1, 16) * s[..., None]).flatten(-2)


def _inv_freq(rot):
    return (1e6 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)).float().to(DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 2 + 1)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    q_lens, ctx = _lens(case)
    B, T, H, G, D = case["batch"], sum(q_lens), case["heads"], case["kv_heads"], case["dim"]
    req = torch.tensor([b for b in range(B) for _ in range(q_lens[b])], device=DEV)
    idx = torch.tensor([i for b in range(B) for i in range(q_lens[b])], device=DEV)
    pos = torch.tensor(ctx, device=DEV)[req] + idx
    npages = [(c + q - 1) // PAGE + 1 for q, c in zip(q_lens, ctx)]
    s = dict(case=case, req=req, idx=idx, pos=pos, T=T, q_max=max(q_lens))
    op = case["op"]
    if op in ("qk", "append"):
        qkv = randn(T, H + 2 * G, D).bfloat16()  # the fused projection's output
        s |= dict(q=qkv[:, :H], k=qkv[:, H:H + G], v=qkv[:, H + G:], inv_freq=_inv_freq(case["rot"]),
                  qw=1 + 0.2 * randn(D), kw=1 + 0.2 * randn(D), axis_pos=None, pair_axis=None)
        if op == "append" and not case["norm"]:
            s["kw"] = None
        s["table_pos"] = pos[None]
        if case["axes"] > 1:  # positions of their own for each axis, the pairs dealt out in runs
            p = torch.stack([pos] + [torch.randint(0, 64, (T,), generator=g, device=DEV)
                                     for _ in range(case["axes"] - 1)])
            s["table_pos"] = p
            s["axis_pos"] = p.int().contiguous()
            n = case["rot"] // 2
            s["pair_axis"] = [j * case["axes"] // n for j in range(n)]
        ax = s["pair_axis"] or [0] * (case["rot"] // 2)
        s["ax"] = torch.tensor(ax, device=DEV)
    if op == "qk":
        s["q_scale"] = 0.02
        s["q_out"] = torch.empty((T, H, D), device=DEV,
                                 dtype=torch.bfloat16 if case["out"] == "bf16" else torch.uint8)
        s["k_out"] = torch.empty((T, G, D), device=DEV, dtype=torch.bfloat16)
        num_phys = max(npages)
    if op == "append":
        # cached pages before the new tokens belong to a shared prefix; each request owns the rest
        first = [c // PAGE for c in ctx]
        n_shared = max(first)
        own_n = [n - f for n, f in zip(npages, first)]
        num_phys = n_shared + sum(own_n)
        pt, at = torch.zeros((B, max(npages)), dtype=torch.int32), n_shared
        for b in range(B):
            pt[b, :first[b]] = torch.arange(first[b], dtype=torch.int32)
            pt[b, first[b]:npages[b]] = torch.arange(at, at + own_n[b], dtype=torch.int32)
            at += own_n[b]
        s |= dict(page_table=pt.to(DEV), n_shared=n_shared)
    if op == "attn":
        num_phys = sum(npages)
        perm = torch.randperm(num_phys, generator=g, device=DEV).int().cpu()
        pt, at = torch.zeros((B, max(npages)), dtype=torch.int32), 0
        for b in range(B):
            pt[b, :npages[b]] = perm[at:at + npages[b]]
            at += npages[b]
        s["page_table"] = pt.to(DEV)
        s["q_scale"] = 1.0
        if case["cache"] == "bf16":
            s["q"] = randn(T, H, D).bfloat16()
        else:
            s["q_scale"] = 4.5 / 448
            s["q"] = (randn(T, H, D) / s["q_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn)
        s["out"] = torch.empty((T, H, D), device=DEV, dtype=torch.bfloat16)
        s["out_lse"] = torch.empty((T, H), device=DEV)
    if op in ("append", "attn"):
        for n in ("kc", "vc"):
            x = randn(num_phys, G, PAGE, D)
            if case["cache"] == "bf16":
                s[n], s[n + "_s"] = x.bfloat16(), None
            else:
                s[n], s[n + "_s"] = _nvfp4(x)
            del x
    if own:
        from paged_top_sparse_gb300 import binding as B_
        quant = case.get("cache") == "nvfp4"
        plan = B_.Plan(q_lens, ctx, H, G, D, 1, max(npages), num_phys,
                       q_dtype="e4m3" if quant else "bf16", kv_dtype="nvfp4" if quant else "bf16")
        s["plan"] = plan
        s["ws"] = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device=DEV)
        B_.sps_plan_upload(plan, s["ws"])
        if op == "attn":
            s["scratch"] = torch.empty(B_.paged_attention_scratch(plan), dtype=torch.uint8,
                                       device=DEV)
        else:
            s["rope"] = B_.Rope(s["inv_freq"], positions=s["axis_pos"], pair_axis=s["pair_axis"],
                                interleaved=case["interleaved"])
        if op == "append" and quant:
            n = s["n_shared"]
            s["values"] = [torch.empty((num_phys - n, G, PAGE, D), dtype=torch.float16, device=DEV)
                           for _ in range(2)]
    return s


# ------------------------------------------------------------------ plain forms

def _norm_rope(s, x, w, to64=False):
    """Norm over the head dim, weight, then the rotation; FP32 (FP64 in front of a quantiser)."""
    dt = torch.float64 if to64 else torch.float32
    x = x.to(dt)
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w.to(dt)
    # angles of far positions need 64 bits
    ang = s["table_pos"][s["ax"]].T.double() * s["inv_freq"].double()
    cos, sin = ang.cos().to(dt)[:, None], ang.sin().to(dt)[:, None]
    rot = s["case"]["rot"]
    r, rest = x[..., :rot], x[..., rot:]
    if s["case"]["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((r, rest), -1)


def _plain_qk(s):
    e4m3 = s["case"]["out"] == "e4m3"
    q = _norm_rope(s, s["q"], s["qw"], e4m3)
    if e4m3:
        q = (q / s["q_scale"]).clamp(-448, 448).float().to(torch.float8_e4m3fn)
    else:
        q = q.bfloat16()
    return {"q": q, "k": _norm_rope(s, s["k"], s["kw"]).bfloat16()}


def _plain_append(s):
    quant = s["case"]["cache"] == "nvfp4"
    page = s["page_table"][s["req"], s["pos"] // PAGE].long()
    slot = s["pos"] % PAGE
    k = _norm_rope(s, s["k"], s["kw"], quant)
    if not quant:
        s["kc"][page, :, slot] = k.bfloat16()
        s["vc"][page, :, slot] = s["v"]
        return {"k": s["kc"], "v": s["vc"]}
    n = s["n_shared"]
    s["kc"][page, :, slot], s["kc_s"][page, :, slot] = _nvfp4(k)
    s["vc"][page, :, slot], s["vc_s"][page, :, slot] = _nvfp4(s["v"].float())
    return {"k": _values(s["kc"][n:], s["kc_s"][n:]).half(),
            "v": _values(s["vc"][n:], s["vc_s"][n:]).half()}


def _gathered(s, n):
    """The cache through the page table, FP32 [batch, kv head, key, D]."""
    c = s[n][s["page_table"].long()]
    c = c.float() if s[n + "_s"] is None else _values(c, s[n + "_s"][s["page_table"].long()])
    return c.transpose(1, 2).flatten(2, 3)


def _plain_attn(s):
    c = s["case"]
    B, H, G, D, Q = c["batch"], c["heads"], c["kv_heads"], c["dim"], s["q_max"]
    q = torch.zeros((B, Q, H, D), device=DEV)
    q[s["req"], s["idx"]] = s["q"].float() * (s["q_scale"] * D ** -0.5)
    pos = torch.zeros((B, Q), dtype=torch.long, device=DEV)
    pos[s["req"], s["idx"]] = s["pos"]
    q = q.view(B, Q, G, H // G, D).permute(0, 2, 3, 1, 4).reshape(B, G, -1, D)
    k = _gathered(s, "kc")
    sc = torch.matmul(q, k.transpose(-1, -2)).view(B, G, H // G, Q, -1)
    del k
    hidden = torch.arange(sc.shape[-1], device=DEV) > pos[..., None]
    sc.masked_fill_(hidden[:, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, G, -1, p.shape[-1]), _gathered(s, "vc")).view(B, G, H // G, Q, D) / l
    lse = (m + l.log()).view(B, H, Q)
    return {"out": o.view(B, H, Q, D).transpose(1, 2)[s["req"], s["idx"]].bfloat16(),
            "lse": lse.transpose(1, 2)[s["req"], s["idx"]].contiguous()}


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"qk": _plain_qk, "append": _plain_append, "attn": _plain_attn}[op](s)
    from paged_top_sparse_gb300 import binding as B
    if op == "qk":
        B.sps_qk_norm_rope(s["plan"], s["q"], s["k"], s["qw"], s["kw"], EPS, s["rope"],
                           s["q_out"], s["q_scale"], s["k_out"], s["ws"])
        q = s["q_out"] if s["case"]["out"] == "bf16" else s["q_out"].view(torch.float8_e4m3fn)
        return {"q": q, "k": s["k_out"]}
    if op == "append":
        B.sps_kv_append_rope(s["plan"], s["k"], s["v"], s["kw"], EPS, s["rope"], s["page_table"],
                             s["kc"], s["vc"], s["kc_s"], s["vc_s"], s["ws"])
        if s["case"]["cache"] == "bf16":
            return {"k": s["kc"], "v": s["vc"]}
        n = s["n_shared"]
        for c, out in zip(("kc", "vc"), s["values"]):
            B.sps_dequantize("nvfp4", s[c][n:], s[c + "_s"][n:], out.numel(), out)
        return {"k": s["values"][0], "v": s["values"][1]}
    B.paged_attention_fwd(s["plan"], s["q"], s["q_scale"], s["kc"], s["vc"], s["kc_s"], s["vc_s"],
                          s["page_table"], s["out"], s["out_lse"], s["scratch"], s["ws"])
    return {"out": s["out"], "lse": s["out_lse"]}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_rows(s, x, w):
    """Rows [T, heads, D] in 64 bits, dimension by dimension pair as complex numbers."""
    x = x.double()
    if w is not None:
        x = x * torch.rsqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
    c, h = s["case"], s["case"]["rot"] // 2
    pairs = torch.arange(h, device=DEV)
    first = 2 * pairs if c["interleaved"] else pairs
    second = first + (1 if c["interleaved"] else h)
    turn = torch.empty((x.shape[0], h), dtype=torch.float64, device=DEV)
    for j in range(h):
        axis = 0 if s["pair_axis"] is None else s["pair_axis"][j]
        turn[:, j] = s["table_pos"][axis].double() * s["inv_freq"][j].double()
    z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.ones_like(turn), turn)[:, None]
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_quantised(x):
    """The NVFP4 value of each element of x [..., D] (no rounding before it), by trying every
    magnitude."""
    b = x.unflatten(-1, (-1, 16))
    s = (b.abs().amax(-1) / 6).clamp(max=448).float().to(torch.float8_e4m3fn).double()[..., None]
    mags = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    far = (b.abs()[..., None] - mags * s[..., None]).abs()
    near = far == far.amin(-1, keepdim=True)
    even = near & (torch.arange(8, device=DEV) % 2 == 0)
    pick = torch.where(even.any(-1), even.int().argmax(-1), near.int().argmax(-1))
    return (mags[pick] * s * torch.sign(b)).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "qk":
        q = _exact_rows(s, s["q"], s["qw"])
        if case["out"] == "e4m3":  # the value that the codes are rounded from
            q = q / s["q_scale"]
        return {"q": q, "k": _exact_rows(s, s["k"], s["kw"])}
    q_lens, ctx = _lens(case)
    G, D, H = case["kv_heads"], case["dim"], case["heads"]
    if case["op"] == "append":
        quant = case["cache"] == "nvfp4"
        k, v = _exact_rows(s, s["k"], s["kw"]), s["v"].double()
        n = s["n_shared"] if quant else 0
        got = {}
        for name, new in (("kc", k), ("vc", v)):
            cache = _values(s[name][n:], s[name + "_s"][n:]).double() if quant else s[name].double()
            if quant and name == "kc":  # rotated keys next to a code's border may go either way
                got["k"] = None
                continue
            new = _exact_quantised(new) if quant else new
            t = 0
            for b in range(case["batch"]):
                for i0 in range(ctx[b] // PAGE, (ctx[b] + q_lens[b] - 1) // PAGE + 1):
                    lo, hi = max(ctx[b], i0 * PAGE), min(ctx[b] + q_lens[b], (i0 + 1) * PAGE)
                    rows = new[t + lo - ctx[b]:t + hi - ctx[b]].transpose(0, 1)
                    cache[int(s["page_table"][b, i0]) - n, :, lo - i0 * PAGE:hi - i0 * PAGE] = rows
                t += q_lens[b]
            got[name[0]] = cache
        return got
    out = torch.empty((s["T"], H, D), dtype=torch.float64, device=DEV)
    lse = torch.empty((s["T"], H), dtype=torch.float64, device=DEV)
    t = 0
    for b in range(case["batch"]):
        n = ctx[b] + q_lens[b]
        pages = s["page_table"][b, :(n - 1) // PAGE + 1].long()
        keys = torch.arange(n, device=DEV)
        for g in range(G):
            kv = []
            for c in ("kc", "vc"):
                x = s[c][pages, g]
                x = x.double() if s[c + "_s"] is None else _values(x, s[c + "_s"][pages, g]).double()
                kv.append(x.reshape(-1, D)[:n])
            for i in range(0, q_lens[b], 1024):
                j = min(q_lens[b], i + 1024)
                rows = s["q"][t + i:t + j, g * (H // G):(g + 1) * (H // G)].double() * s["q_scale"]
                sc = torch.einsum("thd,kd->thk", rows, kv[0]) / math.sqrt(D)
                seen = keys[None] <= ctx[b] + torch.arange(i, j, device=DEV)[:, None]
                sc = torch.where(seen[:, None], sc, -math.inf)
                z = torch.logsumexp(sc, -1)
                out[t + i:t + j, g * (H // G):(g + 1) * (H // G)] = \
                    torch.einsum("thk,kd->thd", torch.exp(sc - z[..., None]), kv[1])
                lse[t + i:t + j, g * (H // G):(g + 1) * (H // G)] = z
        t += q_lens[b]
    return {"out": out, "lse": lse}
