"""Cases and plain forms of the operators around a paged K/V cache held in 8 bits (E4M3 codes, one
FP32 scale for each page and KV head): the append of new tokens (``sps_kv_append_rope``), full
attention (``paged_attention_fwd``) and the sparse forward with its combine
(``sparse_prefill_fwd_f16``, ``partial_combine_f16``) over that cache, and the page tables and slot
maps built on the GPU from request lengths (``sps_page_tables``).

``run`` computes an operator in elementary torch operations, or, where ``own`` is true, with the
library's calls.  Cases are dicts of plain values; ``op`` names the operator and ``lens`` seeds the
lengths of the batch's requests.
"""
import math
import random

import torch

own = False
DEV = "cuda"
PAGE = 128
EPS = 1e-6
E4M3_MAX = 448.0
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases

def _append(name, batch, q, ctx, kv_heads, dim, rot, interleaved=False, norm=True, lens=1):
    return dict(name=name, op="append", batch=batch, q_lo=q[0], q_hi=q[1], c_lo=ctx[0],
                c_hi=ctx[1], heads=kv_heads, kv_heads=kv_heads, dim=dim, rot=rot,
                interleaved=interleaved, norm=norm, lens=lens)


def _attn(name, batch, q, ctx, heads, kv_heads, dim, query="bf16", lens=1):
    return dict(name=name, op="attn", batch=batch, q_lo=q[0], q_hi=q[1], c_lo=ctx[0], c_hi=ctx[1],
                heads=heads, kv_heads=kv_heads, dim=dim, query=query, lens=lens)


def _sparse(name, batch, q, ctx, heads, kv_heads, dim, top_k, query="bf16", lens=1):
    return dict(name=name, op="sparse", batch=batch, q_lo=q[0], q_hi=q[1], c_lo=ctx[0],
                c_hi=ctx[1], heads=heads, kv_heads=kv_heads, dim=dim, top_k=top_k, query=query,
                lens=lens)


def _tables(name, batch, q, ctx, lens=1):
    return dict(name=name, op="tables", batch=batch, q_lo=q[0], q_hi=q[1], c_lo=ctx[0],
                c_hi=ctx[1], lens=lens)


def listed():
    return [
        # the append of a decode step of 64 requests: latency of the smallest launch
        _append("append_decode64", 64, (1, 1), (24576, 40960), 2, 128, 128),
        # chunked prefill, 8 x 512 new tokens, pages that begin and end inside the chunks
        _append("append_chunk", 8, (512, 512), (24576, 40960), 2, 128, 128),
        # ragged prompts of a model with small heads, adjacent pairs, no norm
        _append("append_prompt_d64", 3, (1001, 2777), (0, 900), 8, 64, 64, interleaved=True,
                norm=False),
        # a small ragged batch with one-token requests among it: latency of the attention
        _attn("attn_ragged_d64", 5, (1, 300), (0, 1000), 4, 2, 64),
        # one user at the end of a 128K context
        _attn("attn_decode1_128k", 1, (1, 1), (131071, 131071), 32, 2, 128),
        # a decode step of 64 requests at ~32K each
        _attn("attn_decode64", 64, (1, 1), (24576, 40960), 32, 2, 128),
        # an 8K prompt in full attention, the headline prefill's shape
        _attn("attn_prefill8k", 1, (8192, 8192), (0, 0), 32, 2, 128),
        # chunked prefill, 8 x 512 new tokens over ~32K cached, E4M3 queries
        _attn("attn_chunk32k_e4m3", 8, (512, 512), (24576, 40960), 32, 2, 128, query="e4m3"),
        # the headline prefill itself: an 8K prompt, 16 pages a row
        _sparse("sparse_prefill8k", 1, (8192, 8192), (0, 0), 32, 2, 128, 16),
        # ragged chunks of E4M3 queries over contexts of a few thousand tokens
        _sparse("sparse_chunk_e4m3", 4, (200, 700), (2000, 9000), 32, 4, 128, 16, query="e4m3"),
        # the tables of that decode step: latency
        _tables("tables_decode64", 64, (1, 1), (24576, 40960)),
        # the tables of a large mixed step: 256 requests of up to 512 new tokens
        _tables("tables_chunk256", 256, (1, 512), (0, 40960)),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "sparse", "tables"])
    heads, kv_heads = rng.choice([(32, 2), (4, 2), (28, 4), (8, 8), (32, 8), (6, 1), (16, 4)])
    dim = rng.choice([64, 128, 128])
    rot = rng.choice([r for r in (32, 64, 96, 128) if r <= dim])
    query = rng.choice(["bf16", "bf16", "e4m3"])
    lens = rng.randrange(1 << 20)
    if op == "tables":
        batch = _logint(rng, 1, 256)
        q_hi = 1 if rng.random() < 0.3 else _logint(rng, 2, min(8192, 65536 // batch))
        c_hi = _logint(rng, 16, 65536)
        return _tables("tables", batch, (max(1, q_hi // 2), q_hi),
                       (0 if rng.random() < 0.5 else c_hi // 2, c_hi), lens)
    if op == "append":
        batch = _logint(rng, 1, 32)
        q_hi = 1 if rng.random() < 0.3 else _logint(rng, 2, 8192 // batch)
        c_hi = _logint(rng, 16, 65536)
        return _append("append", batch, (max(1, q_hi // 2), q_hi),
                       (0 if rng.random() < 0.3 else c_hi // 2, c_hi), kv_heads, dim, rot,
                       rng.random() < 0.5, rng.random() < 0.7, lens)
    sparse = op == "sparse"
    batch = _logint(rng, 1, 8 if sparse else 64)
    q_hi = 1 if not sparse and rng.random() < 0.4 else _logint(rng, 2, 4096)
    c_hi = _logint(rng, 16, 16384 if sparse else 65536)
    # at most the work of the largest listed cases
    while batch * heads * q_hi * (c_hi + q_hi) > (2.0e9 if sparse else 5.0e9) or \
            batch * kv_heads * dim * (c_hi + q_hi) > 5.0e8:
        if c_hi > 4 * q_hi and c_hi > 64:
            c_hi //= 2
        elif q_hi > 64:
            q_hi //= 2
        else:
            batch = max(1, batch // 2)
    q, ctx = (max(1, q_hi // 2), q_hi), (0 if rng.random() < 0.3 else c_hi // 2, c_hi)
    if sparse:
        return _sparse("sparse", batch, q, ctx, heads, kv_heads, dim,
                       rng.choice([1, 3, 8, 16, 16, 24]), query, lens)
    return _attn("attn", batch, q, ctx, heads, kv_heads, dim, query, lens)


def _lens(case):
    r = random.Random(case["lens"])
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["batch"])]
    c = [r.randint(case["c_lo"], case["c_hi"]) for _ in range(case["batch"])]
    return q, c


def _pages(n):
    return -(-n // PAGE)


def work(case):
    q, c = _lens(case)
    T, B = sum(q), case["batch"]
    if case["op"] == "tables":
        new = sum(_pages(a + b) - _pages(b) for a, b in zip(q, c))
        return {"bytes": 8 * B + 4 * B + 8 * new + 4 * (B + 1) + 12 * T, "flops": 2 * T}
    G, D, H = case["kv_heads"], case["dim"], case["heads"]
    if case["op"] == "append":
        return {"bytes": 2 * T * G * D * 3, "flops": 8 * T * G * D}
    qo = T * H * D * (2 if case["query"] == "bf16" else 1) + T * H * (2 * D + 4)
    kv = sum(a + b for a, b in zip(q, c))
    if case["op"] == "attn":
        seen = sum(a * b + a * (a + 1) // 2 for a, b in zip(q, c))
    else:  # the pages a row keeps, of those it sees
        k = case["top_k"]
        seen = sum(PAGE * min(k, (b + i) // PAGE + 1) for a, b in zip(q, c) for i in range(a))
        qo += T * H * k * 4
    return {"bytes": 2 * kv * G * D + qo, "flops": 4 * D * H * seen}


# ------------------------------------------------------------------ inputs

def _pow2_scale(amax):
    """The smallest power of two s with amax / s <= 448, within 2^-40 .. 2^40."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1): 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(amax > 0, e, -40).clamp(-40, 40)
    return torch.ldexp(torch.ones_like(amax), e)


def _inv_freq(rot):
    return (1e6 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)).float().to(DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 2 + 1)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    q_lens, ctx = _lens(case)
    B, T = case["batch"], sum(q_lens)
    req = torch.tensor([b for b in range(B) for _ in range(q_lens[b])], device=DEV)
    idx = torch.tensor([i for b in range(B) for i in range(q_lens[b])], device=DEV)
    pos = torch.tensor(ctx, device=DEV)[req] + idx
    npages = [(c + q - 1) // PAGE + 1 for q, c in zip(q_lens, ctx)]
    s = dict(case=case, req=req, idx=idx, pos=pos, T=T, q_max=max(q_lens))
    op = case["op"]
    if op == "tables":
        have = [_pages(c) for c in ctx]
        held = sum(have)
        ids = torch.randperm(held + sum(npages), generator=g, device=DEV).int()
        pt, at = torch.full((B, max(npages) + 3), -1, dtype=torch.int32, device=DEV), 0
        for b in range(B):
            pt[b, :have[b]] = ids[at:at + have[b]]
            at += have[b]
        s |= dict(page_table=pt, free=ids[held:].clone(), first=torch.tensor([7, 0], dtype=torch.int32, device=DEV),
                  state=torch.zeros(2, dtype=torch.int32, device=DEV),
                  q_lens=torch.tensor(q_lens, dtype=torch.int32, device=DEV),
                  ctx=torch.tensor(ctx, dtype=torch.int32, device=DEV),
                  slots=torch.empty(T + 5, dtype=torch.int64, device=DEV),
                  positions=torch.empty(T + 5, dtype=torch.int32, device=DEV),
                  starts=torch.empty(B + 1, dtype=torch.int32, device=DEV),
                  status=torch.zeros(1, dtype=torch.int32, device=DEV))
        # seven pages of the list are gone; room enough is left
        s["free"] = torch.cat((s["free"], ids.new_full((7,), 0)))
        return s
    H, G, D = case["heads"], case["kv_heads"], case["dim"]
    if op == "append":
        qkv = randn(T, 3 * G, D).bfloat16()  # the fused projection's output
        s |= dict(k=qkv[:, G:2 * G], v=qkv[:, 2 * G:], inv_freq=_inv_freq(case["rot"]),
                  kw=1 + 0.2 * randn(D) if case["norm"] else None)
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
        # a request's touched pages: logical number, request, slots that hold earlier tokens
        touched = [(b, p) for b in range(B) for p in range(first[b], npages[b])]
        s["t_phys"] = torch.tensor([int(pt[b, p]) for b, p in touched], device=DEV)
        s["t_kept"] = torch.tensor([max(0, min(PAGE, ctx[b] - p * PAGE)) for b, p in touched], device=DEV)
    else:
        num_phys = sum(npages)
        perm = torch.randperm(num_phys, generator=g, device=DEV).int().cpu()
        pt, at = torch.zeros((B, max(npages)), dtype=torch.int32), 0
        for b in range(B):
            pt[b, :npages[b]] = perm[at:at + npages[b]]
            at += npages[b]
        s["page_table"] = pt.to(DEV)
        s["q_scale"] = 1.0
        if case["query"] == "bf16":
            s["q"] = randn(T, H, D).bfloat16()
        else:
            s["q_scale"] = 4.5 / 448
            s["q"] = (randn(T, H, D) / s["q_scale"]).clamp(-448, 448).to(F8)
        s["out"] = torch.empty((T, H, D), device=DEV, dtype=torch.bfloat16)
        s["out_lse"] = torch.empty((T, H), device=DEV)
    for n in ("kc", "vc"):  # pages of different magnitude, as tokens are
        x = randn(num_phys, G, PAGE, D)
        gain = torch.rand((num_phys, G), generator=g, device=DEV)
        x *= (0.5 + gain if n == "kc" else torch.exp2(4 * gain - 2))[:, :, None, None]
        s[n + "_s"] = _pow2_scale(x.abs().amax((2, 3)))
        s[n] = (x / s[n + "_s"][:, :, None, None]).to(F8).view(torch.uint8)
        del x
    if op == "sparse":
        # pages as a selection leaves them: the own one and others at random, ascending, -1 behind
        k, n = case["top_k"], max(npages)
        own_page = (pos // PAGE)[:, None, None]
        page = torch.arange(n, device=DEV)
        score = torch.rand((T, H, n), generator=g, device=DEV)
        score = torch.where(page == own_page, 2.0, score).masked_fill_(page > own_page, -1.0)
        val, at = score.topk(min(k, n), -1)
        at = torch.where(val < 0, n, at).sort(-1).values
        at = torch.where(at == n, -1, at).int()
        s["sel"] = torch.full((T, H, k), -1, dtype=torch.int32, device=DEV)
        s["sel"][..., :at.shape[-1]] = at
        del score
    if own:
        from paged_top_sparse_gb300 import binding as B_
        plan = B_.Plan(q_lens, ctx, H, G, D, case.get("top_k", 1), max(npages), num_phys,
                       q_dtype=case.get("query", "bf16"), kv_dtype="e4m3")
        s["plan"] = plan
        s["ws"] = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device=DEV)
        B_.sps_plan_upload(plan, s["ws"])
        if op == "attn":
            s["scratch"] = torch.empty(B_.paged_attention_scratch(plan), dtype=torch.uint8,
                                       device=DEV)
        elif op == "append":
            s["rope"] = B_.Rope(s["inv_freq"], interleaved=case["interleaved"])
        else:
            s["partial"] = torch.empty((case["top_k"], T * H, D), dtype=torch.float16, device=DEV)
            s["lse"] = torch.empty((case["top_k"], T * H), device=DEV)
    return s


# ------------------------------------------------------------------ plain forms

def _norm_rope(s, x, w):
    """Norm over the head dim, weight, then the rotation, FP64 in front of the quantiser."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w.double()
    ang = s["pos"].double()[:, None] * s["inv_freq"].double()
    cos, sin = ang.cos()[:, None], ang.sin()[:, None]
    rot = s["case"]["rot"]
    r, rest = x[..., :rot], x[..., rot:]
    if s["case"]["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((r, rest), -1)


def _plain_append(s):
    page = s["page_table"][s["req"], s["pos"] // PAGE].long()
    slot = s["pos"] % PAGE
    kept = torch.arange(PAGE, device=DEV) < s["t_kept"][:, None]  # [touched page][slot]
    for n, new in (("kc", _norm_rope(s, s["k"], s["kw"])), ("vc", s["v"].double())):
        codes, scale = s[n], s[n + "_s"]
        G = scale.shape[1]
        amax = torch.zeros(scale.shape, device=DEV)
        amax.index_reduce_(0, page, new.abs().amax(-1).float(), "amax")
        old = scale[s["t_phys"]]
        now = _pow2_scale(amax[s["t_phys"]])
        now = torch.where(s["t_kept"][:, None] > 0, torch.maximum(old, now), now)
        scale[s["t_phys"]] = now
        rows = codes[s["t_phys"]]
        moved = (rows.view(F8).float() * (old / now)[:, :, None, None]).to(F8).view(torch.uint8)
        grown = kept[:, None] & (now > old)[:, :, None]
        codes[s["t_phys"]] = torch.where(grown[..., None], moved, rows)
        q = (new.float() / scale[page][..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(F8)
        codes[page, :, slot] = q.view(torch.uint8)
    return _append_out(s)


def _append_out(s):
    n = s["n_shared"]
    return {"k": s["kc"][n:].view(F8), "k_scale": s["kc_s"][n:], "v": s["vc"][n:].view(F8),
            "v_scale": s["vc_s"][n:]}


def _gathered(s, n):
    """The cache through the page table, FP32 [batch, kv head, key, D]."""
    pt = s["page_table"].long()
    c = s[n][pt].view(F8).float() * s[n + "_s"][pt][..., None, None]
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
    n = sc.shape[-1]
    hidden = torch.arange(n, device=DEV) > pos[..., None]
    if c["op"] == "sparse":
        sel = torch.zeros((s["T"], H, n // PAGE + 1), dtype=torch.bool, device=DEV)
        sel.scatter_(-1, s["sel"].long() % (n // PAGE + 1), True)  # -1: the column behind the pages
        kept = torch.zeros((B, Q, H, n // PAGE), dtype=torch.bool, device=DEV)
        kept[..., 0] = True  # rows that pad the batch
        kept[s["req"], s["idx"]] = sel[..., :-1]
        kept = kept.view(B, Q, G, H // G, -1).permute(0, 2, 3, 1, 4)
        sc.view(*sc.shape[:-1], -1, PAGE).masked_fill_(~kept[..., None], -math.inf)
        del kept, sel
    sc.masked_fill_(hidden[:, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, G, -1, p.shape[-1]), _gathered(s, "vc")).view(B, G, H // G, Q, D) / l
    lse = (m + l.log()).view(B, H, Q)
    return {"out": o.view(B, H, Q, D).transpose(1, 2)[s["req"], s["idx"]].bfloat16(),
            "lse": lse.transpose(1, 2)[s["req"], s["idx"]].contiguous()}


def _plain_tables(s):
    s["state"].copy_(s["first"])
    q, c, T = s["q_lens"].long(), s["ctx"].long(), s["T"]
    have, need = -(-c // PAGE), -(-(c + q) // PAGE)
    took = (need - have).cumsum(0)
    starts = torch.zeros_like(s["starts"])
    starts[1:] = q.cumsum(0)
    at = s["state"][0] + (took - (need - have))  # each request's first page in the list
    table = s["page_table"]
    p = torch.arange(table.shape[1], device=DEV)
    new = (p >= have[:, None]) & (p < need[:, None])
    src = (at[:, None] + p - have[:, None]).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where(new, s["free"][src], table))
    s["state"][0] += took[-1]
    t = torch.arange(s["slots"].numel(), device=DEV)
    b = torch.searchsorted(starts, t, right=True).sub_(1).clamp_(0, q.numel() - 1)
    pos = torch.where(t < T, c[b] + t - starts[b], 0)
    slots = torch.where(t < T, table[b, pos // PAGE].long() * PAGE + pos % PAGE, -1)
    return {"page_table": table, "slots": slots, "positions": pos.int(), "starts": starts,
            "state": s["state"], "status": s["status"]}


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"append": _plain_append, "attn": _plain_attn, "sparse": _plain_attn,
                "tables": _plain_tables}[op](s)
    from paged_top_sparse_gb300 import binding as B
    if op == "append":
        B.sps_kv_append_rope(s["plan"], s["k"], s["v"], s["kw"], EPS, s["rope"], s["page_table"],
                             s["kc"], s["vc"], s["kc_s"], s["vc_s"], s["ws"])
        return _append_out(s)
    if op == "tables":
        s["state"].copy_(s["first"])
        B.sps_page_tables(s["q_lens"], s["ctx"], s["free"], s["state"], s["page_table"],
                          s["slots"], s["positions"], s["starts"], s["status"])
        return {"page_table": s["page_table"], "slots": s["slots"], "positions": s["positions"],
                "starts": s["starts"], "state": s["state"], "status": s["status"]}
    if op == "attn":
        B.paged_attention_fwd(s["plan"], s["q"], s["q_scale"], s["kc"], s["vc"], s["kc_s"],
                              s["vc_s"], s["page_table"], s["out"], s["out_lse"], s["scratch"],
                              s["ws"])
        return {"out": s["out"], "lse": s["out_lse"]}
    D = s["case"]["dim"]
    B.sparse_prefill_fwd_f16(s["plan"], s["q"], s["q_scale"], s["kc"], s["vc"], s["kc_s"],
                             s["vc_s"], s["page_table"], s["sel"], s["partial"], s["lse"], s["ws"])
    B.partial_combine_f16(s["partial"], s["lse"], s["out"].view(-1, D), s["out_lse"].view(-1))
    return {"out": s["out"], "lse": s["out_lse"]}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_append(s, q_lens, ctx):
    """Values: request by request, page by page.  Rotated keys next to a code's border may go either
    way, so keys have no single answer."""
    codes, scale, t = s["vc"].view(F8).double(), s["vc_s"].double(), 0
    for b in range(len(q_lens)):
        end = ctx[b] + q_lens[b]
        for p in range(ctx[b] // PAGE, (end - 1) // PAGE + 1):
            phys, lo, hi = int(s["page_table"][b, p]), max(ctx[b], p * PAGE), min(end, (p + 1) * PAGE)
            new = s["v"][t + lo - ctx[b]:t + hi - ctx[b]].double().transpose(0, 1)  # [head][token][D]
            a = new.abs().amax((1, 2))
            two = torch.exp2(torch.ceil(torch.log2(a.clamp(min=2.0 ** -60) / E4M3_MAX))).clamp(2.0 ** -40, 2.0 ** 40)
            if lo > p * PAGE:
                was = scale[phys].clone()
                two = torch.maximum(two, was)
                kept = codes[phys, :, :lo - p * PAGE] * (was / two)[:, None, None]
                codes[phys, :, :lo - p * PAGE] = _nearest_e4m3(kept)
            scale[phys] = two
            codes[phys, :, lo - p * PAGE:hi - p * PAGE] = _nearest_e4m3(new / two[:, None, None])
        t += q_lens[b]
    n = s["n_shared"]
    return {"k": None, "k_scale": None, "v": codes[n:], "v_scale": scale[n:]}


def _nearest_e4m3(x):
    """The nearest value of four significant bits above 2^-6, and multiples of 2^-9 below it."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    s = prepare(case, seed)
    q_lens, ctx = _lens(case)
    if case["op"] == "tables":
        return None  # whole numbers
    if case["op"] == "append":
        return _exact_append(s, q_lens, ctx)
    G, D, H = case["kv_heads"], case["dim"], case["heads"]
    out = torch.empty((s["T"], H, D), dtype=torch.float64, device=DEV)
    lse = torch.empty((s["T"], H), dtype=torch.float64, device=DEV)
    t = 0
    for b in range(case["batch"]):
        n = ctx[b] + q_lens[b]
        pages = s["page_table"][b, :(n - 1) // PAGE + 1].long()
        keys = torch.arange(n, device=DEV)
        for g in range(G):
            hs = slice(g * (H // G), (g + 1) * (H // G))
            k, v = ((s[c][pages, g].view(F8).double() * s[c + "_s"][pages, g].double()[:, None, None])
                    .reshape(-1, D)[:n] for c in ("kc", "vc"))
            for i in range(0, q_lens[b], 1024):
                j = min(q_lens[b], i + 1024)
                rows = s["q"][t + i:t + j, hs].double() * s["q_scale"]
                sc = torch.einsum("thd,kd->thk", rows, k) / math.sqrt(D)
                seen = (keys[None] <= ctx[b] + torch.arange(i, j, device=DEV)[:, None])[:, None]
                if case["op"] == "sparse":
                    picked = torch.zeros((j - i, H // G, pages.numel() + 1), device=DEV)
                    at = s["sel"][t + i:t + j, hs].long()
                    picked.scatter_(-1, torch.where(at < 0, pages.numel(), at), 1.0)
                    seen = seen & (picked[..., keys // PAGE] > 0)
                sc = torch.where(seen, sc, -math.inf)
                z = torch.logsumexp(sc, -1)
                out[t + i:t + j, hs] = torch.einsum("thk,kd->thd", torch.exp(sc - z[..., None]), v)
                lse[t + i:t + j, hs] = z
        t += q_lens[b]
    return {"out": out, "lse": lse}
