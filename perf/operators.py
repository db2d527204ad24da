"""The operators of a paged serving step around the indexer, as measurable cases.

A serving step over a paged key cache plans its pages from the request lengths, rotates the new queries and
keys, writes the new keys and values into their pages, and attends over the pages: over every key of the
prefix, or over the tokens that the indexer picked.  Each case below is one call of one of these operators.
`run` computes it with elementary torch operations, or (own = True) with the framework's kernels.
"""
import math

import torch

own = False

DEV = "cuda"
FP8 = torch.float8_e4m3fn


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decode step's bookkeeping: 64 requests, one new token each, contexts up to 128K, 64-key pages
        dict(name="plan_decode_64", op="plan", n_seq=64, page=64, ctx=131072, new_lo=1, new_hi=1, width=2049),
        # a batch of prompts admitted at once, most of them fresh, ragged lengths
        dict(name="plan_prompts_500", op="plan", n_seq=500, page=64, ctx=4096, new_lo=1, new_hi=1024, width=96),
        # the indexer queries of a prefill chunk of 8192 at the end of a 128K prompt: 64 of 128 dims, half layout
        dict(name="rope_chunk_8k", op="rope", tokens=8192, heads=64, dim=128, rot=64, start=0, layout="half",
             dtype="bf16", pos=122880, factor=40.0, backward=False),
        # a decode batch's queries, whole head, interleaved
        dict(name="rope_decode_64", op="rope", tokens=64, heads=32, dim=128, rot=128, start=0,
             layout="interleaved", dtype="bf16", pos=131071, factor=1.0, backward=False),
        # the gradient of a query with a position part behind the rest of the head, fp32, odd sizes
        dict(name="rope_grad_odd", op="rope", tokens=4093, heads=7, dim=192, rot=64, start=128,
             layout="interleaved", dtype="fp32", pos=60000, factor=4.0, backward=True),
        # the indexer keys of a prefill chunk, rotated and stored in fp8 with a scale for each key
        dict(name="write_index_keys_8k", op="write", tokens=8192, heads=1, dim=128, fp8=True, values=False, rot=64,
             layout="half", page=64, pages=160, pos=122880),
        # keys and values of a ragged prompt batch into bf16 pages
        dict(name="write_kv_4099", op="write", tokens=4099, heads=8, dim=128, fp8=False, values=True, rot=128,
             layout="half", page=64, pages=96, pos=5000),
        # a decode batch over ragged contexts of up to 16K tokens, four query heads to a key head
        dict(name="attn_decode_64x16k", op="attn", n_seq=64, new_lo=1, new_hi=1, ctx_lo=8192, ctx_hi=16384, heads=32,
             kv_heads=8, dim=128, page=64, fp8=False),
        # a prefill chunk at the end of a 32K context
        dict(name="attn_chunk_2k_32k", op="attn", n_seq=1, new_lo=2048, new_hi=2048, ctx_lo=32768, ctx_hi=32768,
             heads=32, kv_heads=8, dim=128, page=64, fp8=False),
        # chunks and decodes in one call, fp8 pages of 16 keys, heads of 64, five query heads to a key head
        dict(name="attn_mixed_fp8", op="attn", n_seq=9, new_lo=0, new_hi=515, ctx_lo=515, ctx_hi=5003, heads=20,
             kv_heads=4, dim=64, page=16, fp8=True),
        # a decode batch over the tokens that the indexer picked, one key head for all query heads
        dict(name="selected_decode_64", op="selected", n_seq=64, new=1, ctx_lo=12000, ctx_hi=16384, heads=64,
             kv_heads=1, dim=128, page=64, fp8=False, topk=2048),
        # a chunk in the middle of a prompt over its picked tokens, fp8 pages
        dict(name="selected_chunk_1000", op="selected", n_seq=1, new=1000, ctx_lo=32768, ctx_hi=32768, heads=32,
             kv_heads=4, dim=128, page=64, fp8=True, topk=2048),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "write", "attn", "attn", "selected"])
    if op == "plan":
        page = rng.choice([16, 64, 128])
        ctx = _spread(rng, 500, 131072)
        hi = _spread(rng, 1, 1024)
        return dict(op=op, n_seq=_spread(rng, 1, 500), page=page, ctx=ctx, new_lo=rng.choice([0, 1]), new_hi=hi,
                    width=-(-(ctx + hi) // page) + rng.randrange(4))
    if op == "rope":
        dim = rng.choice([64, 80, 128, 192, 256])
        layout = rng.choice(["half", "interleaved"])
        whole = rng.random() < 0.4
        rot = dim if whole else rng.choice([16, 20, 32, 64])
        start = 0 if whole or rng.random() < 0.5 else dim - rot
        heads = _spread(rng, 1, 64)
        return dict(op=op, tokens=_spread(rng, 1, 8192 * 64 * 128 // (heads * dim * 2)) if heads * dim > 4096
                    else _spread(rng, 1, 8192), heads=heads, dim=dim, rot=rot, start=start, layout=layout,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), pos=_spread(rng, 1, 1000000),
                    factor=rng.choice([1.0, 4.0, 40.0]), backward=rng.random() < 0.3)
    if op == "write":
        heads = rng.choice([1, 2, 3, 8])
        page = rng.choice([16, 64, 100])
        tokens = _spread(rng, 1, 8192 if heads == 1 else 4099)
        dim = rng.choice([64, 128])
        return dict(op=op, tokens=tokens, heads=heads, dim=dim, fp8=rng.random() < 0.5,
                    values=rng.random() < 0.6, rot=rng.choice([0, 32, 64]), layout=rng.choice(["half", "interleaved"]),
                    page=page, pages=-(-tokens // page) + 1 + rng.randrange(8), pos=_spread(rng, 1, 131072))
    kv = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 128])
    page = rng.choice([16, 48, 64, 128])
    if op == "attn":
        heads = kv * rng.choice([1, 3, 4, 8])
        if rng.random() < 0.5:   # decode
            n, ctx, new = _spread(rng, 1, 64), _spread(rng, 100, 16384), rng.choice([1, 1, 2, 4])
        else:
            n, ctx, new = rng.choice([1, 1, 2, 5]), _spread(rng, 300, 8192), _spread(rng, 16, 700)
        new = min(new, ctx)
        lo = rng.choice([0, 1, new]) if n > 1 else new
        return dict(op=op, n_seq=n, new_lo=min(lo, new), new_hi=new, ctx_lo=max(new, ctx // 2), ctx_hi=ctx,
                    heads=heads, kv_heads=kv, dim=dim, page=page, fp8=rng.random() < 0.5)
    heads = kv * rng.choice([1, 4, 8, 16])
    n = rng.choice([1, 2, 16, 64])
    new = 1 if n > 2 else _spread(rng, 1, 500)
    ctx = max(new, _spread(rng, 300, 16384))
    return dict(op=op, n_seq=n, new=new, ctx_lo=max(new, ctx - ctx // 4), ctx_hi=ctx, heads=heads, kv_heads=kv,
                dim=dim, page=page, fp8=rng.random() < 0.5, topk=rng.choice([100, 256, 512, 1024, 2048]))


# ---------------------------------------------------------------- inputs

def _rng(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _ints(g, lo, hi, n):
    return torch.randint(int(lo), int(hi) + 1, (n,), generator=g, device=DEV, dtype=torch.int32)


def _shared(g, lo, hi, n):
    """Lengths spread evenly over [lo, hi] and shuffled: the same sum for every seed."""
    at = torch.linspace(hi, lo, n, device=DEV, dtype=torch.float64).round().to(torch.int32)
    return at[torch.randperm(n, generator=g, device=DEV)]


def _inv_freq(rot, base, factor):
    """Rotary frequencies (fp64, radians a position); factor > 1: stretched for contexts `factor` times as long,
    the low frequencies by the whole factor, the high ones not at all, a ramp between, with the attention's
    temperature in mscale."""
    j = torch.arange(0, rot, 2, dtype=torch.float64)
    f = base ** (-j / rot)
    if factor <= 1.0:
        return f.to(DEV), 1.0
    original = 4096

    def dim_of(turns):
        return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
    lo, hi = max(math.floor(dim_of(32)), 0), min(math.ceil(dim_of(1)), rot - 1)
    ramp = ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 0.001)).clamp(0, 1)
    return (f * (1 - ramp) + f / factor * ramp).to(DEV), 0.1 * math.log(factor) + 1.0


def _pool(g, slots, heads, dim, fp8):
    """A page pool's rows [slots, heads, dim] and, for fp8, their scales."""
    rows = torch.empty((slots, heads, dim), dtype=torch.uint8 if fp8 else torch.bfloat16, device=DEV)
    scale = torch.empty((slots, heads), dtype=torch.float32, device=DEV) if fp8 else None
    step = max(1, (1 << 27) // (heads * dim))
    for s in range(0, slots, step):
        x = torch.randn((min(step, slots - s), heads, dim), generator=g, device=DEV)
        if fp8:
            sc = x.abs().amax(-1) / 448
            scale[s:s + step] = sc
            rows[s:s + step] = (x / sc[..., None]).to(FP8).view(torch.uint8)
        else:
            rows[s:s + step] = x
    return rows, scale


def _paged(case, seed, new):
    """Ragged sequences over shuffled pages."""
    g = _rng(seed)
    n, page, kv, dim = case["n_seq"], case["page"], case["kv_heads"], case["dim"]
    lens = _ints(g, case["ctx_lo"], case["ctx_hi"], n)
    q_start = torch.zeros(n + 1, dtype=torch.int32, device=DEV)
    q_start[1:] = new.cumsum(0)
    tokens = int(q_start[-1])
    width = -(-case["ctx_hi"] // page)
    n_pages = n * width + 3
    table = torch.randperm(n_pages, generator=g, device=DEV)[:n * width].to(torch.int32).view(n, width).contiguous()
    k, ks = _pool(g, n_pages * page, kv, dim, case["fp8"])
    v, vs = _pool(g, n_pages * page, kv, dim, case["fp8"])
    shape = (n_pages, page, kv, dim)
    # logits of standard deviation 2: some keys matter much more than others
    q = (2 * torch.randn((tokens, case["heads"], dim), generator=g, device=DEV)).to(torch.bfloat16)
    s = dict(q=q, k_pages=k.view(shape), v_pages=v.view(shape), table=table, q_start=q_start, lens=lens,
             k_scale=None if ks is None else ks.view(shape[:3]), v_scale=None if vs is None else vs.view(shape[:3]))
    return s, g


def _seq_of(q_start, tokens):
    t = torch.arange(tokens, dtype=torch.int32, device=q_start.device)
    b = torch.searchsorted(q_start[1:].contiguous(), t, right=True)
    return b, t - q_start[b]


def prepare(case, seed):
    op = case["op"]
    g = _rng(seed)
    if op == "plan":
        n, page, width = case["n_seq"], case["page"], case["width"]
        cached = _ints(g, 0, case["ctx"], n)
        new = _shared(g, case["new_lo"], case["new_hi"], n)
        total = int(new.sum())
        table = torch.full((n, width), -1, dtype=torch.int32, device=DEV)
        have = (cached + page - 1) // page
        ids = torch.randperm(n * width, generator=g, device=DEV).to(torch.int32)
        owned = torch.arange(width, device=DEV)[None, :] < have[:, None]
        table[owned] = ids.view(n, width)[owned]
        free = ids.view(n, width)[~owned].contiguous()
        # the serving loop's token buffers are padded to a multiple of 64
        return dict(case=case, cached=cached, new=new, table=table, free=free, tokens=(total + 63) // 64 * 64)
    if op == "rope":
        dt = dict(bf16=torch.bfloat16, fp16=torch.float16, fp32=torch.float32)[case["dtype"]]
        x = torch.randn((case["tokens"], case["heads"], case["dim"]), generator=g, device=DEV).to(dt)
        pos = (torch.arange(case["tokens"], dtype=torch.int32, device=DEV) + case["pos"]
               - _ints(g, 0, min(case["pos"], 100), 1))
        f, m = _inv_freq(case["rot"], 10000.0, case["factor"])
        return dict(case=case, x=x, pos=pos, f=f, m=m, out=torch.empty_like(x))
    if op == "write":
        T, H, D, page, pages = (case[c] for c in ("tokens", "heads", "dim", "page", "pages"))
        rows = [torch.randn((T, H, D), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]
        # whole pages in shuffled order, the first one begun by an earlier chunk
        perm = torch.randperm(pages, generator=g, device=DEV)
        at = torch.arange(T, device=DEV) + int(_ints(g, 0, min(page - 1, pages * page - T), 1))
        slots = perm[at // page] * page + at % page
        kind = torch.uint8 if case["fp8"] else torch.bfloat16
        s = dict(case=case, k=rows[0], v=rows[1] if case["values"] else None, slots=slots,
                 pos=torch.arange(T, dtype=torch.int32, device=DEV) + case["pos"], rot=case["rot"])
        for n in ("k", "v") if case["values"] else ("k",):
            s[n + "_pages"] = torch.zeros((pages, page, H, D), dtype=kind, device=DEV)
            s[n + "_scale"] = torch.zeros((pages, page, H), device=DEV) if case["fp8"] else None
        s["f"], s["m"] = _inv_freq(case["rot"], 10000.0, 1.0) if case["rot"] else (None, 1.0)
        return s
    if op == "attn":
        new = _shared(g, case["new_lo"], case["new_hi"], case["n_seq"])
        s, _ = _paged(case, seed + 1, new)
        s.update(case=case, out=torch.empty_like(s["q"]), max_new=case["new_hi"])
        s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=DEV)
        return s
    new = torch.full((case["n_seq"],), case["new"], dtype=torch.int32, device=DEV)
    s, g = _paged(case, seed + 1, new)
    tokens, topk = s["q"].shape[0], case["topk"]
    b, i = _seq_of(s["q_start"], tokens)
    pos = s["lens"][b] - case["new"] + i   # token's place in its sequence
    # distinct random tokens of the prefix in no order, -1 behind them where the prefix is short: what a top-k leaves
    idx = torch.full((tokens, topk), -1, dtype=torch.int32, device=DEV)
    hi = int(s["lens"].max())
    for t0 in range(0, tokens, 256):
        p = pos[t0:t0 + 256].long()
        r = torch.rand((p.numel(), hi), generator=g, device=DEV)
        r.masked_fill_(torch.arange(hi, device=DEV)[None, :] > p[:, None], -1.0)
        val, at = r.topk(min(topk, hi), dim=1)
        idx[t0:t0 + 256, :at.shape[1]] = torch.where(val >= 0, at, -1).to(torch.int32)
    s.update(case=case, idx=idx, pos=pos, out=torch.empty_like(s["q"]))
    s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms

def _plain_plan(s):
    page, table, T = s["case"]["page"], s["table"], s["tokens"]
    cached, new = s["cached"].long(), s["new"].long()
    n, width = table.shape
    have = (cached + page - 1) // page
    need = (cached + new + page - 1) // page - have
    first = need.cumsum(0) - need
    col = torch.arange(width, device=table.device)[None, :] - have[:, None]
    fresh = (col >= 0) & (col < need[:, None])
    at = (first[:, None] + col).clamp(0, max(s["free"].numel() - 1, 0))
    table = torch.where(fresh, s["free"][at], table)
    q_start = torch.zeros(n + 1, dtype=torch.int32, device=table.device)
    q_start[1:] = new.cumsum(0)
    t = torch.arange(T, device=table.device)
    b = torch.searchsorted(q_start[1:].long().contiguous(), t, right=True)
    live = b < n
    b = b.clamp(max=n - 1)
    pos = cached[b] + t - q_start[b]
    slot = table[b, (pos // page).clamp(0, width - 1)].long() * page + pos % page
    return dict(table=table, q_start=q_start, lens=(cached + new).to(torch.int32),
                slots=torch.where(live, slot, -1), positions=torch.where(live, pos, -1).to(torch.int32),
                taken=need.sum().to(torch.int32).reshape(1))


def _plain_rope(x, pos, f, m, layout, start, backward):
    rot = 2 * f.numel()
    angle = pos.double()[:, None] * f[None, :]
    c, sn = (angle.cos() * m).float()[:, None, :], (angle.sin() * m).float()[:, None, :]
    if backward:
        sn = -sn
    y = x.float()
    part = y[..., start:start + rot]
    if layout == "half":
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        turned = torch.cat([a * c - b * sn, a * sn + b * c], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * c - b * sn, a * sn + b * c], -1).flatten(-2)
    return torch.cat([y[..., :start], turned, y[..., start + rot:]], -1).to(x.dtype)


def _plain_write(rows, slots, pages, scale):
    flat = pages.view(-1, *pages.shape[2:])
    if scale is None:
        flat[slots] = rows.to(pages.dtype)
        return
    x = rows.float()
    amax = x.abs().amax(-1)
    # a tensor divisor: a plain number would be turned into a product with its reciprocal
    sc = torch.where(amax > 0, amax / torch.full_like(amax, 448), 1.0)
    flat[slots] = (x / sc[..., None]).to(FP8).view(torch.uint8)
    scale.view(-1, scale.shape[2])[slots] = sc


def _values(pages, scale, rows):
    """fp32 values [..., heads, dim] of the pool rows `rows`."""
    flat = pages.view(-1, *pages.shape[2:])[rows]
    if scale is None:
        return flat.float()
    return flat.view(FP8).float() * scale.view(-1, scale.shape[2])[rows][..., None]


def _soft(score, seen, values):
    """softmax over the last axis of score (where seen) times values, and the log of its sum; 0 and -inf where
    nothing is seen."""
    score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    total = score.sum(-1, keepdim=True)
    out = torch.matmul(score, values) / torch.where(total > 0, total, 1.0)
    return out, (top + total.log()).squeeze(-1)


def _plain_attention(s):
    q, page, table, lens, q_start = s["q"], s["case"]["page"], s["table"], s["lens"].long(), s["q_start"]
    T, H, D = q.shape
    n, KH = table.shape[0], s["k_pages"].shape[2]
    G, N, M = H // KH, s["case"]["ctx_hi"], max(1, s["case"]["new_hi"])
    t = torch.arange(N, device=q.device)
    rows = table[:, t // page].long() * page + t % page                    # [n, N]
    k = _values(s["k_pages"], s["k_scale"], rows).permute(0, 2, 3, 1).contiguous()   # [n, KH, D, N]
    b, i = _seq_of(q_start, T)
    qp = torch.zeros((n, M, H, D), device=q.device)
    qp[b, i] = q.float() / math.sqrt(D)
    qp = qp.view(n, M, KH, G, D).transpose(1, 2).reshape(n, KH, M * G, D)
    score = torch.matmul(qp, k)
    del k
    new = (q_start[1:] - q_start[:-1]).long()
    pos = (lens - new)[:, None] + torch.arange(M, device=q.device)          # [n, M]
    seen = (t[None, None, :] <= pos[:, :, None]) & (t < lens[:, None])[:, None, :]
    seen = seen[:, None, :, None, :].expand(n, KH, M, G, N)
    v = _values(s["v_pages"], s["v_scale"], rows).transpose(1, 2).contiguous()       # [n, KH, N, D]
    # keys behind a sequence's end are whatever the page holds
    v.masked_fill_((t >= lens[:, None])[:, None, :, None], 0.0)
    out, lse = _soft(score, seen.reshape(n, KH, M * G, N), v)
    out = out.view(n, KH, M, G, D).transpose(1, 2)[b, i].reshape(T, H, D)
    lse = lse.view(n, KH, M, G).transpose(1, 2)[b, i].reshape(T, H)
    return out.to(q.dtype), lse


def _plain_selected(s):
    q, page, idx = s["q"], s["case"]["page"], s["idx"].long()
    T, H, D = q.shape
    KH = s["k_pages"].shape[2]
    G = H // KH
    b, _ = _seq_of(s["q_start"], T)
    seen = (idx >= 0) & (idx <= s["pos"][:, None])
    at = torch.where(seen, idx, 0)
    rows = s["table"][b[:, None], at // page].long() * page + at % page     # [T, topk]
    k = _values(s["k_pages"], s["k_scale"], rows).permute(0, 2, 3, 1).contiguous()
    score = torch.matmul((q.float() / math.sqrt(D)).view(T, KH, G, D), k)
    del k
    v = _values(s["v_pages"], s["v_scale"], rows).transpose(1, 2).contiguous()
    out, lse = _soft(score, seen[:, None, None, :].expand_as(score), v)
    return out.reshape(T, H, D).to(q.dtype), lse.reshape(T, H)


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import long_context_sparse_block_amd as misa
        if op == "plan":
            p = misa.misa_plan_pages(s["cached"], s["new"], s["free"], s["table"], c["page"], s["tokens"])
            return dict(table=s["table"], q_start=p.q_start, lens=p.kv_lens, slots=p.slots, positions=p.positions,
                        taken=p.n_taken)
        if op == "rope":
            return misa.misa_rope(s["x"], s["pos"], s["f"], layout=c["layout"], rot_start=c["start"], mscale=s["m"],
                                  backward=c["backward"], out=s["out"])
        if op == "write":
            misa.misa_write_pages(s["k"], s["slots"], s["k_pages"], s["k_scale"], v=s["v"], v_pages=s.get("v_pages"),
                                  v_scale_pages=s.get("v_scale"), positions=s["pos"] if c["rot"] else None,
                                  inv_freq=s["f"], layout=c["layout"], mscale=s["m"])
        elif op == "attn":
            return misa.misa_attention_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["q_start"], s["lens"],
                                             s["k_scale"], s["v_scale"], max_new=s["max_new"], out=s["out"],
                                             lse=s["lse"])
        else:
            return misa.misa_attention_selected(s["q"], s["k_pages"], s["v_pages"], s["table"], s["q_start"],
                                                s["lens"], s["idx"], s["k_scale"], s["v_scale"], out=s["out"],
                                                lse=s["lse"])
    elif op == "plan":
        return _plain_plan(s)
    elif op == "rope":
        return _plain_rope(s["x"], s["pos"], s["f"], s["m"], c["layout"], c["start"], c["backward"])
    elif op == "write":
        k = s["k"].float()   # rounded (or quantised) once, after the rotation
        k = _plain_rope(k, s["pos"], s["f"], s["m"], c["layout"], 0, False) if c["rot"] else k
        _plain_write(k, s["slots"], s["k_pages"], s["k_scale"])
        if c["values"]:
            _plain_write(s["v"], s["slots"], s["v_pages"], s["v_scale"])
    elif op == "attn":
        return _plain_attention(s)
    else:
        return _plain_selected(s)
    # the pages after the write, fp8 codes as the values they stand for, beside their scales
    return [x.view(FP8) if x.dtype == torch.uint8 else x
            for x in (s["k_pages"], s["k_scale"], s.get("v_pages"), s.get("v_scale")) if x is not None]


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "plan":
        tokens = case["n_seq"] * (case["new_lo"] + case["new_hi"]) / 2
        pages = tokens / case["page"]
        return dict(bytes=case["n_seq"] * 16 + tokens * 12 + pages * 8, flops=0)
    if op == "rope":
        return dict(bytes=2 * case["tokens"] * case["heads"] * case["dim"] * (4 if case["dtype"] == "fp32" else 2),
                    flops=3 * case["tokens"] * case["heads"] * case["rot"])
    if op == "write":
        rows = case["tokens"] * case["heads"] * (2 if case["values"] else 1)
        return dict(bytes=rows * (case["dim"] * (3 if case["fp8"] else 4) + (4 if case["fp8"] else 0))
                    + 8 * case["tokens"], flops=3 * case["tokens"] * case["heads"] * case["rot"])
    row = case["dim"] * (1 if case["fp8"] else 2) + (4 if case["fp8"] else 0)
    ctx = (case["ctx_lo"] + case["ctx_hi"]) / 2
    if op == "attn":
        new = (case["new_lo"] + case["new_hi"]) / 2
        keys = ctx - (new - 1) / 2   # seen by a query, on average
        tokens = case["n_seq"] * new
        kv = case["n_seq"] * ctx
    else:
        tokens = case["n_seq"] * case["new"]
        keys = min(case["topk"], ctx)
        # distinct tokens read: at most every query's own picks, at most the whole prefix
        kv = case["n_seq"] * min(ctx, case["new"] * keys)
    return dict(bytes=2 * kv * case["kv_heads"] * row + tokens * case["heads"] * (4 * case["dim"] + 4)
                + (4 * tokens * case["topk"] if op == "selected" else 0),
                flops=4 * tokens * keys * case["heads"] * case["dim"])


# ---------------------------------------------------------------- the definition, in 64 bits

def _exact_rope(x, pos, f, m, layout, start, backward):
    """Each pair as a complex number times m exp(i angle) (its conjugate for the gradient)."""
    half = f.numel()
    j = torch.arange(half, device=x.device)
    ia, ib = (start + j, start + half + j) if layout == "half" else (start + 2 * j, start + 2 * j + 1)
    y = x.double().clone()
    angle = pos.double().view(-1, 1, 1) * f.view(1, 1, -1) * (-1.0 if backward else 1.0)
    z = torch.complex(y[..., ia], y[..., ib]) * torch.polar(torch.full_like(angle, m), angle)
    y[..., ia], y[..., ib] = z.real, z.imag
    return y


def _e4m3(x):
    """fp64 -> the nearest e4m3 value (ties to even), |x| <= 448."""
    e = torch.floor(torch.log2(x.abs().clamp(min=1e-30))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def _exact_rows(s, name, b, t):
    """fp64 [len(t), heads, dim] of tokens t of sequence b."""
    page = s["case"]["page"]
    p = s["table"][b].long()[t // page]
    got = s[name + "_pages"][p, t % page]
    if s[name + "_scale"] is None:
        return got.double()
    return got.view(FP8).double() * s[name + "_scale"][p, t % page].double()[..., None]


def _exact_one(q, k, v, seen):
    """q [R, D], k [N, D], v [N, D], seen [R, N]: outputs and log-sums by torch's own softmax in fp64."""
    score = (q @ k.t()) / math.sqrt(q.shape[1])
    score.masked_fill_(~seen, -math.inf)
    lse = torch.logsumexp(score, -1)
    w = torch.exp(score - lse[:, None])
    w[lse == -math.inf] = 0.0
    return w @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return None
    if op == "rope":
        return _exact_rope(s["x"], s["pos"], s["f"], s["m"], case["layout"], case["start"], case["backward"])
    if op == "write":
        k = s["k"].double()
        if case["rot"]:
            k = _exact_rope(s["k"], s["pos"], s["f"], s["m"], case["layout"], 0, False)
        got = []
        for name, x in (("k", k), ("v", s["v"].double() if case["values"] else None)):
            if x is None:
                continue
            pages = torch.zeros(s[name + "_pages"].shape, dtype=torch.float64, device=DEV)
            flat = pages.view(-1, *pages.shape[2:])
            if case["fp8"]:
                sc = (x.abs().amax(-1) / 448).float().double()   # the scale is held in 32 bits
                sc[sc == 0] = 1.0
                flat[s["slots"]] = _e4m3((x / sc[..., None]).float().double())   # a quotient of 32 bits
                scale = torch.zeros(s[name + "_scale"].shape, dtype=torch.float64, device=DEV)
                scale.view(-1, scale.shape[2])[s["slots"]] = sc
                got += [pages, scale]
            else:
                flat[s["slots"]] = x
                got.append(pages)
        return got
    T, H, D = s["q"].shape
    KH = case["kv_heads"]
    G = H // KH
    out = torch.zeros((T, H, D), dtype=torch.float64, device=DEV)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=DEV)
    start = s["q_start"].tolist()
    for b in range(case["n_seq"]):
        t0, t1, n = start[b], start[b + 1], int(s["lens"][b])
        if t1 == t0 or n == 0:
            continue
        t = torch.arange(n, device=DEV)
        k, v = _exact_rows(s, "k", b, t), _exact_rows(s, "v", b, t)
        pos = n - (t1 - t0) + torch.arange(t1 - t0, device=DEV)
        if op == "attn":
            for h in range(KH):
                q = s["q"][t0:t1, h * G:(h + 1) * G].double().reshape(-1, D)
                o, e = _exact_one(q, k[:, h], v[:, h], t[None, :] <= pos.repeat_interleave(G)[:, None])
                out[t0:t1, h * G:(h + 1) * G] = o.view(t1 - t0, G, D)
                lse[t0:t1, h * G:(h + 1) * G] = e.view(t1 - t0, G)
            continue
        for i in range(t1 - t0):
            at = s["idx"][t0 + i].long()
            at = at[(at >= 0) & (at <= pos[i])]
            ki, vi = k[at].transpose(0, 1), v[at].transpose(0, 1)            # [KH, picked, D]
            score = torch.matmul(s["q"][t0 + i].double().view(KH, G, D), ki.transpose(1, 2).contiguous())
            score /= math.sqrt(D)
            e = torch.logsumexp(score, -1)
            out[t0 + i] = torch.matmul(torch.exp(score - e[..., None]), vi.contiguous()).view(H, D)
            lse[t0 + i] = e.view(H)
    return out, lse
