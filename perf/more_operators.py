"""The operators of a serving step that verifies drafted tokens on an e4m3 checkpoint, as measurable cases.

Such a step quantises its activations in blocks of 128 and multiplies them with e4m3 weights, plans the trees of drafted
tokens of its sequences (which node descends from which, and at what position it stands), attends from every node to the
cached prefix and the node's own ancestors, and, once a path of a tree is accepted, moves that path's keys and values to
where the cached prefix goes on.  Each case below is one call of one of these operators.  `run` computes it with
elementary torch operations, or (own = True) with the framework's kernels.
"""
import math

import torch

own = False

DEV = "cuda"
FP8 = torch.float8_e4m3fn
TYPES = dict(bf16=torch.bfloat16, fp16=torch.float16, fp32=torch.float32)


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # the activations of a decode batch before a projection
        dict(name="quantize_decode_64", op="quantize", rows=64, cols=2048, dtype="bf16", block_rows=1),
        # the hidden states of a prefill chunk of 8192
        dict(name="quantize_chunk_8k", op="quantize", rows=8192, cols=4096, dtype="bf16", block_rows=1),
        # the projection to the indexer's queries (64 heads of 128) in a decode batch: bound by the weights
        dict(name="product_decode_64", op="product", m=64, n=8192, k=2048),
        # odd sizes throughout: a ragged prompt, a last block of 96 columns, an odd width
        dict(name="product_odd", op="product", m=515, n=4099, k=1504),
        # the same projection in a prefill chunk of 8192, from a hidden size of 4096
        dict(name="product_chunk_8k", op="product", m=8192, n=8192, k=4096),
        # one decode step's trees: 64 requests with 32 drafted tokens each
        dict(name="tree_plan_64x32", op="plan", n_seq=64, new_lo=32, new_hi=32, ctx=16384),
        # many requests with trees of all sizes, among them ones without a draft
        dict(name="tree_plan_500", op="plan", n_seq=500, new_lo=0, new_hi=256, ctx=131072),
        # one request with a large tree: where latency counts
        dict(name="tree_attn_one", op="attn", n_seq=1, new_lo=64, new_hi=64, ctx_lo=8192, ctx_hi=8192, heads=32,
             kv_heads=8, dim=128, page=64, fp8=False),
        # a decode batch over ragged contexts of up to 16K tokens, 16 drafted tokens for each request
        dict(name="tree_attn_64x16k", op="attn", n_seq=64, new_lo=16, new_hi=16, ctx_lo=8192, ctx_hi=16384, heads=32,
             kv_heads=8, dim=128, page=64, fp8=False),
        # trees of 1 to 257 tokens in one call, e4m3 pages of 16 keys, heads of 64, five query heads to a key head
        dict(name="tree_attn_mixed_fp8", op="attn", n_seq=9, new_lo=1, new_hi=257, ctx_lo=515, ctx_hi=5003, heads=20,
             kv_heads=4, dim=64, page=16, fp8=True),
        # the accepted paths of a decode batch, keys and values of 8 heads in bf16
        dict(name="keep_path_64", op="keep", n_seq=64, new=32, most=8, ctx=500, heads=8, dim=128, page=64, fp8=False,
             values=True),
        # the same for the index keys of 500 requests: one head of 128 in e4m3 with a scale for each key
        dict(name="keep_index_keys_500", op="keep", n_seq=500, new=64, most=12, ctx=300, heads=1, dim=128, page=64,
             fp8=True, values=False),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "plan", "attn", "attn", "keep"])
    if op == "quantize":
        cols = 16 * _spread(rng, 1, 512)
        return dict(op=op, rows=_spread(rng, 1, min(8192, 8192 * 2048 // cols)), cols=cols,
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), block_rows=rng.choice([1, 1, 128]))
    if op == "product":
        k = 16 * _spread(rng, 8, 512)
        n = _spread(rng, 16, 8192)
        return dict(op=op, m=_spread(rng, 1, min(8192, 8192 * 8192 * 4096 // (n * k))), n=n, k=k)
    if op == "plan":
        hi = _spread(rng, 1, 256)
        return dict(op=op, n_seq=_spread(rng, 1, 500), new_lo=rng.choice([0, 1, hi]), new_hi=hi,
                    ctx=_spread(rng, 500, 131072))
    if op == "attn":
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 3, 4, 8])
        n, ctx = _spread(rng, 1, 64), _spread(rng, 300, 16384)
        hi = _spread(rng, 1, max(1, min(256, 1024 * 12288 * 32 // (n * ctx * heads))))
        return dict(op=op, n_seq=n, new_lo=rng.choice([1, hi]), new_hi=hi, ctx_lo=max(hi, ctx // 2), ctx_hi=max(hi, ctx),
                    heads=heads, kv_heads=kv, dim=rng.choice([64, 128]), page=rng.choice([16, 48, 64, 128]),
                    fp8=rng.random() < 0.5)
    new = _spread(rng, 1, 64)
    fp8 = rng.random() < 0.5
    values = rng.random() < 0.6
    return dict(op=op, n_seq=_spread(rng, 1, 64 if values else 500), new=new, most=rng.randint(1, 12),
                ctx=_spread(rng, 1, 500), heads=rng.choice([1, 2, 8]) if values else 1, dim=rng.choice([64, 128]),
                page=rng.choice([16, 48, 64]), fp8=fp8, values=values)


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


def _starts(new):
    q_start = torch.zeros(new.numel() + 1, dtype=torch.int32, device=DEV)
    q_start[1:] = new.cumsum(0)
    return q_start


def _hidden(g, rows, cols):
    """Activations: channels of different sizes, a few of them much larger than the rest."""
    size = torch.exp(0.5 * torch.randn(cols, generator=g, device=DEV))
    size[torch.rand(cols, generator=g, device=DEV) < 0.005] *= 20
    return torch.randn((rows, cols), generator=g, device=DEV) * size


def _trees(g, q_start, tokens):
    """Parents of every new token, relative to its sequence: the first is the last verified token (a child of the cached
    prefix, -1), each other a child of one of the eight before it."""
    t = torch.arange(tokens, device=DEV)
    b = torch.searchsorted(q_start[1:].contiguous(), t.to(torch.int32), right=True)
    live = b < q_start.numel() - 1
    i = t - q_start[b.clamp(max=q_start.numel() - 2)]
    back = 1 + (torch.rand(tokens, generator=g, device=DEV) * i.clamp(max=8)).long()
    return torch.where(live, i - back.minimum(i + 1), -1).to(torch.int32)


def _pool(g, slots, heads, dim, fp8):
    """A page pool's rows [slots, heads, dim] and, for e4m3, their scales."""
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


def _paged(g, case, values=True):
    """Ragged sequences' keys (and values) over shuffled pages."""
    n, page, kv, dim = case["n_seq"], case["page"], case.get("kv_heads", case["heads"]), case["dim"]
    most = case["ctx_hi"] if "ctx_hi" in case else case["ctx"] + case["new"]
    width = -(-most // page)
    n_pages = n * width + 3
    table = torch.randperm(n_pages, generator=g, device=DEV)[:n * width].to(torch.int32).view(n, width).contiguous()
    shape = (n_pages, page, kv, dim)
    s = dict(table=table, v_pages=None, v_scale=None)
    for name in ("k", "v") if values else ("k",):
        rows, scale = _pool(g, n_pages * page, kv, dim, case["fp8"])
        s[name + "_pages"] = rows.view(shape)
        s[name + "_scale"] = None if scale is None else scale.view(shape[:3])
    return s


def prepare(case, seed):
    op = case["op"]
    g = _rng(seed)
    if op == "quantize":
        return dict(case=case, x=_hidden(g, case["rows"], case["cols"]).to(TYPES[case["dtype"]]))
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        x8, xs = _plain_quantize(_hidden(g, m, k), 1)
        w8, ws = _plain_quantize(torch.randn((n, k), generator=g, device=DEV) / math.sqrt(k), 128)
        return dict(case=case, x8=x8, xs=xs, w8=w8, ws=ws, out=torch.empty((m, n), dtype=torch.bfloat16, device=DEV))
    if op == "plan":
        new = _shared(g, case["new_lo"], case["new_hi"], case["n_seq"])
        q_start = _starts(new)
        # the serving loop's token buffers are padded to a multiple of 64
        tokens = (int(q_start[-1]) + 63) // 64 * 64
        return dict(case=case, q_start=q_start, lens=_ints(g, 0, case["ctx"], case["n_seq"]) + new,
                    parents=_trees(g, q_start, tokens), words=max(1, -(-case["new_hi"] // 32)))
    if op == "attn":
        new = _shared(g, case["new_lo"], case["new_hi"], case["n_seq"])
        q_start = _starts(new)
        tokens = int(q_start[-1])
        lens = _ints(g, case["ctx_lo"], case["ctx_hi"], case["n_seq"])
        parents = _trees(g, q_start, tokens)
        s = _paged(g, case)
        # logits of standard deviation 2: some keys matter much more than others
        q = (2 * torch.randn((tokens, case["heads"], case["dim"]), generator=g, device=DEV)).to(torch.bfloat16)
        mask, _ = _plain_plan(parents, q_start, lens, max(1, -(-case["new_hi"] // 32)))
        s.update(case=case, q=q, q_start=q_start, lens=lens, parents=parents, mask=mask, out=torch.empty_like(q),
                 lse=torch.empty(q.shape[:2], dtype=torch.float32, device=DEV))
        return s
    s = _paged(g, case, case["values"])
    n, new = case["n_seq"], case["new"]
    # Accepted paths: the first node and, in order, some of the nodes behind those whose places they take, as trees laid
    # out level by level have them (so a second pass over the same pages moves the same rows again), or a chain.
    keep = _ints(g, 1, min(case["most"], new), n)
    path = torch.full((n, case["most"]), -1, dtype=torch.int32, device=DEV)
    rank = torch.rand((n, new), generator=g, device=DEV)
    rank.masked_fill_(torch.arange(new, device=DEV)[None] < keep[:, None], 2.0)
    nodes = rank.argsort(1)                                    # the nodes behind the kept places, in no order
    col = torch.arange(case["most"], device=DEV)[None]
    late = torch.where(col[:, :new] < keep[:, None] - 1, nodes[:, :case["most"]], new).sort(1).values
    chain = (new - keep < keep - 1)[:, None]
    width = late.shape[1]
    path[:, 1:width + 1] = torch.where(chain, col[:, 1:width + 1], late[:, :case["most"] - 1]).to(torch.int32)
    path[:, 0] = 0
    path.masked_fill_(col >= keep[:, None], -1)
    s.update(case=case, path=path, q_start=_starts(torch.full((n,), new, dtype=torch.int32, device=DEV)),
             lens=_ints(g, 0, case["ctx"], n) + new, kept=torch.empty(n, dtype=torch.int32, device=DEV))
    return s


# ---------------------------------------------------------------- plain forms

def _plain_quantize(x, block_rows):
    """e4m3 codes (as bytes) of x [R, K] and the scales of its blocks of block_rows x 128."""
    r, k = x.shape
    up, across = -(-r // block_rows), -(-k // 128)
    y = torch.zeros((up * block_rows, across * 128), device=x.device)
    y[:r, :k] = x
    y = y.view(up, block_rows, across, 128)
    amax = y.abs().amax((1, 3))
    # a tensor divisor: a plain number would be turned into a product with its reciprocal
    scale = torch.where(amax > 0, (amax / torch.full_like(amax, 448)).clamp(min=2.0 ** -126), 1.0)
    codes = (y / scale[:, None, :, None]).to(FP8).view(torch.uint8)
    return codes.view(up * block_rows, across * 128)[:r, :k].contiguous(), scale


def _plain_product(x8, xs, w8, ws):
    k = x8.shape[1]
    x = x8.view(FP8).float() * xs.repeat_interleave(128, 1)[:, :k]
    w = w8.view(FP8).float() * ws.repeat_interleave(128, 0)[:w8.shape[0]].repeat_interleave(128, 1)[:, :k]
    return torch.matmul(x, w.t()).to(torch.bfloat16)


def _seq_of(q_start, tokens):
    t = torch.arange(tokens, dtype=torch.int32, device=q_start.device)
    b = torch.searchsorted(q_start[1:].contiguous(), t, right=True)
    live = b < q_start.numel() - 1
    b = b.clamp(max=q_start.numel() - 2)
    return b, (t - q_start[b]).long(), live


def _plain_plan(parents, q_start, lens, words):
    """Ancestor bits [tokens, words] (int32, a node's own bit among them) and positions of drafted tokens."""
    T, width = parents.numel(), 32 * words
    b, i, live = _seq_of(q_start, T)
    # sees[t, j]: node t descends from node j of its sequence, or is it
    sees = (torch.arange(width, device=parents.device)[None] == i[:, None]) & live[:, None]
    none = T   # a row that sees nothing
    up = torch.where(live & (parents >= 0), q_start[b].long() + parents, none)
    sees = torch.cat([sees, sees.new_zeros((1, width))])
    up = torch.cat([up, up.new_full((1,), none)])
    for _ in range(max(1, (width - 1).bit_length())):   # ancestors twice as far each time
        sees = sees | sees[up]
        up = up[up]
    sees = sees[:T]
    new = (q_start[1:] - q_start[:-1])
    pos = (lens - new)[b] + sees.sum(1) - 1
    bits = (sees.view(T, words, 32).long() << torch.arange(32, device=parents.device)).sum(2)
    bits = torch.where(bits >= 1 << 31, bits - (1 << 32), bits)
    return bits.to(torch.int32), torch.where(live, pos, -1).to(torch.int32)


def _values(pages, scale, rows):
    """fp32 values [..., heads, dim] of the pool rows `rows`."""
    flat = pages.view(-1, *pages.shape[2:])[rows]
    if scale is None:
        return flat.float()
    return flat.view(FP8).float() * scale.view(-1, scale.shape[2])[rows][..., None]


def _plain_attention(s):
    q, page, table, lens, q_start = s["q"], s["case"]["page"], s["table"], s["lens"].long(), s["q_start"]
    T, H, D = q.shape
    n, KH = table.shape[0], s["k_pages"].shape[2]
    G, N, M = H // KH, s["case"]["ctx_hi"], s["case"]["new_hi"]
    t = torch.arange(N, device=q.device)
    rows = table[:, t // page].long() * page + t % page                    # [n, N]
    k = _values(s["k_pages"], s["k_scale"], rows).permute(0, 2, 3, 1).contiguous()   # [n, KH, D, N]
    b, i, _ = _seq_of(q_start, T)
    qp = torch.zeros((n, M, H, D), device=q.device)
    qp[b, i] = q.float() / math.sqrt(D)
    score = torch.matmul(qp.view(n, M, KH, G, D).transpose(1, 2).reshape(n, KH, M * G, D), k)
    del k
    # a node sees the cached tokens, and the drafted ones whose bits its mask has
    words = s["mask"].shape[1]
    bits = ((s["mask"][:, :, None] >> torch.arange(32, device=q.device, dtype=torch.int32)) & 1).bool().view(T, 32 * words)
    mask = torch.zeros((n, M, 32 * words), dtype=torch.bool, device=q.device)
    mask[b, i] = bits
    first = lens - (q_start[1:] - q_start[:-1]).long()                     # the first drafted token's place
    node = t[None] - first[:, None]                                        # [n, N]
    drafted = mask.gather(2, node.clamp(0, 32 * words - 1)[:, None].expand(n, M, N))
    seen = ((node < 0)[:, None] | drafted) & (t < lens[:, None])[:, None]
    seen = seen[:, None, :, None, :].expand(n, KH, M, G, N).reshape(n, KH, M * G, N)
    v = _values(s["v_pages"], s["v_scale"], rows).transpose(1, 2).contiguous()       # [n, KH, N, D]
    # keys behind a sequence's end are whatever the page holds
    v.masked_fill_((t >= lens[:, None])[:, None, :, None], 0.0)
    score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    total = score.sum(-1, keepdim=True)
    out = torch.matmul(score, v) / torch.where(total > 0, total, 1.0)
    lse = (top + total.log()).squeeze(-1)
    out = out.view(n, KH, M, G, D).transpose(1, 2)[b, i].reshape(T, H, D)
    return out.to(q.dtype), lse.view(n, KH, M, G).transpose(1, 2)[b, i].reshape(T, H)


def _plain_keep(s):
    path, page, table = s["path"].long(), s["case"]["page"], s["table"].long()
    first = (s["lens"] - (s["q_start"][1:] - s["q_start"][:-1])).long()
    on = path >= 0
    col = torch.arange(path.shape[1], device=path.device)[None].expand_as(path)
    b = torch.arange(path.shape[0], device=path.device)[:, None].expand_as(path)[on]

    def slot(at):
        at = (first[:, None] + at)[on]
        return table[b, at // page] * page + at % page
    src, dst = slot(path), slot(col)
    pools = [x for x in (s["k_pages"], s["k_scale"], s["v_pages"], s["v_scale"]) if x is not None]
    got = [x.view(-1, *x.shape[2:])[src] for x in pools]   # all read before any is written
    [x.view(-1, *x.shape[2:]).index_copy_(0, dst, y) for x, y in zip(pools, got)]
    return (first + on.sum(1)).to(torch.int32)


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import long_context_sparse_block_amd as misa
        if op == "quantize":
            codes, scale = misa.misa_quantize_blocks(s["x"], c["block_rows"])
        elif op == "product":
            return misa.misa_matmul_q8(s["x8"], s["xs"], s["w8"], s["ws"], out=s["out"])
        elif op == "plan":
            return misa.misa_plan_tree(s["parents"], s["q_start"], s["lens"], s["words"])
        elif op == "attn":
            return misa.misa_attention_tree(s["q"], s["k_pages"], s["v_pages"], s["table"], s["q_start"], s["lens"],
                                            s["mask"], s["k_scale"], s["v_scale"], max_new=c["new_hi"], out=s["out"],
                                            lse=s["lse"])
        else:
            kept = misa.misa_keep_path(s["path"], s["q_start"], s["lens"], s["table"], s["k_pages"], s["k_scale"],
                                       s["v_pages"], s["v_scale"], kept_lens=s["kept"])
    elif op == "quantize":
        codes, scale = _plain_quantize(s["x"].float(), c["block_rows"])
    elif op == "product":
        return _plain_product(s["x8"], s["xs"], s["w8"], s["ws"])
    elif op == "plan":
        return _plain_plan(s["parents"], s["q_start"], s["lens"], s["words"])
    elif op == "attn":
        return _plain_attention(s)
    else:
        kept = _plain_keep(s)
    if op == "quantize":   # codes as the values they stand for
        return codes.view(FP8), scale
    return [kept] + [x.view(FP8) if x.dtype == torch.uint8 else x
                     for x in (s["k_pages"], s["k_scale"], s["v_pages"], s["v_scale"]) if x is not None]


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["cols"]
        blocks = -(-case["rows"] // case["block_rows"]) * -(-case["cols"] // 128)
        return dict(bytes=n * ((4 if case["dtype"] == "fp32" else 2) + 1) + 4 * blocks, flops=2 * n)
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        across = -(-k // 128)
        return dict(bytes=m * k + n * k + 2 * m * n + 4 * across * (m + -(-n // 128)), flops=2 * m * n * k)
    if op == "keep":
        row = case["dim"] * (1 if case["fp8"] else 2) + (4 if case["fp8"] else 0)
        moved = case["n_seq"] * max(0, (min(case["most"], case["new"]) - 1) / 2)
        return dict(bytes=2 * moved * case["heads"] * row * (2 if case["values"] else 1)
                    + 4 * case["n_seq"] * (case["most"] + 3), flops=0)
    new = (case["new_lo"] + case["new_hi"]) / 2
    tokens, words = case["n_seq"] * new, max(1, -(-case["new_hi"] // 32))
    if op == "plan":
        return dict(bytes=tokens * (8 + 4 * words) + 8 * case["n_seq"], flops=0)
    row = case["dim"] * (1 if case["fp8"] else 2) + (4 if case["fp8"] else 0)
    ctx = (case["ctx_lo"] + case["ctx_hi"]) / 2
    return dict(bytes=2 * case["n_seq"] * ctx * case["kv_heads"] * row
                + tokens * (case["heads"] * (4 * case["dim"] + 4) + 4 * words),
                flops=4 * tokens * (ctx - new + 1) * case["heads"] * case["dim"])


# ---------------------------------------------------------------- the definition, in 64 bits

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


def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return None
    s = prepare(case, seed)
    if op == "keep":   # whole rows move, row by row
        page, path, first = case["page"], s["path"].tolist(), (s["lens"] - case["new"]).tolist()
        table, src, dst = s["table"].tolist(), [], []
        for b, nodes in enumerate(path):
            for i, node in enumerate(nodes):
                if node >= 0:
                    for at, to in ((first[b] + node, src), (first[b] + i, dst)):
                        to.append(table[b][at // page] * page + at % page)
        got = [None]
        for x in (s["k_pages"], s["k_scale"], s["v_pages"], s["v_scale"]):
            if x is not None:
                y = (x.view(FP8) if x.dtype == torch.uint8 else x).double().view(-1, *x.shape[2:])
                old = y.clone()
                for i, j in zip(src, dst):
                    y[j] = old[i]
                got.append(y.view(x.shape))
        return got
    if op == "quantize":
        x, r = s["x"].double(), case["block_rows"]
        codes, scales = [], []
        for i in range(0, x.shape[0], 4096 if r == 1 else r):
            part = x[i:i + (4096 if r == 1 else r)]
            row, codes_of = [], []
            for j in range(0, x.shape[1], 128):
                y = part[:, j:j + 128]
                top = y.abs().amax(1) if r == 1 else y.abs().max().reshape(1)
                sc = (top / 448).float().double().clamp(min=2.0 ** -126)   # the scale is held in 32 bits
                sc[top == 0] = 1.0
                codes_of.append(_e4m3((y / sc[:, None]).float().double()))   # a quotient of 32 bits
                row.append(sc[:, None])
            codes.append(torch.cat(codes_of, 1))
            scales.append(torch.cat(row, 1))
        return torch.cat(codes), torch.cat(scales)
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        x, w = s["x8"].view(FP8).double(), s["w8"].view(FP8).double()
        y = torch.zeros((m, n), dtype=torch.float64, device=DEV)
        ws = s["ws"].double()[torch.arange(n, device=DEV) // 128]
        for j in range(0, k, 128):
            y += (x[:, j:j + 128] * s["xs"][:, j // 128, None].double()) @ (w[:, j:j + 128] * ws[:, j // 128, None]).t()
        return y
    T, H, D = s["q"].shape
    G = H // case["kv_heads"]
    out = torch.zeros((T, H, D), dtype=torch.float64, device=DEV)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=DEV)
    start, parents = s["q_start"].tolist(), s["parents"].tolist()
    for b in range(case["n_seq"]):
        t0, t1, n = start[b], start[b + 1], int(s["lens"][b])
        if t1 == t0:
            continue
        m = t1 - t0
        tree = torch.zeros((m, m), dtype=torch.bool)
        for i in range(m):
            j = i
            while j >= 0:
                tree[i, j] = True
                j = parents[t0 + j]
        seen = torch.cat([torch.ones((m, n - m), dtype=torch.bool), tree], 1).to(DEV)
        t = torch.arange(n, device=DEV)
        k, v = _exact_rows(s, "k", b, t), _exact_rows(s, "v", b, t)
        for h in range(H):
            score = (s["q"][t0:t1, h].double() @ k[:, h // G].t()) / math.sqrt(D)
            score.masked_fill_(~seen, -math.inf)
            lse[t0:t1, h] = torch.logsumexp(score, -1)
            out[t0:t1, h] = torch.softmax(score, -1) @ v[:, h // G]
    return out, lse
