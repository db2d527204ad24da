"""e4m3 blocks and their products on the GPU, against 64-bit forms, and a verifying step put together from them and the
drafted trees' calls."""
import math

import pytest
import torch

import long_context_sparse_block_amd as misa
import tree_helpers as th

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the -m gpu tests need an MI355X")
    misa.load()


def hidden(g, rows, cols):
    return torch.randn((rows, cols), generator=g) * torch.exp(torch.randn(cols, generator=g))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 128), (3, 144), (17, 2048), (128, 112), (129, 272), (300, 1504)])
def test_quantize(rows, cols, block_rows, dtype):
    x = hidden(torch.Generator().manual_seed(rows + cols), rows, cols).to(dtype)
    x[rows // 2, :cols // 2] = 0
    if rows > 128:
        x[:128, :min(cols, 128)] = 0   # a block of zeros
    codes, scale = th.quantize(x, block_rows)
    got, s = misa.misa_quantize_blocks(x.cuda(), block_rows)
    assert got.dtype == torch.uint8
    assert torch.equal(s.cpu(), scale)
    assert torch.equal(got.cpu(), codes)
    wide = torch.full((rows + 1, cols + 24), float("nan"), dtype=dtype, device="cuda")   # rows of a wider matrix
    wide[:rows, 8:8 + cols] = x.cuda()
    out = torch.full((rows, cols), 7, dtype=torch.uint8, device="cuda").view(FP8), torch.full_like(s, 7)
    a, b = misa.misa_quantize_blocks(wide[:rows, 8:8 + cols], block_rows, codes=out[0], scale=out[1])
    assert a is out[0] and b is out[1]
    assert torch.equal(a.view(torch.uint8).cpu(), codes) and torch.equal(b.cpu(), scale)


def test_quantize_borders():
    """Quotients on and next to the borders between codes, in fp32 and at scales from the least to the largest: every
    code is that of the correctly rounded quotient."""
    g = torch.Generator().manual_seed(21)
    border = torch.cat([torch.arange(8, 16) + 0.5, torch.arange(16) + 0.5])   # of mantissas 1.xxx, and below the least
    rows = []
    for e in list(range(-125, 118, 9)) + [-80, -81, -79, 119, 120]:
        top = (1 + torch.rand(8, generator=g)) * 2.0 ** min(e + 8, 127)
        s = top / torch.full_like(top, 448)
        k = border[torch.randint(0, 24, (8, 127), generator=g)] * 2.0 ** torch.randint(-10, 5, (8, 127), generator=g)
        x = (k * s[:, None]).clamp(max=top.amax().item())
        x = x.view(torch.int32) + torch.randint(-2, 3, x.shape, generator=g).to(torch.int32)   # a few steps beside
        x = x.view(torch.float32).abs().minimum(top[:, None]) * (torch.randint(0, 2, x.shape, generator=g) * 2 - 1)
        rows.append(torch.cat([top[:, None], x], 1))
    x = torch.cat(rows)
    x[3, 5], x[4, 6] = -0.0, 0.0
    codes, scale = th.quantize(x, 1)
    got, s = misa.misa_quantize_blocks(x.cuda())
    assert torch.equal(s.cpu(), scale)
    assert torch.equal(got.cpu(), codes)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_extremes(block_rows):
    """Tiny values (scales at their least), the largest, NaN and infinities."""
    x = torch.randn((300, 256), generator=torch.Generator().manual_seed(2))
    x[0:128] *= 2.0 ** -140
    x[128:256, :128] *= 2.0 ** 120
    x[128:256, 128:] *= 2.0 ** -149 / x[128:256, 128:].abs().max() * 3
    x[260, 3], x[270, 200], x[271, 201] = float("nan"), math.inf, -math.inf
    codes, scale = th.quantize(x, block_rows)
    got, s = misa.misa_quantize_blocks(x.cuda(), block_rows)
    got = got.cpu()
    assert torch.equal(s.cpu(), scale)
    nan = (codes & 0x7F) == 0x7F
    assert nan.any() and torch.equal((got & 0x7F) == 0x7F, nan)
    assert torch.equal(got[~nan], codes[~nan])


def test_quantize_is_the_queries_rule():
    g = torch.Generator().manual_seed(4)
    q = torch.randn((2, 5, 16, 128), generator=g).bfloat16().cuda()
    q[0, 1, 3] = 0
    sh = misa.make_shape(2, 5, 64, 10, 16, 16)
    c, s = misa.misa_quantize_q(sh, q)
    got, scale = misa.misa_quantize_blocks(q.view(10, 2048))
    assert torch.equal(got.view(c.shape), c) and torch.equal(scale.view(s.shape), s)


def operands(seed, m, n, k):
    g = torch.Generator().manual_seed(seed)
    x8, xs = th.quantize(hidden(g, m, k).bfloat16(), 1)
    w8, ws = th.quantize(torch.randn((n, k), generator=g) * torch.exp(torch.randn((n, 1), generator=g)), 128)
    return x8, xs, w8, ws


SIZES = [(1, 1, 16), (1, 128, 128), (1, 2048, 2048), (2, 17, 144), (15, 130, 256), (16, 64, 384), (17, 257, 1504),
         (33, 127, 2064), (48, 300, 1024), (64, 1024, 512), (65, 129, 640), (100, 4099, 272), (128, 128, 128),
         (129, 255, 1920), (200, 1, 528), (257, 383, 144), (300, 513, 2048), (513, 300, 16), (1000, 130, 400),
         (2, 16, 16384), (70, 96, 16400), (1500, 700, 256),
         # forms that the sizes above do not reach: 32 columns to a workgroup, each size of tile, parts of the blocks
         (5, 4500, 272), (30, 4200, 144), (60, 4130, 400), (128, 8200, 256), (515, 4099, 1504), (700, 8200, 272),
         (4000, 4000, 528), (3990, 4090, 144), (65, 40, 8208), (120, 500, 4112), (300, 65, 12304),
         (500, 1003, 5008), (500, 515, 12304)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_product(m, n, k):
    ops = operands(m + n + k, m, n, k)
    got = misa.misa_matmul_q8(*(t.cuda() for t in ops))
    th.check_product(got, *ops)
    # codes by their own type, from rows of wider matrices, into columns of a wider one
    x8, xs, w8, ws = (t.cuda() for t in ops)
    wide = torch.full((m + 1, k + 48), 0x7F, dtype=torch.uint8, device="cuda")
    wide[:m, 32:32 + k] = x8
    tall = torch.full((n + 1, k + 16), 0x7F, dtype=torch.uint8, device="cuda")
    tall[:n, 16:16 + k] = w8
    out = torch.full((m + 1, n + 5), 7.0, dtype=torch.bfloat16, device="cuda")
    r = misa.misa_matmul_q8(wide[:m, 32:32 + k].view(FP8), xs, tall[:n, 16:16 + k].view(FP8), ws, out=out[:m, 3:3 + n])
    assert torch.equal(r, got)
    assert (out[m:] == 7).all() and (out[:, :3] == 7).all() and (out[:, 3 + n:] == 7).all()


@pytest.mark.parametrize("m,n,k", [(1, 40, 1024), (16, 64, 128), (40, 300, 528), (100, 300, 1024), (515, 300, 272)])
def test_product_of_terms_that_cancel(m, n, k):
    """Rows whose second half cancels the first in another order, over values of very different sizes: what is left is
    some 10^-4 of the terms."""
    g = torch.Generator().manual_seed(m + k)
    x, w = ((torch.randn((r, k), generator=g) * torch.exp(2 * torch.randn((r, k), generator=g))).clamp(-440, 440) for r in (m, n))
    x8, w8 = x.to(FP8).view(torch.uint8), w.to(FP8).view(torch.uint8)
    order = torch.randperm(k // 2, generator=g)
    x8[:, k // 2:], w8[:, k // 2:] = x8[:, :k // 2][:, order], (w8[:, :k // 2] ^ 0x80)[:, order]
    x8[:, 0] = 0x30
    ones = torch.ones((m, -(-k // 128))), torch.ones((-(-n // 128), -(-k // 128)))
    th.check_product(misa.misa_matmul_q8(x8.cuda(), ones[0].cuda(), w8.cuda(), ones[1].cuda()), x8, ones[0], w8, ones[1])


def test_product_repeats_and_shows_nan():
    m, n, k = 70, 300, 1040
    ops = operands(8, m, n, k)
    x8, xs, w8, ws = (t.cuda() for t in ops)
    ref = misa.misa_matmul_q8(x8, xs, w8, ws)
    assert torch.equal(misa.misa_matmul_q8(x8, xs, w8, ws), ref)
    x8[3, 1039], w8[299, 5], xs[60, 2] = 0x7F, 0xFF, float("nan")
    got = misa.misa_matmul_q8(x8, xs, w8, ws)
    bad = torch.zeros((m, n), dtype=torch.bool, device="cuda")
    bad[3], bad[60], bad[:, 299] = True, True, True
    assert torch.equal(got.isnan(), bad)
    assert torch.equal(got[~bad], ref[~bad])
    ws[0, 1] = float("inf")
    assert not torch.isfinite(misa.misa_matmul_q8(x8, xs, w8, ws)[:, :128]).any()


@pytest.mark.parametrize("m,n,k", [(4, 128, 8192), (64, 2048, 1024), (300, 300, 4096), (120, 500, 4112)])
def test_product_in_graphs_and_on_streams(m, n, k):
    ops = operands(9, m, n, k)
    x8, xs, w8, ws = (t.cuda() for t in ops)
    x = torch.randn((m, k), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    ref = misa.misa_matmul_q8(x8, xs, w8, ws)
    c, s = misa.misa_quantize_blocks(x)
    chained = misa.misa_matmul_q8(c, s, w8, ws)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            a, b = misa.misa_quantize_blocks(x)
            outs = misa.misa_matmul_q8(a, b, w8, ws), misa.misa_matmul_q8(x8, xs, w8, ws)
        graphs.append((g, outs))
    for _ in range(3):
        for g, outs in graphs:
            outs[0].zero_(), outs[1].zero_()
            g.replay()
        again = misa.misa_matmul_q8(x8, xs, w8, ws, stream=torch.cuda.Stream())
        torch.cuda.synchronize()
        for _, outs in graphs:
            assert torch.equal(outs[0], chained) and torch.equal(outs[1], ref)
        assert torch.equal(again, ref)


def test_rows_past_4_gib():
    """Row offsets that pass 32 bits: the last rows of 2^31 + codes, and of an output of as many elements."""
    m, n, k = 140000, 16, 16384
    x8 = torch.zeros((m, k), dtype=torch.uint8, device="cuda")
    g = torch.Generator().manual_seed(6)
    part = operands(10, 40, n, k)
    x8[-40:] = part[0].cuda()
    xs = torch.ones((m, 128), device="cuda")
    xs[-40:] = part[1].cuda()
    out = misa.misa_matmul_q8(x8, xs, part[2].cuda(), part[3].cuda())
    assert (out[:-40] == 0).all()
    th.check_product(out[-40:], *part)
    del x8, xs, out
    x = torch.zeros((m, k), dtype=torch.bfloat16, device="cuda")
    tail = torch.randn((40, k), generator=g).bfloat16()
    x[-40:] = tail.cuda()
    codes, scale = misa.misa_quantize_blocks(x)
    want = th.quantize(tail, 1)
    assert torch.equal(codes[-40:].cpu(), want[0]) and torch.equal(scale[-40:].cpu(), want[1])
    assert (scale[:-40] == 1).all()


def test_refused_calls_raise():
    x8 = torch.zeros((4, 256), dtype=torch.uint8, device="cuda")
    xs, ws = torch.ones((4, 2), device="cuda"), torch.ones((1, 2), device="cuda")
    w8 = torch.zeros((20, 256), dtype=torch.uint8, device="cuda")
    for bad in (dict(x=x8[:, :128]), dict(xs=xs[:, :1]), dict(ws=xs), dict(w=w8.view(torch.int8)), dict(w=w8.t()),
                dict(xs=xs.half()), dict(x=x8.cpu()), dict(x=None), dict(out=torch.zeros((4, 20), device="cuda")),
                dict(out=torch.zeros((20, 4), dtype=torch.bfloat16, device="cuda").t()),
                dict(ws_=torch.zeros(64, dtype=torch.uint8))):
        a = dict(x=x8, xs=xs, w=w8, ws=ws, out=None, ws_=None)
        a.update(bad)
        with pytest.raises(ValueError):
            misa.misa_matmul_q8(a["x"], a["xs"], a["w"], a["ws"], out=a["out"], ws=a["ws_"])
    with pytest.raises(misa.MisaError):   # 8 columns past a 16-byte border
        misa.misa_matmul_q8(torch.zeros((4, 264), dtype=torch.uint8, device="cuda")[:, 8:], xs, w8, ws)
    with pytest.raises(misa.MisaError):
        misa.misa_matmul_q8(x8[:, :24], xs[:, :1].contiguous(), w8[:, :24], ws[:, :1].contiguous())
    with pytest.raises(misa.MisaError):   # rows of the output that overlap
        misa.misa_matmul_q8(x8, xs, w8, ws, out=torch.zeros(100, dtype=torch.bfloat16, device="cuda").as_strided((4, 20), (10, 1)))
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    for call in (lambda: misa.misa_quantize_blocks(x, 2), lambda: misa.misa_quantize_blocks(x.double()),
                 lambda: misa.misa_quantize_blocks(x.view(2, 2, 256)), lambda: misa.misa_quantize_blocks(x, codes=x),
                 lambda: misa.misa_quantize_blocks(x, scale=xs.t()), lambda: misa.misa_quantize_blocks(x.t())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: misa.misa_quantize_blocks(x[:, :24]), lambda: misa.misa_quantize_blocks(x[:, 4:132])):
        with pytest.raises(misa.MisaError):
            call()
    assert misa.misa_matmul_q8(x8[:0], xs[:0], w8, ws).shape == (0, 20)
    assert misa.misa_quantize_blocks(x[:0])[0].shape == (0, 256)


# ---------------------------------------------------------------- a verifying step

def test_a_verifying_step_equals_decoding_the_kept_path():
    """One layer over two requests: hidden states -> e4m3 blocks -> product to q, k, v -> rotation by the trees'
    positions -> pages -> tree attention -> e4m3 blocks -> output product.  Then the accepted path is kept in the pages,
    and the same tokens decoded one after another give the same pages, and so bit for bit the same next step; their
    attention agrees within both kernels' bounds (tree_helpers.attention: half a bf16 step of the output and of each
    weight, and the scores' fp32 error twice; twice that for two kernels)."""
    g = torch.Generator().manual_seed(12)
    H, KH, D, hid, page, width = 8, 2, 128, 512, 16, 12
    dev = "cuda"
    wide = (H + 2 * KH) * D
    w_in = misa.misa_quantize_blocks((torch.randn((wide, hid), generator=g) / math.sqrt(hid)).to(dev), 128)
    w_out = misa.misa_quantize_blocks((torch.randn((hid, H * D), generator=g) / math.sqrt(H * D)).to(dev), 128)
    f, ms = misa.rope_inv_freq(64, device=dev)
    i32 = dict(dtype=torch.int32, device=dev)

    def project(x):
        return misa.misa_matmul_q8(*misa.misa_quantize_blocks(x.bfloat16().to(dev)), *w_in).view(x.shape[0], -1, D)

    def new_cache():
        shape = (2 * width, page, KH, D)
        return dict(k=torch.zeros(shape, dtype=torch.bfloat16, device=dev), v=torch.zeros(shape, dtype=torch.bfloat16, device=dev),
                    table=torch.full((2, width), -1, **i32), free=torch.arange(2 * width, **i32))

    def step(c, y, cached, new, parents=None):
        """New tokens' q, k, v rows through the attention and the output's product."""
        T = y.shape[0]
        p = misa.misa_plan_pages(cached, new, c["free"], c["table"], page, T)
        c["free"] = c["free"][int(p.n_taken):]
        pos = p.positions
        if parents is not None:
            tree = misa.misa_plan_tree(parents, p.q_start, p.kv_lens, 1)
            pos = tree.positions
        q = misa.misa_rope(y[:, :H], pos, f, mscale=ms)
        misa.misa_write_pages(y[:, H:H + KH], p.slots, c["k"], v=y[:, H + KH:], v_pages=c["v"], positions=pos, inv_freq=f,
                              mscale=ms)
        args = (q, c["k"], c["v"], c["table"], p.q_start, p.kv_lens)
        o, _ = (misa.misa_attention_paged(*args, max_new=T) if parents is None
                else misa.misa_attention_tree(*args, tree.mask, max_new=T))
        return q, o, misa.misa_matmul_q8(*misa.misa_quantize_blocks(o.view(T, H * D)), *w_out), p

    def rows(c, b, n):
        t = torch.arange(n, device=dev)
        e = c["table"][b].long()[t // page]
        return torch.stack([c["k"][e, t % page], c["v"][e, t % page]])

    prompt = [37, 30]
    trees = [[-1, 0, 0, 1, 1, 2, 3, 6], [-1, 0, 1, 0, 3]]
    path = torch.tensor([[0, 1, 3, 6], [0, 3, 4, -1]], **i32)
    first, drafts, after = (project(torch.randn((n, hid), generator=g)) for n in (sum(prompt), 13, 2))

    c = new_cache()
    *_, p = step(c, first, torch.zeros(2, **i32), torch.tensor(prompt, **i32))
    q, out, _, p = step(c, drafts, p.kv_lens, torch.tensor([8, 5], **i32), torch.tensor(sum(trees, []), **i32))
    kept = misa.misa_keep_path(path, p.q_start, p.kv_lens, c["table"], c["k"], v_pages=c["v"])
    assert kept.tolist() == [41, 33]
    last = step(c, after, kept, torch.ones(2, **i32))

    d = new_cache()
    *_, p = step(d, first, torch.zeros(2, **i32), torch.tensor(prompt, **i32))
    lens = p.kv_lens
    for i in range(4):
        on = [b for b in range(2) if path[b, i] >= 0]
        at = torch.tensor([int(path[b, i]) + 8 * b for b in on], device=dev)
        q1, one, _, p = step(d, drafts[at], lens, torch.tensor([int(b in on) for b in range(2)], **i32))
        lens = p.kv_lens
        assert torch.equal(q1, q[at])
        for j, b in enumerate(on):
            k, v = (x.double().abs().amax(0).repeat_interleave(H // KH, 0) for x in rows(d, b, int(lens[b])))   # [H, D]
            mag = (q1[j].double().abs() * k).sum(1) / math.sqrt(D)
            e = ((D + 8) * mag + 8 * (1 + mag)) * 2.0 ** -24
            o = out[at[j]].double()
            bound = 2 * (2.0 ** -8 * (o.abs() * (1 + 2.0 ** -7)) + (2.0 ** -8 + 2 * e + int(lens[b]) * 2.0 ** -24)[:, None] * v * 1.01)
            assert bool(((one[j].double() - o).abs() <= bound).all())
    assert lens.tolist() == kept.tolist()
    for b in range(2):
        assert torch.equal(rows(c, b, int(kept[b])), rows(d, b, int(kept[b])))
    # the pages being equal, a step over them is the same bit for bit
    again = step(d, after, lens, torch.ones(2, **i32))
    for x, y in zip(last[:3], again[:3]):
        assert torch.equal(x, y)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_captured_verifying_step(fp8):
    """The whole step in one graph, replayed with other lengths, trees, paths and hidden states: the same bits as eager
    calls, in the pages too."""
    g = torch.Generator().manual_seed(31)
    H, KH, D, hid, page, width, n, T = 8, 2, 64, 384, 16, 30, 3, 40
    dev, i32 = "cuda", dict(dtype=torch.int32, device="cuda")
    wide = (H + 2 * KH) * D
    w_in = misa.misa_quantize_blocks((torch.randn((wide, hid), generator=g) / math.sqrt(hid)).to(dev), 128)
    w_out = misa.misa_quantize_blocks((torch.randn((hid, H * D), generator=g) / math.sqrt(H * D)).to(dev), 128)
    f, ms = misa.rope_inv_freq(D, device=dev)
    shape = (n * width, page, KH, D)

    def inputs(seed, cached, new):
        g = torch.Generator().manual_seed(seed)
        parents = sum((th.random_parents(g, m, "tree") for m in new), [])
        path = torch.full((n, 5), -1, dtype=torch.int32)
        for b, m in enumerate(new):
            node, up = m - 1, []
            while node >= 0:
                up.append(node)
                node = parents[sum(new[:b]) + node]
            up = sorted(up)[:5]
            path[b, :len(up)] = torch.tensor(up, dtype=torch.int32)
        k = torch.randn(shape, generator=g)
        v = torch.randn(shape, generator=g)
        order = torch.randperm(n * width, generator=g).to(torch.int32)
        table = torch.full((n, width), -1, dtype=torch.int32)
        for b, c in enumerate(cached):
            taken = -(-c // page)
            table[b, :taken] = order[:taken]
            order = order[taken:]
        free = torch.zeros(n * width, dtype=torch.int32)
        free[:len(order)] = order
        s = dict(hidden=torch.randn((T, hid), generator=g).bfloat16(), parents=torch.tensor(parents + [0] * (T - len(parents)), dtype=torch.int32),
                 path=path, cached=torch.tensor(cached, dtype=torch.int32), new=torch.tensor(new, dtype=torch.int32), table=table,
                 free=free, k=k.bfloat16(), v=v.bfloat16())
        if fp8:
            s["k"], s["v"] = (x.to(torch.float8_e4m3fn).view(torch.uint8) for x in (k, v))
            s["ks"], s["vs"] = (0.5 + torch.rand(shape[:3], generator=g) for _ in range(2))
        return {name: x.to(dev) for name, x in s.items()}

    def step(s):
        y = misa.misa_matmul_q8(*misa.misa_quantize_blocks(s["hidden"]), *w_in).view(T, -1, D)
        p = misa.misa_plan_pages(s["cached"], s["new"], s["free"], s["table"], page, T)
        tree = misa.misa_plan_tree(s["parents"], p.q_start, p.kv_lens, 1)
        q = misa.misa_rope(y[:, :H], tree.positions, f, mscale=ms)
        ks, vs = s.get("ks"), s.get("vs")
        misa.misa_write_pages(y[:, H:H + KH], p.slots, s["k"], ks, v=y[:, H + KH:], v_pages=s["v"], v_scale_pages=vs,
                              positions=tree.positions, inv_freq=f, mscale=ms)
        o, _ = misa.misa_attention_tree(q, s["k"], s["v"], s["table"], p.q_start, p.kv_lens, tree.mask, ks, vs, max_new=16,
                                        out=torch.zeros_like(q))
        out = misa.misa_matmul_q8(*misa.misa_quantize_blocks(o.view(T, H * D)), *w_out)
        kept = misa.misa_keep_path(s["path"], p.q_start, p.kv_lens, s["table"], s["k"], ks, s["v"], vs)
        return o, out, kept

    cases = [(1, [100, 333, 7], [9, 16, 12]), (2, [0, 464, 31], [16, 1, 16]), (3, [50, 0, 201], [0, 13, 5])]
    wants = []
    for c in cases:
        s = inputs(*c)
        wants.append((step(s), s))
    static = inputs(*cases[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(static)
    for c, (want, after) in list(zip(cases, wants)) * 2:
        for name, x in inputs(*c).items():
            static[name].copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
        for name in after:
            assert torch.equal(static[name].view(torch.uint8), after[name].view(torch.uint8)), name
