"""Narrow paths of drafted trees, workspaces of the caller's and places past 32 bits on the GPU, against 64-bit forms."""
import pytest
import torch

import long_context_sparse_block_amd as misa
import tree_helpers as th
from test_gpu_products import operands
from test_gpu_tree import batch, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the -m gpu tests need an MI355X")
    misa.load()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("nodes", [[0], [3], [-1], [0, 4, -1, 9, 2, 5, 0]])
def test_paths_of_one_entry(nodes, fp8):
    """A first node or a later one alone, none, and one that is no new token of its sequence."""
    n, page, heads, dim, new = len(nodes), 16, 2, 64, 6
    g = torch.Generator().manual_seed(n)
    lens = [new + int(torch.randint(0, 60, (1,), generator=g)) for _ in nodes]
    width = -(-max(lens) // page)
    table = torch.randperm(n * width, generator=g).to(torch.int32).view(n, width)
    shape = (n * width, page, heads, dim)
    pools = []
    for _ in range(2):
        pools.append(torch.randint(0, 256, shape, generator=g).to(torch.uint8) if fp8 else torch.randn(shape, generator=g).bfloat16())
        if fp8:
            pools.append(torch.rand(shape[:3], generator=g))
    q_start = torch.tensor(starts([new] * n), dtype=torch.int32)
    path = torch.tensor(nodes, dtype=torch.int32).view(n, 1)
    want, kept = th.keep(path, q_start, lens, table, page, pools)
    got = [x.cuda() for x in pools]
    k, ks, v, vs = got if fp8 else (got[0], None, got[1], None)
    r = misa.misa_keep_path(path.cuda(), q_start.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), table.cuda(),
                            k, ks, v, vs)
    assert r.tolist() == kept == [x - new + (0 <= i < new) for x, i in zip(lens, nodes)]
    for x, y in zip(got, want):
        assert torch.equal(x.cpu(), y)


# ---------------------------------------------------------------- workspaces of the caller's

GUARD = 512


class Scratch:
    """One buffer for calls of different sizes: exactly the bytes that a call asks for, of NaN as fp32 and as bf16, and
    guard bytes behind them."""

    def __init__(self, most):
        self.buf = torch.empty(most + GUARD, dtype=torch.uint8, device="cuda")

    def of(self, need):
        assert 0 < need <= self.buf.numel() - GUARD
        self.need = need
        self.buf[:need] = 0xFF
        self.buf[need:] = 0x5A
        return self.buf[:need]

    def whole(self):
        return bool((self.buf[self.need:] == 0x5A).all())


def tree_need(p, d, max_new):
    """misa_attention_tree_workspace_bytes of a batch."""
    kp = d["k_pages"]
    fp8 = d["k_scale_pages"] is not None
    pages = misa.KvPages(kp.data_ptr(), d["v_pages"].data_ptr(), d["k_scale_pages"].data_ptr() if fp8 else 0,
                         d["v_scale_pages"].data_ptr() if fp8 else 0, d["block_table"].data_ptr(), d["block_table"].shape[1],
                         kp.shape[0], kp.shape[1], int(fp8))
    q = d["q"]
    shape = misa.AttnShape(d["kv_lens"].numel(), q.shape[1], kp.shape[2], q.shape[2], q.shape[0], q.stride(0), q.stride(1),
                           max_new, q.shape[2] ** -0.5)
    return misa.misa_attention_tree_workspace_bytes(shape, pages)


TREES = [   # lens, new, heads, kv heads, head_dim, page, e4m3, with the bound on new tokens
    ([9000], [16], 8, 2, 128, 64, False, True),                    # halves of the keys, one tree
    ([3000, 5000, 800], [12, 30, 1], 8, 2, 128, 64, False, False),   # both kernels
    ([700], [333], 4, 2, 64, 64, False, True),
    ([4000, 100, 2000], [16, 3, 9], 8, 2, 64, 16, True, True),
    ([6000, 5000, 1], [20, 18, 1], 6, 3, 128, 48, True, False),
    ([300, 900, 17, 2500], [3, 4, 2, 1], 8, 2, 128, 64, True, True),   # few rows alone
    ([2600, 1800], [9, 40], 40, 1, 64, 64, False, False),
]


def trees():
    out = []
    for i, (lens, new, heads, kv, dim, page, fp8, bound) in enumerate(TREES):
        p, mask = batch(50 + i, lens, new, heads, kv, dim, page, fp8)
        d = p.gpu()
        args = [d[k] for k in ("q", "k_pages", "v_pages", "block_table", "q_start", "kv_lens")]
        kw = dict(k_scale_pages=d["k_scale_pages"], v_scale_pages=d["v_scale_pages"], max_new=max(new) if bound else 0,
                  want_lse=True)
        out.append((p, d, args, mask, mask.cuda(), kw))
    return out


def test_trees_in_one_workspace():
    """Calls of different batches one after another in one buffer, eager, on a stream of its own and in graphs: each takes
    no more than it asks for, reads nothing that it has not written, and leaves the next one right."""
    calls = trees()
    needs = [tree_need(p, d, kw["max_new"]) for p, d, _, _, _, kw in calls]
    assert all(n > 0 for n in needs) and len(set(needs)) > 3
    s = Scratch(max(needs))
    want = []
    for (p, _, args, mask, m, kw), need in zip(calls, needs):
        out, lse = misa.misa_attention_tree(*args, m, ws=s.of(need), **kw)
        torch.cuda.synchronize()
        assert s.whole()
        th.check_attention(p, out, lse, mask)
        want.append((out, lse))
        with pytest.raises(misa.MisaError):
            misa.misa_attention_tree(*args, m, ws=s.of(need)[:need - 1], **kw)
    # without filling it anew, in another order, over what the call before left; then behind one another on two streams
    ready = torch.cuda.Event()
    for stream in (None, torch.cuda.Stream(), torch.cuda.Stream()):
        if stream is not None:
            ready.record()
            stream.wait_event(ready)
        for i in [*range(len(calls))[::-1], 0, 3, 1]:
            _, _, args, _, m, kw = calls[i]
            out, lse = misa.misa_attention_tree(*args, m, ws=s.buf[:needs[i]], stream=stream, **kw)
            if stream is not None:
                torch.cuda.current_stream().wait_stream(stream)
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])
    graphs = []
    for i, (_, _, args, _, m, kw) in enumerate(calls):
        kw = dict(kw, out=torch.zeros_like(want[i][0]), lse=torch.zeros_like(want[i][1]))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            misa.misa_attention_tree(*args, m, ws=s.buf[:needs[i]], **kw)
        graphs.append((g, kw))
    for order in (range(len(graphs)), range(len(graphs))[::-1], range(len(graphs))):
        for i in order:
            graphs[i][1]["out"].zero_(), graphs[i][1]["lse"].zero_()
            graphs[i][0].replay()
        torch.cuda.synchronize()
        s.buf[:max(needs)] = 0xFF
        for (_, kw), (out, lse) in zip(graphs, want):
            assert torch.equal(kw["out"], out) and torch.equal(kw["lse"], lse)


def test_products_in_one_workspace():
    sizes = [(64, 128, 8192), (500, 1003, 5008), (120, 500, 4112), (300, 65, 12304), (64, 128, 8192)]
    needs = [misa.misa_matmul_q8_workspace_bytes(*z) for z in sizes]
    assert all(n > 0 for n in needs)
    s = Scratch(max(needs))
    ops = [operands(60 + i, *z) for i, z in enumerate(sizes)]
    dev = [[t.cuda() for t in o] for o in ops]
    want = []
    for o, d, need in zip(ops, dev, needs):
        got = misa.misa_matmul_q8(*d, ws=s.of(need))
        torch.cuda.synchronize()
        assert s.whole()
        th.check_product(got, *o)
        assert torch.equal(got, misa.misa_matmul_q8(*d))
        want.append(got)
        with pytest.raises(misa.MisaError):
            misa.misa_matmul_q8(*d, ws=s.buf[:need - 1])
        with pytest.raises(misa.MisaError):
            misa.misa_matmul_q8(*d, ws=s.buf[4:need + 4])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    for i in (1, 0, 3, 2, 4):
        got = misa.misa_matmul_q8(*dev[i], ws=s.buf[:needs[i]], stream=stream)
        torch.cuda.current_stream().wait_stream(stream)
        assert torch.equal(got, want[i])
    outs = [torch.zeros_like(w) for w in want]
    graphs = []
    for i, d in enumerate(dev):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            misa.misa_matmul_q8(*d, out=outs[i], ws=s.buf[:needs[i]])
        graphs.append(g)
    for order in ((0, 1, 2, 3, 4), (4, 2, 0, 3, 1), (3, 1, 4, 0, 2)):
        for i in order:
            outs[i].zero_()
            graphs[i].replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


# ---------------------------------------------------------------- offsets past 32 bits

def apart(rows, cols, stride, dtype, fill):
    """[rows, cols] whose rows begin `stride` elements apart, the rest of the first and last ones' neighbourhood `fill`."""
    buf = torch.empty(rows * stride, dtype=dtype, device="cuda")
    view = buf.view(rows, stride)
    view[:, :cols + 64] = fill
    view[:, -64:] = fill
    return view


@pytest.mark.parametrize("m,n,k", [(1040, 1100, 272), (40, 1100, 1504), (1040, 33, 528), (300, 1050, 8208)])
def test_products_past_4_gib(m, n, k):
    """Rows of x, of w and of the output whose places pass 2^32 bytes (the output's 2^32 elements too, where it has more
    than 1024 rows): rows of codes as far apart as the call takes them, 4 MiB."""
    ops = operands(m + k, m, n, k)
    x8, xs, w8, ws = (t.cuda() for t in ops)
    far, ostride = 1 << 22, (1 << 22) + 40
    assert max(m, n) * far > 1 << 32 and (m <= 1024 or m * ostride > 1 << 32)
    x, w = (apart(r, k, far, torch.uint8, 0x7F) for r in (m, n))
    x[:, :k], w[:, :k] = x8, w8
    out = apart(m, n, ostride, torch.bfloat16, 7.0)
    got = misa.misa_matmul_q8(x[:, :k], xs, w[:, :k], ws, out=out[:, 8:8 + n])
    th.check_product(got, *ops)
    assert torch.equal(got, misa.misa_matmul_q8(x8, xs, w8, ws))
    assert (out[:, :8] == 7).all() and (out[:, 8 + n:n + 64] == 7).all() and (out[:, -64:] == 7).all()


def test_few_rows_past_4_gib():
    """The output's rows 2^28 elements apart: the places of k_matmul_rows' stores, and of its whole products."""
    m, n, k = 20, 70, 400
    ops = operands(71, m, n, k)
    out = apart(m, n, 1 << 28, torch.bfloat16, 7.0)
    got = misa.misa_matmul_q8(*(t.cuda() for t in ops), out=out[:, :n])
    th.check_product(got, *ops)
    assert (out[:, n:n + 64] == 7).all() and (out[:, -64:] == 7).all()


@pytest.mark.parametrize("m,n,k,stride", [(70, 40, 256, 16), (300, 130, 528, 144), (33, 70, 400, 0), (131, 300, 272, 0), (77, 4099, 272, 256)])
def test_products_of_rows_that_share_codes(m, n, k, stride):
    """x as windows of one run of codes, or one row for all; the codes behind the last window are NaN."""
    size = (m - 1) * stride + k
    x8 = th.quantize(torch.randn((1, -(-size // 16) * 16), generator=torch.Generator().manual_seed(m)), 1)[0]
    _, _, w8, ws = operands(m + n, 1, n, k)
    xs = 0.5 + torch.rand((m, -(-k // 128)), generator=torch.Generator().manual_seed(n))
    run = torch.full((size + 65536,), 0x7F, dtype=torch.uint8, device="cuda")
    run[:size] = x8[0, :size].cuda()
    rows = x8[0].as_strided((m, k), (stride, 1))
    got = misa.misa_matmul_q8(run.as_strided((m, k), (stride, 1)), xs.cuda(), w8.cuda(), ws.cuda())
    th.check_product(got, rows.contiguous(), xs, w8, ws)
    assert torch.equal(got, misa.misa_matmul_q8(rows.contiguous().cuda(), xs.cuda(), w8.cuda(), ws.cuda()))
