"""Where the paged serving operators can go wrong: every count of key splits, batches of many sequences, rows that
see nothing, NaN among the keys, pools past 4 GiB, dirty and shared workspaces, calls side by side.

Where two results are compared with each other, both come from the same arithmetic in the same order and are equal
to the last bit."""
import pytest
import torch

import long_context_sparse_block_amd as misa
import serving_helpers as ref
from long_context_sparse_block_amd._lib import MISA_K_BF16, MISA_K_FP8_E4M3
from gpu_helpers import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the -m gpu tests need an MI355X")
    misa.load()


def run(p, idx=None, **kw):
    d = p.gpu()
    if idx is None:
        return misa.misa_attention_paged(**d, want_lse=True, **kw)
    return misa.misa_attention_selected(**d, idx=idx.cuda(), want_lse=True, **kw)


def check(p, idx=None, **kw):
    out, lse = run(p, idx, **kw)
    torch.cuda.synchronize()
    ref.check_attention(p, out, lse, idx)
    return out, lse


# ---------------------------------------------------------------- key splits

# 512 keys make a split at these batch sizes; the join reads 2 or 4 splits at a time, so counts of every remainder
DECODE_SPLITS = [2, 3, 5, 9, 13, 17, 18, 19, 33, 34, 35, 36]


@pytest.mark.parametrize("dim,fp8", [(64, False), (64, True), (128, False), (128, True)])
def test_decode_split_counts(dim, fp8):
    say("decode splits", dim, fp8)
    lens = [512 * k - 7 * i for i, k in enumerate(DECODE_SPLITS)]
    check(ref.Paged(dim + fp8, lens, [1] * len(lens), 2, 1, dim, 64, fp8))


@pytest.mark.parametrize("dim,fp8", [(64, False), (128, False), (64, True)])
def test_chunk_split_counts(dim, fp8):
    say("chunk splits", dim, fp8)
    lens = [512 * k - 5 * i for i, k in enumerate([2, 3, 5, 9, 17, 18, 31])]
    check(ref.Paged(dim + 7 + fp8, lens, [9, 12, 9, 10, 9, 11, 9], 4, 1, dim, 64, fp8))


@pytest.mark.parametrize("topk", [129, 300, 515, 800, 1100, 1666, 2048, 4099])
@pytest.mark.parametrize("heads,dim", [(8, 64), (40, 64), (40, 128)])
def test_selected_split_counts(topk, heads, dim):
    say("selected splits", topk, heads, dim)
    p = ref.Paged(topk, [4500], [3], heads, 1, dim, 64)
    check(p, p.select(topk, 0.1))


# ---------------------------------------------------------------- batches

@pytest.mark.parametrize("n", [65, 300, 4200])
@pytest.mark.parametrize("chunks", [False, True])
def test_many_sequences(n, chunks):
    say("many sequences", n, chunks)
    g = torch.Generator().manual_seed(n)
    lens = torch.randint(0, 40, (n,), generator=g)
    new = (torch.rand((n,), generator=g) * 3).long().clamp(max=2)
    if chunks:
        far = torch.randperm(n, generator=g)[:6]
        lens[far] += 60
        new[far] = torch.tensor([40, 1, 33, 17, 60, 2])
    new = torch.minimum(new, lens)
    p = ref.Paged(n + 1, lens.tolist(), new.tolist(), 2, 1, 64, 8, width=13 if chunks else 600)
    check(p)
    check(p, p.select(5, 0.2))


def test_rows_that_see_nothing():
    # more new tokens than the sequence holds: the first ones stand before its start
    for lens, new in (([3, 0, 50], [5, 2, 1]), ([10, 700], [60, 1]), ([0], [40])):
        for fp8 in (False, True):
            p = ref.Paged(3, lens, new, 4, 2, 64, 16, fp8, width=200)
            out, lse = check(p)
            check(p, p.select(9))
            dead = max(new[0] - lens[0], 0)
            assert bool((out[:dead] == 0).all()) and bool((lse[:dead] == -float("inf")).all())


def test_lengths_past_the_table():
    p = ref.Paged(4, [160, 33], [1, 1], 8, 2, 128, 16, width=10)
    base = run(p)
    p.kv_lens = torch.tensor([165, 33], dtype=torch.int32)   # five tokens have no table entry
    for a, b in zip(run(p), base):
        assert torch.equal(a, b)


def test_no_tokens():
    p = ref.Paged(5, [30, 20], [0, 0], 4, 2, 64, 16)
    idx = torch.empty((0, 7), dtype=torch.int32)
    assert run(p)[0].shape == (0, 4, 64) and run(p, idx)[0].shape == (0, 4, 64)
    pages = torch.full((3, 4, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    misa.misa_write_pages(torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda"),
                          torch.empty((0,), dtype=torch.int64, device="cuda"), pages)
    f, _ = misa.rope_inv_freq(64)
    y = misa.misa_rope(torch.empty((0, 4, 64), device="cuda"), torch.empty((0,), dtype=torch.int32, device="cuda"), f)
    assert y.shape == (0, 4, 64) and bool((pages == 5).all())


# ---------------------------------------------------------------- NaN

def poison(p, which, b, tok):
    """NaN in one kv head's row of a token that its sequence holds."""
    page, r = int(p.table[b, tok // p.page]), tok % p.page
    if p.fp8:
        p.scale[which][page, r, 0] = float("nan")
    else:
        p.pages[which][page, r, 0, 3] = float("nan")


@pytest.mark.parametrize("which", [0, 1], ids=["key", "value"])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,new", [([400, 90], [1, 1]), ([5000, 60], [1, 1]), ([400, 90], [40, 1]), ([5000, 60], [40, 1])])
def test_nan_is_seen_by_those_who_see_it(lens, new, fp8, which):
    say("nan", lens, new, fp8, which)
    G = 4
    base = ref.Paged(6, lens, new, 2 * G, 2, 64, 16, fp8)
    clean, clean_lse = run(base)
    p = ref.Paged(6, lens, new, 2 * G, 2, 64, 16, fp8)
    poison(p, which, 0, 70)
    out, lse = run(p)
    m = new[0]
    # head group 0 of sequence 0 sees the row; other groups and sequences do not
    nan = torch.isnan(out[:m, :G])
    assert bool(nan.all()) if which == 0 or fp8 else bool(nan[..., 3].all())
    assert torch.equal(out[:m, G:], clean[:m, G:]) and torch.equal(out[m:], clean[m:])
    if which == 0:
        assert bool(torch.isnan(lse[:m, :G]).all())
    else:
        assert torch.equal(lse, clean_lse)
    # over selected tokens: those who list it
    idx = torch.arange(3, dtype=torch.int32).expand(p.tokens, 3).clone()
    plain = run(p, idx)[0]
    idx[0, 1] = 70
    out = run(p, idx)[0]
    assert not bool(torch.isnan(plain).any()) and bool(torch.isnan(out[0, :G, 3]).all())
    assert torch.equal(out[1:], plain[1:])


def test_nan_keys_ahead_stay_ahead():
    """A NaN in a new token's key does not reach the new tokens before it."""
    p = ref.Paged(7, [300], [50], 4, 2, 128, 16)
    want, want_lse, tol, ltol = ref.attention(p)
    poison(p, 0, 0, 280)   # the new token 30
    out, lse = (x.double().cpu() for x in run(p))
    assert bool(((out[:30] - want[:30]).abs() <= tol[:30]).all())
    assert bool(((lse[:30] - want_lse[:30]).abs() <= ltol[:30]).all())
    assert bool(torch.isnan(out[30:, :2]).all())
    assert bool(((out[30:, 2:] - want[30:, 2:]).abs() <= tol[30:, 2:]).all())


# ---------------------------------------------------------------- pools past 4 GiB

@pytest.mark.parametrize("fp8", [False, True])
def test_pool_past_4_gib(fp8):
    """Pages at the end of a large pool hold and give the same as in a small one."""
    say("large pool", fp8)
    page, KH, D = 64, 8, 128
    big, small = (70_000 if fp8 else 40_000), 12      # 4.6 and 5.2 GB a pool
    kind = torch.uint8 if fp8 else torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(1)
    lens, new = [300, 130, 70], [90, 1, 70]
    T = sum(new)
    q_start = torch.tensor([0, 90, 91, 161], dtype=torch.int32, device="cuda")
    kv = torch.tensor(lens, dtype=torch.int32, device="cuda")
    k, v = (torch.randn((sum(lens), KH, D), generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn((T, 32, D), generator=g, device="cuda").bfloat16()
    idx = torch.randint(0, 60, (T, 40), generator=g, device="cuda", dtype=torch.int32)
    got = []
    for n_pages in (small, big):
        pools = [torch.zeros((n_pages, page, KH, D), dtype=kind, device="cuda") for _ in range(2)]
        scales = [torch.zeros((n_pages, page, KH), device="cuda") if fp8 else None for _ in range(2)]
        ids = n_pages - 1 - torch.randperm(small, generator=torch.Generator().manual_seed(2))
        table = torch.zeros((3, 5), dtype=torch.int32)
        table[0, :5], table[1, :3], table[2, :2] = ids[:5], ids[5:8], ids[8:10]
        slots = torch.cat([table[b].long()[torch.arange(n) // page] * page + torch.arange(n) % page
                           for b, n in enumerate(lens)]).cuda()
        misa.misa_write_pages(k, slots, pools[0], scales[0], v=v, v_pages=pools[1], v_scale_pages=scales[1])
        at = (q, pools[0], pools[1], table.cuda(), q_start, kv)
        got.append((misa.misa_attention_paged(*at, *scales)[0], misa.misa_attention_selected(*at, idx, *scales)[0],
                    pools[0].view(-1, KH, D)[slots], pools[1].view(-1, KH, D)[slots]))
        del pools, scales
    torch.cuda.synchronize()
    for a, b in zip(*got):
        assert torch.equal(a, b)


# ---------------------------------------------------------------- workspaces, streams, graphs

def batches():
    dec = ref.Paged(8, [5003, 2111, 40], [1, 1, 1], 16, 2, 128, 64)
    mix = ref.Paged(9, [4100, 300, 70], [70, 1, 20], 8, 2, 64, 16, True)
    sel = ref.Paged(10, [3000, 80], [2, 1], 8, 1, 128, 64, True)
    big = ref.Paged(11, [2500], [2], 66, 1, 64, 64)
    return [(dec, None), (mix, None), (sel, sel.select(2048)), (big, big.select(2000))]


def ws_bytes(p, idx):
    kd = MISA_K_FP8_E4M3 if p.fp8 else MISA_K_BF16
    shape = misa.AttnShape(len(p.kv_lens), p.heads, p.kv_heads, p.dim, p.tokens, 0, 0, 0, 1.0)
    pages = misa.KvPages(None, None, None, None, None, p.width, p.pages[0].shape[0], p.page, kd)
    if idx is None:
        return misa.misa_attention_paged_workspace_bytes(shape, pages)
    return misa.misa_attention_selected_workspace_bytes(shape, pages, idx.shape[1])


def test_dirty_workspace_changes_nothing():
    for p, idx in batches():
        base = run(p, idx)
        n = ws_bytes(p, idx)
        assert n > 0   # these batches split their keys
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN throughout
        for _ in range(2):
            for a, b in zip(run(p, idx, ws=ws), base):
                assert torch.equal(a, b)


def test_two_streams_at_once():
    jobs = batches()
    base = [run(p, i) for p, i in jobs]
    dev = [(p.gpu(), None if i is None else i.cuda()) for p, i in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = []
    for _ in range(5):
        for (d, i), s in zip(dev, streams):
            with torch.cuda.stream(s):
                got.append(misa.misa_attention_paged(**d) if i is None else misa.misa_attention_selected(**d, idx=i))
    torch.cuda.synchronize()
    for n, (out, _) in enumerate(got):
        assert torch.equal(out, base[n % len(jobs)][0])


def test_two_graphs_share_a_workspace():
    jobs = batches()[:2]
    base = [run(p, i) for p, i in jobs]
    ws = torch.empty((max(ws_bytes(p, i) for p, i in jobs),), dtype=torch.uint8, device="cuda")
    dev = [p.gpu() for p, _ in jobs]
    outs = [torch.empty_like(b[0]) for b in base]
    for d, o in zip(dev, outs):
        misa.misa_attention_paged(**d, out=o, ws=ws)
    torch.cuda.synchronize()
    graphs = []
    for d, o in zip(dev, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            misa.misa_attention_paged(**d, out=o, ws=ws)
        graphs.append(g)
    for rep in range(4):
        for n in (0, 1, 1, 0):
            outs[n].fill_(3)
            graphs[n].replay()
            torch.cuda.synchronize()
            assert torch.equal(outs[n], base[n][0]), (rep, n)
            ws.fill_(rep)
            assert torch.equal(run(*jobs[n])[0], base[n][0])


# ---------------------------------------------------------------- plans of many sequences

@pytest.mark.parametrize("n,page,most,live", [(1024, 16, 3, 1.0), (1025, 16, 3, 1.0), (1537, 64, 400, 0.1), (5000, 8, 1, 0.05),
                                              (65535, 32, 2, 0.5), (65535, 32, 0, 0.0)])
@pytest.mark.parametrize("hold", [0, 50])
def test_plan_of_many_sequences(n, page, most, live, hold):
    """Runs of sequences without new tokens, tokens of a workgroup in many runs, and a free list that runs out."""
    say("plan", n, page, most, live, hold)
    g = torch.Generator().manual_seed(n + hold)
    cached = torch.randint(0, 100, (n,), generator=g)
    new = torch.randint(0, most + 1, (n,), generator=g) * (torch.rand((n,), generator=g) < live)
    width = int((-(-(cached + new) // page)).max()) + 1
    have = -(-cached // page)
    ids = torch.randperm(int(have.sum()) + n + 10, generator=g).to(torch.int32)
    table = torch.full((n, width), -7, dtype=torch.int32)
    table[torch.arange(width)[None, :] < have[:, None]] = ids[:int(have.sum())]
    need = int((-(-(cached + new) // page) - have).sum())
    free = ids[int(have.sum()):][:max(0, need - hold)].contiguous()
    T = int(new.sum()) + 30
    want = ref.plan(cached.tolist(), new.tolist(), free.tolist(), table, page, T)
    t = table.cuda()
    i32 = torch.int32
    got = misa.misa_plan_pages(cached.to(i32).cuda(), new.to(i32).cuda(), free.cuda(), t, page, T)
    torch.cuda.synchronize()
    assert t.tolist() == want["table"]
    assert got.q_start.tolist() == want["q_start"] and got.kv_lens.tolist() == want["kv_lens"]
    assert got.positions.tolist() == want["positions"] and got.slots.tolist() == want["slots"]
    assert got.n_taken.tolist() == want["n_taken"]


# ---------------------------------------------------------------- codes of rotated rows

@pytest.mark.parametrize("layout,start", [("half", 0), ("half", 3), ("interleaved", 16)])
def test_rotated_codes_are_those_of_the_true_values(layout, start):
    """Scales and codes are one fp32 quotient of the rotated row each, rounded once.  A quotient within the fp64 error of
    the rotation (2^-50 for these angles) of an fp32 border is met once in about 2^25 values, so 13 million codes and
    100 000 scales come out equal but for at most one of either, by a step."""
    say("rotated codes", layout, start)
    T, H, D, rot = 12800, 8, 128, 32
    g = torch.Generator(device="cuda").manual_seed(5)
    k = torch.randn((T, H, D), generator=g, device="cuda").bfloat16()
    pos = torch.randint(0, 64, (T,), generator=g, device="cuda", dtype=torch.int32)
    f, _ = misa.rope_inv_freq(rot)
    pages = torch.zeros((T // 64, 64, H, D), dtype=torch.uint8, device="cuda")
    scale = torch.zeros((T // 64, 64, H), device="cuda")
    misa.misa_write_pages(k, torch.arange(T, device="cuda"), pages, scale, positions=pos, inv_freq=f, layout=layout,
                          rot_start=start)
    want = ref.rope(k.cpu(), pos.cpu(), f.cpu(), layout, start, 1.0).cuda()
    sc = (want.abs().amax(-1) / 448).float()
    codes = (want / sc.double()[..., None]).float().to(torch.float8_e4m3fn).view(torch.uint8)
    assert int((scale.view(T, H) != sc).sum()) <= 1
    assert int((pages.view(T, H, D) != codes).sum()) <= 1


# ---------------------------------------------------------------- argument checks

def outcome(check, *args):
    try:
        return check(*args)
    except ValueError as e:
        return str(e)


def test_built_argument_checks_equal_the_plain_ones():
    from long_context_sparse_block_amd import serving
    x = torch.zeros((5, 4, 8), device="cuda")
    one = torch.zeros((1, 1, 8), device="cuda")
    for t in (x, x.half(), x[:, ::2], x[..., ::2], x.transpose(0, 1), x[:0], x[0], one, one.expand(5, 1, 8), x[:, :, :1]):
        for dtype in (torch.float32, torch.int32):
            for shape in ((5, 4, 8), (5, 4), x.shape, t.shape, (5, 4, 9), ()):
                args = (t, dtype, shape, "x", 0)
                assert outcome(serving._dense, *args) == outcome(serving._dense_py, *args), args[1:]
        for dtypes in ((torch.float32,), (torch.bfloat16, torch.float16), {torch.float32: 2}):
            for shape in (None, x.shape, (5, 4, 9)):
                args = (t, dtypes, "x", 0, shape)
                assert outcome(serving._rows, *args) == outcome(serving._rows_py, *args), args[1:]
    for t in (x, x.bfloat16(), x.byte()[None], x.bfloat16()[None], x.bfloat16()[None].transpose(1, 2),
              x.to(torch.float8_e4m3fn)[None], x.bfloat16()[0], x.bfloat16()[0, 0]):
        for heads, dim in ((4, 8), (1, 8), (5, 4), (4, 4)):
            args = (t, heads, dim, "x", 0)
            assert outcome(serving._pool, *args) == outcome(serving._pool_py, *args), (t.shape, args[1:])
    ws, at = serving._scratch(1000, x)
    assert ws.shape == (1000,) and ws.dtype == torch.uint8 and ws.device == x.device and at == ws.data_ptr()
    assert "cuda:1" in outcome(serving._pool, x.bfloat16(), 1, 8, "x", 1)
    assert "cuda:1" in outcome(serving._dense, x, torch.float32, (5, 4, 8), "x", 1)
    assert "cuda:1" in outcome(serving._rows, x, (torch.float32,), "x", 1)
