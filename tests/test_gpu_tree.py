"""Trees of drafted tokens on the GPU: their plan, attention over them and the move of a kept path, against 64-bit
forms."""
import math

import pytest
import torch

import long_context_sparse_block_amd as misa
import tree_helpers as th
from serving_helpers import Paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the -m gpu tests need an MI355X")
    misa.load()


def starts(new, at=0):
    out = [at]
    for m in new:
        out.append(out[-1] + m)
    return out


PLANS = {
    "one": ([1], "tree", 1, 0, 0),
    "some": ([5, 0, 1, 33, 32, 31, 0], "tree", 2, 3, 0),
    "chains": ([64, 7, 65], "chain", 3, 0, 0),
    "stars": ([40, 2], "star", 2, 20, 0),
    "forest": ([9, 1], "forest", 1, 0, 0),
    "rows_in_front": ([6, 4], "tree", 1, 5, 3),
    "past_the_words": ([100, 40], "tree", 1, 0, 0),
    "past_the_lds": ([2100], "chain", 66, 1, 0),
    "large": ([700, 300], "tree", 23, 9000, 0),
    "many": ([i % 5 for i in range(300)], "tree", 1, 40, 0),
    "padded_more_than_filled": ([3, 0, 2], "tree", 2, 70000, 9),
}


@pytest.mark.parametrize("name", PLANS)
def test_plan(name):
    new, kind, words, pad, front = PLANS[name]
    g = torch.Generator().manual_seed(7)
    parents = [5] * front
    for m in new:
        parents += th.random_parents(g, m, kind)
    parents += [3] * pad
    q_start = starts(new, front)
    lens = [m + int(torch.randint(0, 5000, (1,), generator=g)) for m in new]
    T = len(parents)
    mask, pos = th.plan(parents, q_start, lens, T, words)
    i32 = dict(dtype=torch.int32, device="cuda")
    args = torch.tensor(parents, **i32), torch.tensor(q_start, **i32), torch.tensor(lens, **i32), words
    dirty = misa.TreePlan(torch.full((T, words), 77, **i32), torch.full((T,), 77, **i32))
    for p in (misa.misa_plan_tree(*args), misa.misa_plan_tree(*args, plan=dirty)):
        assert torch.equal(p.mask.cpu(), mask)
        assert torch.equal(p.positions.cpu(), pos)


def test_plan_of_parents_that_name_no_earlier_token():
    parents = [-1, 0, 2, 9, -7, 3, 2 ** 31 - 1, -2 ** 31, 6]   # 2: itself, 9: later, the rest: nobody
    want = th.ancestors(parents)
    assert want.sum(1).tolist() == [1, 2, 1, 1, 1, 2, 1, 1, 2]
    i32 = dict(dtype=torch.int32, device="cuda")
    p = misa.misa_plan_tree(torch.tensor(parents, **i32), torch.tensor([0, 9], **i32), torch.tensor([9], **i32), 1)
    assert torch.equal(p.mask.cpu(), th.pack(want, 1))
    assert p.positions.tolist() == [0, 1, 0, 0, 0, 1, 0, 0, 1]


def batch(seed, lens, new, heads, kv, dim, page, fp8, kind="tree", words=None, **kw):
    p = Paged(seed, lens, new, heads, kv, dim, page, fp8, **kw)
    g = torch.Generator().manual_seed(seed + 1)
    parents = sum((th.random_parents(g, m, kind) for m in new), []) + [0] * (p.q.shape[0] - p.tokens)
    words = max(1, -(-max(new) // 32)) if words is None else words
    mask, _ = th.plan(parents, p.q_start.tolist(), lens, p.q.shape[0], words)
    return p, mask


def attend(p, mask, **kw):
    d = p.gpu()
    order = ("q", "k_pages", "v_pages", "block_table", "q_start", "kv_lens")
    return misa.misa_attention_tree(*(d[k] for k in order), mask.cuda(), d["k_scale_pages"], d["v_scale_pages"],
                                    want_lse=True, **kw)


CASES = {   # lens, new, heads, kv heads, page
    "decode": ([100, 33, 1, 64], [1, 1, 1, 1], 8, 2, 16),
    "no_prefix": ([5, 40, 130, 1], [5, 40, 130, 1], 4, 4, 64),
    "few_rows": ([300, 900, 17], [3, 4, 2], 8, 2, 64),
    "rows_16_17": ([64, 65, 200], [4, 5, 4], 8, 2, 64),
    "rows_33": ([129, 700], [33, 8], 4, 4, 48),
    "rows_65": ([500, 1000, 66], [17, 0, 65], 12, 3, 16),
    "long_splits": ([9000, 4000], [20, 31], 8, 2, 64),
    "word_edges": ([95, 96, 97, 128, 161], [31, 32, 33, 64, 97], 2, 2, 32),
    "group_of_40": ([333, 77], [3, 9], 40, 1, 16),
    "one_long_tree": ([700], [333], 4, 2, 64),
    "rows_64": ([9000], [16], 8, 2, 64),                        # at most 64 rows of a kv head, cut in splits
    "rows_64_short": ([16, 30, 45, 97, 64, 20], [16, 15, 1, 12, 9, 16], 8, 2, 16),   # the same, some over one half of a tile's keys
    "rows_20_of_40": ([6000, 5000, 1], [20, 18, 1], 6, 3, 64),
}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("name", CASES)
def test_attention(name, dim, fp8):
    lens, new, heads, kv, page = CASES[name]
    p, mask = batch(11, lens, new, heads, kv, dim, page, fp8)
    out, lse = attend(p, mask)
    th.check_attention(p, out, lse, mask)
    bound, _ = misa.misa_attention_tree(*(p.gpu()[k] for k in ("q", "k_pages", "v_pages", "block_table", "q_start",
                                                               "kv_lens")), mask.cuda(), p.gpu()["k_scale_pages"],
                                        p.gpu()["v_scale_pages"], max_new=max(new))
    th.check_attention(p, bound, lse, mask)


@pytest.mark.parametrize("dim,fp8", [(64, False), (128, True)])
@pytest.mark.parametrize("name", ["few_rows", "rows_33", "word_edges", "no_prefix", "rows_64_short"])
def test_attention_under_any_mask(name, dim, fp8):
    """Masks that no tree gives: a token without itself, without anything, with later ones, bits behind the sequence's
    tokens; and words more than needed."""
    lens, new, heads, kv, page = CASES[name]
    p, mask = batch(13, lens, new, heads, kv, dim, page, fp8, words=4)
    g = torch.Generator().manual_seed(5)
    mask = torch.randint(-2 ** 31, 2 ** 31, mask.shape, generator=g).to(torch.int32)
    mask[::3] = 0
    out, lse = attend(p, mask)
    th.check_attention(p, out, lse, mask)
    if name == "no_prefix":
        assert (lse[0] == -math.inf).all() and (out[0] == 0).all()


def test_words_that_do_not_reach_all_tokens():
    p, mask = batch(17, [200, 90], [70, 20], 4, 2, 128, 16, False, words=1)
    out, lse = attend(p, mask)
    th.check_attention(p, out, lse, mask)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [[3, 2], [40, 129]])
def test_a_chain_is_causal_attention(new, fp8):
    lens = [400, 1300]
    p, mask = batch(19, lens, new, 8, 2, 128, 64, fp8, kind="chain")
    out, lse = attend(p, mask)
    d = p.gpu()
    ref, rl = misa.misa_attention_paged(**d, want_lse=True)
    assert torch.equal(out, ref) and torch.equal(lse, rl)


def test_scale_strides_padding_and_lse():
    p, mask = batch(23, [150, 40, 3], [9, 0, 3], 6, 3, 64, 16, False, pad_rows=5)
    d = p.gpu()
    wide = torch.full((p.q.shape[0], 8, 72), float("nan"), dtype=torch.bfloat16, device="cuda")
    q = wide[:, 1:7, :64]
    q.copy_(d["q"])
    out = torch.full((p.q.shape[0], 6, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((p.q.shape[0], 6), 7.0, device="cuda")
    for scale in (-0.3, 0.05):
        misa.misa_attention_tree(q, d["k_pages"], d["v_pages"], d["block_table"], d["q_start"], d["kv_lens"], mask.cuda(),
                                 scale=scale, out=out, lse=lse, max_new=9)
        th.check_attention(p, out, lse, mask, scale=scale)
        assert (out[p.tokens:] == 7).all() and (lse[p.tokens:] == 7).all()


def test_other_sequences_never_see_a_bad_draft():
    """NaN in one sequence's drafted keys and values stays in that sequence."""
    p, mask = batch(29, [100, 100, 100], [6, 6, 6], 4, 2, 128, 16, False)
    clean, _ = attend(p, mask)
    for t in range(94, 100):
        e = int(p.table[1, t // 16])
        p.pages[0][e, t % 16] = float("nan")
        p.pages[1][e, t % 16] = float("nan")
    out, _ = attend(p, mask)
    assert torch.equal(out[:6], clean[:6]) and torch.equal(out[12:], clean[12:])
    assert out[6:12].isnan().any()


def test_lengths_past_the_table_and_below_the_new_tokens():
    """Positions are those of the true length; keys without an entry are not read; a length below the count of new
    tokens (no caller's plan) faults nothing."""
    p, mask = batch(31, [64, 64], [4, 4], 4, 2, 64, 16, False)
    d = p.gpu()
    order = ("q", "k_pages", "v_pages", "block_table", "q_start", "kv_lens")
    d["kv_lens"] = torch.tensor([100, 2], dtype=torch.int32, device="cuda")
    out, lse = misa.misa_attention_tree(*(d[k] for k in order), mask.cuda(), want_lse=True)
    # sequence 0: 96 cached tokens, of which the table holds 64, and no new one; all rows see these 64
    k, v = p.rows(0, 0, torch.arange(64)), p.rows(1, 0, torch.arange(64))
    for h in range(4):
        s = p.q[:4, h].double() @ k[:, h // 2].T / 8
        assert torch.allclose(lse[:4, h].double().cpu(), torch.logsumexp(s, 1), rtol=0, atol=1e-5)
    assert torch.isfinite(out[:4]).all()
    # sequence 1: new tokens at positions -2 .. 1: what is at 0 and 1 are its third and fourth
    sees = th.unpack(mask)[4:8, 2:4]
    assert torch.equal((lse[4:8] == -math.inf).all(1).cpu(), ~sees.any(1))


def test_graph_streams_and_shared_workspace():
    p, mask = batch(37, [3000, 5000, 800], [12, 30, 1], 8, 2, 128, 64, False)
    d = p.gpu()
    m = mask.cuda()
    parents = torch.tensor([0] * p.tokens, dtype=torch.int32, device="cuda")
    args = [d[k] for k in ("q", "k_pages", "v_pages", "block_table", "q_start", "kv_lens")]
    ref, rl = misa.misa_attention_tree(*args, m, want_lse=True)
    want = misa.misa_plan_tree(parents, d["q_start"], d["kv_lens"], 1)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        out, lse = torch.zeros_like(ref), torch.zeros_like(rl)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            tree = misa.misa_plan_tree(parents, d["q_start"], d["kv_lens"], 1)
            misa.misa_attention_tree(*args, m, out=out, lse=lse)
        graphs.append((graph, out, lse, tree))
    for _ in range(3):
        for graph, out, lse, tree in graphs:
            out.zero_(), lse.zero_(), tree.mask.zero_()
            graph.replay()
        ref2, _ = misa.misa_attention_tree(*args, m)
        torch.cuda.synchronize()
        for _, out, lse, tree in graphs:
            assert torch.equal(out, ref) and torch.equal(lse, rl)
            assert torch.equal(tree.mask, want.mask) and torch.equal(tree.positions, want.positions)
        assert torch.equal(ref2, ref)
    # a replay with other lengths, on another stream
    other = torch.cuda.Stream()
    d["kv_lens"].copy_(torch.tensor([2000, 4000, 1], dtype=torch.int32))
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        graphs[0][0].replay()
    out, lse = misa.misa_attention_tree(*args, m, want_lse=True, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert torch.equal(out, graphs[0][1]) and torch.equal(lse, graphs[0][2])


KEEP = {   # paths, new tokens
    "some": ([[0, 3, 4, 7], [0, 1, 2, -1], [2, 5, -1, -1], [-1, 0, 1, 2]], [8, 3, 6, 4]),
    "shift_by_one": ([[1, 2, 3, 4, 5, 6, 7, 8, 9, 10]], [11]),
    "not_rising": ([[0, 2, 2, 5], [3, 1, 4, 5], [0, 6, 7, 8], [-5, 1, 2, 3]], [7, 7, 7, 7]),
    "past_the_tokens": ([[0, 2, 5], [0, 2, 5], [0, 0, 0]], [5, 6, 0]),
    "long": ([[2 * i for i in range(100)], list(range(3, 103))], [200, 150]),
    "groups_of_64": ([list(range(1, 66)) + [-1] * 65, list(range(64)) + [70] + [-1] * 65, list(range(2, 132))], [140] * 3),
}


@pytest.mark.parametrize("form", ["bf16", "e4m3", "index_keys", "rows_of_8"])
@pytest.mark.parametrize("name", KEEP)
def test_keep_path(name, form):
    paths, new = KEEP[name]
    heads, dim, page, fp8, values = dict(bf16=(3, 64, 16, False, True), e4m3=(2, 128, 20, True, True),
                                         index_keys=(1, 128, 64, True, False), rows_of_8=(3, 8, 7, True, True))[form]
    g = torch.Generator().manual_seed(3)
    lens = [m + int(torch.randint(0, 100, (1,), generator=g)) for m in new]
    n, width = len(new), max(-(-x // page) for x in lens)
    pages = n * width + 2
    table = torch.randperm(pages, generator=g)[:n * width].to(torch.int32).view(n, width)
    pools = []
    for _ in range(2 if values else 1):
        shape = (pages, page, heads, dim)
        pools.append(torch.randint(0, 256, shape, generator=g).to(torch.uint8) if fp8
                     else torch.randn(shape, generator=g).bfloat16())
        if fp8:
            pools.append(torch.rand(shape[:3], generator=g))
    path = torch.tensor(paths, dtype=torch.int32)
    q_start = torch.tensor(starts(new), dtype=torch.int32)
    want, kept = th.keep(path, q_start, lens, table, page, pools)
    got = [x.cuda() for x in pools]
    if form == "index_keys":   # the pools may leave one head out
        got[0] = got[0].view(pages, page, dim)
        got[1] = got[1].view(pages, page)
    k, ks = got[0], got[1] if fp8 else None
    v, vs = (got[2] if fp8 else got[1], got[3] if fp8 else None) if values else (None, None)
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    r = misa.misa_keep_path(path.cuda(), q_start.cuda(), lens_t, table.cuda(), k, ks, v, vs)
    assert r.tolist() == kept
    for x, y in zip(got, want):
        assert torch.equal(x.cpu().view(y.shape), y)


def test_keep_path_leaves_what_has_no_page():
    page, heads, dim = 4, 2, 64
    k = torch.randn((6, page, heads, dim)).bfloat16()
    table = torch.tensor([[0, -1, 9, 2], [1, 3, 4, 5]], dtype=torch.int32)   # entries 1 and 2 of the first name no page
    path = torch.tensor([[2, 6, 9, 13], [1, 2, 9, 13]], dtype=torch.int32)
    q_start, lens = torch.tensor([0, 14, 28], dtype=torch.int32), [16, 24]   # the second's end is past its table
    want, kept = th.keep(path, q_start, lens, table, page, [k])
    got = k.cuda()
    r = misa.misa_keep_path(path.cuda(), q_start.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), table.cuda(), got)
    assert r.tolist() == kept == [6, 14]
    assert torch.equal(got.cpu(), want[0])


def test_refused_calls_raise():
    i32 = dict(dtype=torch.int32, device="cuda")
    up, qs, kv = torch.zeros(4, **i32), torch.tensor([0, 4], **i32), torch.tensor([9], **i32)
    with pytest.raises(ValueError, match="q_start"):
        misa.misa_plan_tree(up, qs[:1], kv, 1)
    with pytest.raises(ValueError, match="mask"):
        misa.misa_plan_tree(up, qs, kv, 2, plan=misa.TreePlan(torch.zeros((4, 1), **i32), up.clone()))
    with pytest.raises(misa.MisaError):
        misa.misa_plan_tree(up, qs, kv, 0)
    with pytest.raises(misa.MisaError):
        misa.misa_plan_tree(up, qs, kv, 1, plan=misa.TreePlan(torch.zeros((4, 1), **i32), up))
    p, mask = batch(41, [20], [4], 4, 2, 64, 16, False)
    d = p.gpu()
    args = [d[k] for k in ("q", "k_pages", "v_pages", "block_table", "q_start", "kv_lens")]
    for bad in (None, mask.cuda()[:3], mask.cuda().long(), mask, mask.cuda().float()):
        with pytest.raises(ValueError, match="mask"):
            misa.misa_attention_tree(*args, bad)
    path = torch.zeros((1, 2), **i32)
    with pytest.raises(misa.MisaError):
        misa.misa_keep_path(path, d["q_start"], d["kv_lens"], d["block_table"], d["k_pages"], kept_lens=d["kv_lens"])
    with pytest.raises(misa.MisaError):
        misa.misa_keep_path(path, d["q_start"], d["kv_lens"], d["block_table"], d["k_pages"], v_pages=d["k_pages"])
    with pytest.raises(ValueError, match="path"):
        misa.misa_keep_path(path.long(), d["q_start"], d["kv_lens"], d["block_table"], d["k_pages"])
    with pytest.raises(ValueError, match="v_pages"):
        misa.misa_keep_path(path, d["q_start"], d["kv_lens"], d["block_table"], d["k_pages"], v_pages=d["v_pages"][:1])
