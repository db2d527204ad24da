"""NaN and infinities among the keys and values of the paged attention calls: a row shows those that it sees, however
its keys are split, and none that it does not."""
import math

import pytest
import torch

import long_context_sparse_block_amd as misa
import serving_helpers as ref
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


def rows_of(p, b, toks):
    toks = torch.as_tensor(list(toks), dtype=torch.long)
    return p.table[b].long()[toks // p.page], toks % p.page


def poison(p, which, b, toks, head=0, value=float("nan")):
    """`value` in a kv head's rows (head None: all heads') of tokens that sequence b holds."""
    page, r = rows_of(p, b, toks)
    heads = range(p.kv_heads) if head is None else [head]
    for h in heads:
        if p.fp8:
            p.scale[which][page, r, h] = value
        else:
            p.pages[which][page, r, h, 3] = value


# ---------------------------------------------------------------- key splits

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [1, 40])
def test_nan_through_whole_splits(new, fp8):
    """NaN keys from the sequence's start on, 32 more each time: some of these runs are whole key splits, beside clean
    ones, wherever the splits are cut."""
    say("nan splits", new, fp8)
    p = ref.Paged(21, [4608, 300], [new, 1], 8, 2, 64, 16, fp8, width=600)
    clean, clean_lse = run(p)
    for n in range(32, 2400, 32):
        poison(p, 0, 0, range(n - 32, n))
        out, lse = run(p)
        assert bool(torch.isnan(out[:new, :4]).all()) and bool(torch.isnan(lse[:new, :4]).all()), n
        assert torch.equal(out[:new, 4:], clean[:new, 4:]) and torch.equal(out[new:], clean[new:]), n
        assert torch.equal(lse[:new, 4:], clean_lse[:new, 4:]) and torch.equal(lse[new:], clean_lse[new:]), n


def test_nan_in_the_only_key_of_a_split():
    p = ref.Paged(24, [4609, 300], [1, 1], 8, 2, 64, 16, width=600)
    clean, _ = run(p)
    poison(p, 0, 0, [4608])
    out, lse = run(p)
    assert bool(torch.isnan(out[0, :4]).all()) and bool(torch.isnan(lse[0, :4]).all())
    assert torch.equal(out[0, 4:], clean[0, 4:]) and torch.equal(out[1], clean[1])


@pytest.mark.parametrize("heads", [8, 40])
@pytest.mark.parametrize("dim,fp8", [(64, False), (128, True)])
def test_nan_through_whole_splits_of_a_list(dim, fp8, heads):
    say("nan splits of a list", dim, fp8, heads)
    p = ref.Paged(22, [4500], [2], heads, 1, dim, 64, fp8)
    poison(p, 0, 0, range(1400))
    clean = torch.arange(1400, 1400 + 2048, dtype=torch.int32)
    for n in range(32, 1400, 32):
        idx = clean.expand(2, 2048).clone()
        idx[0, :n] -= 1400
        out, lse = run(p, idx)
        assert bool(torch.isnan(out[0]).all()) and bool(torch.isnan(lse[0]).all()), n
        assert bool(torch.isfinite(out[1]).all()) and bool(torch.isfinite(lse[1]).all()), n


@pytest.mark.parametrize("which", [0, 1], ids=["key", "value"])
@pytest.mark.parametrize("new", [1, 40])
def test_nan_among_keys_far_below_the_maximum(new, which):
    """A NaN in a key range whose scores lie hundreds under the others': its weights are 0 in 32 bits, NaN stays."""
    say("nan far below", new, which)
    p = ref.Paged(23, [4700], [new], 4, 1, 64, 16)
    p.q.fill_(2.0)
    page, r = rows_of(p, 0, range(4700))
    p.pages[0][page, r] = 0.0
    page, r = rows_of(p, 0, range(2400, 4700))
    p.pages[0][page, r] = 2.5                     # scores 320, the others 0
    poison(p, which, 0, [70])
    out, lse = run(p, scale=1.0)
    assert bool(torch.isnan(out[:, :, 3]).all())
    assert bool(torch.isnan(lse).all()) == (which == 0)


# ---------------------------------------------------------------- entries that are absent

@pytest.mark.parametrize("bad", ["nan", "inf"])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,kv_heads,dim,topk", [(8, 2, 128, 77), (8, 2, 64, 1101), (40, 1, 128, 300), (70, 1, 64, 2048)])
def test_a_token_that_no_list_names_reaches_no_row(heads, kv_heads, dim, topk, fp8, bad):
    """Lists with holes, of lengths that end inside a tile, one with nothing in it, none with token 0 or a token of its
    page: what that page holds, and which page the table names for it, changes nothing."""
    say("unlisted", heads, kv_heads, dim, topk, fp8, bad)
    def make():
        p = ref.Paged(25, [2300, 60], [4, 1], heads, kv_heads, dim, 16, fp8)
        idx = p.select(topk, 0.3)
        idx[idx < 16] = -1
        idx[2] = -1
        idx[3, 64:] = -1      # whole tiles without an entry
        idx[3, :5] = torch.tensor([-1, 100000, 17, -7, 2299])
        at = int(p.table[0, 0])   # let that page be the pool's first
        was = p.table.clone()
        p.table[was == 0], p.table[was == at] = at, 0
        for rows in (p.pages, p.vals) + ((p.scale, p.codes) if fp8 else ()):
            for x in rows:
                first = x[0].clone()
                x[0], x[at] = x[at].clone(), first
        return p, idx
    p, idx = make()
    want = run(p, idx)
    ref.check_attention(p, *want, idx)
    for which in (0, 1):
        for b in (0, 1):
            poison(p, which, b, range(16), head=None, value=float(bad))
    for a, b in zip(run(p, idx), want):
        assert torch.equal(a, b)
    # the page was given back: another sequence's, or none
    for entry in (-1, 10 ** 6, 0):
        p.table[:, 0] = entry
        p.pages[0][0].view(torch.uint8).fill_(0x7F)
        p.pages[1][0].view(torch.uint8).fill_(0x7F)
        for a, b in zip(run(p, idx), want):
            assert torch.equal(a, b)


# ---------------------------------------------------------------- infinities

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [1, 40])
def test_an_infinite_value_shows_where_it_is_seen(new, fp8):
    """Infinite or NaN (a weight's second part may be 0) in the elements it enters, nothing elsewhere."""
    say("infinite value", new, fp8)
    p = ref.Paged(26, [400, 90], [new, 1], 8, 2, 64, 16, fp8)
    clean, clean_lse = run(p)
    poison(p, 1, 0, [70], value=math.inf)
    out, lse = run(p)
    bad = ~torch.isfinite(out[:new, :4])
    assert bool(bad.all()) if fp8 else bool(bad[..., 3].all()) and int(bad.sum()) == new * 4
    assert torch.equal(out[:new, 4:], clean[:new, 4:]) and torch.equal(out[new:], clean[new:]) and torch.equal(lse, clean_lse)


@pytest.mark.parametrize("new", [1, 40])
def test_infinite_scores(new):
    """A score of plus infinity gives NaN in out and lse; one of minus infinity is a weight of 0."""
    say("infinite score", new)
    p = ref.Paged(27, [400, 90], [new, 1], 8, 2, 64, 16)
    p.q[:new, :4, 3] = 1.0
    want = run(p)
    poison(p, 0, 0, [70], value=math.inf)
    out, lse = run(p)
    assert bool(torch.isnan(out[:new, :4]).all()) and bool(torch.isnan(lse[:new, :4]).all())
    assert torch.equal(out[:new, 4:], want[0][:new, 4:]) and torch.equal(out[new:], want[0][new:])
    poison(p, 0, 0, [70], value=-math.inf)
    idx = torch.arange(400, dtype=torch.int32).expand(p.tokens, 400).clone()
    without = idx.clone()
    without[:, 70] = -1
    out, lse = run(p)
    picked, picked_lse = run(p, idx)
    want, want_lse, tol, ltol = ref.attention(p, without)
    for o, l in ((out, lse), (picked, picked_lse)):
        o, l = o.double().cpu()[:new, :4], l.double().cpu()[:new, :4]
        assert bool(((o - want[:new, :4]).abs() <= tol[:new, :4]).all())
        assert bool(((l - want_lse[:new, :4]).abs() <= ltol[:new, :4]).all())
