"""Lengths at the edges of what the paged attention calls take: past the block table, many key splits of few and of
many sequences."""
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


@pytest.mark.parametrize("new", [4, 20])
def test_new_tokens_past_the_table(new):
    """Positions follow the true length, as in the page plan; keys without a table entry are not read.  Here 160 keys
    have one, and the new tokens stand at 165 - new ..: a row at 160 or later sees all 160."""
    say("past the table", new)
    p = ref.Paged(41, [160], [new], 8, 2, 128, 16, width=10)
    p.kv_lens = torch.tensor([165], dtype=torch.int32)
    out, lse = run(p)
    lists = torch.arange(200, dtype=torch.int32).expand(new, 200).clone()
    picked, picked_lse = run(p, lists)
    # the same rows as decodes, a sequence each, of the keys that they see
    pos = [p.pos(t) for t in range(new)]
    p.table = p.table.expand(new, 10).contiguous()
    p.kv_lens = torch.tensor([min(x + 1, 160) for x in pos], dtype=torch.int32)
    p.q_start = torch.arange(new + 1, dtype=torch.int32)
    ref.check_attention(p, out, lse)
    ref.check_attention(p, picked, picked_lse)


# ---------------------------------------------------------------- key splits

def check(p, idx=None, **kw):
    out, lse = run(p, idx, **kw)
    torch.cuda.synchronize()
    ref.check_attention(p, out, lse, idx)
    return out, lse


def ws_bytes(p, max_new=0):
    shape = misa.AttnShape(len(p.kv_lens), p.heads, p.kv_heads, p.dim, p.tokens, 0, 0, max_new, 1.0)
    pages = misa.KvPages(None, None, None, None, None, p.width, p.pages[0].shape[0], p.page, int(p.fp8))
    return misa.misa_attention_paged_workspace_bytes(shape, pages)


# The join goes through a row's splits four at a time where there are at most four, else eight at a time: one group,
# whole and with every remainder, and several.
JOINED = [2, 3, 4, 5, 6, 7, 8, 9, 15, 16, 17, 24, 32]


@pytest.mark.parametrize("dim,fp8", [(64, False), (64, True), (128, False), (128, True)])
@pytest.mark.parametrize("max_new", [0, 1])
def test_decodes_of_every_count_of_splits(dim, fp8, max_new):
    say("splits of decodes", dim, fp8, max_new)
    lens = [512 * k - 7 * i for i, k in enumerate(JOINED)]   # 512 keys make a split at this size
    p = ref.Paged(42, lens, [1] * len(lens), 2, 1, dim, 64, fp8)
    assert ws_bytes(p, max_new) >= len(lens) * 2 * 32 * (dim + 2) * 4   # room for 32 splits of each
    check(p, max_new=max_new)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,kv_heads", [(4, 2), (40, 1)])
def test_splits_of_rows_placed_by_the_batch_or_by_the_unit(heads, kv_heads, fp8):
    """Few sequences with many rows beside ones with few: parts of the few are kept unit by unit, those of the many where
    the batch has them; with decodes only, all are."""
    say("placed splits", heads, kv_heads, fp8)
    for new in ([70, 1, 2, 33, 1], [1, 1, 1, 1, 1], [200, 0, 0, 0, 1]):
        p = ref.Paged(43, [2300, 1700, 40, 2900, 999], new, heads, kv_heads, 64, 16, fp8)
        assert ws_bytes(p) > 0
        check(p)
        check(p, max_new=max(new))   # (split otherwise, perhaps)


@pytest.mark.parametrize("dim,fp8", [(64, True), (128, False)])
def test_key_splits_among_more_than_4096_sequences(dim, fp8):
    """So many lengths are not summed: each chunk's keys are shared evenly among the splits."""
    say("splits among many", dim, fp8)
    n = 4200
    lens, new = [0] * n, [0] * n
    for b, l, m in ((0, 2500, 40), (1023, 3001, 17), (1024, 64, 64), (2222, 700, 9), (4199, 2900, 50)):
        lens[b], new[b] = l, m
    p = ref.Paged(44, lens, new, 8, 1, dim, 16, fp8)
    assert ws_bytes(p) > 0
    check(p)
