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
