"""Attention over drafted trees has no backward pass: asked for a gradient it says so."""
import pytest
import torch

import long_context_sparse_block_amd as misa
from test_gpu_tree import batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the -m gpu tests need an MI355X")
    misa.load()


def call(leaf, **kw):
    p, mask = batch(43, [60, 90], [4, 9], 4, 2, 64, 16, False)
    d = p.gpu()
    if leaf:
        d[leaf].requires_grad_()
    args = [d[k] for k in ("q", "k_pages", "v_pages", "block_table", "q_start", "kv_lens")]
    return misa.misa_attention_tree(*args, mask.cuda(), **kw)


@pytest.mark.parametrize("leaf", ["q", "k_pages", "v_pages"])
def test_a_gradient_that_is_asked_for_is_an_error(leaf):
    plain, rl = call(None, want_lse=True)
    assert not plain.requires_grad and not rl.requires_grad
    for kw in (dict(), dict(want_lse=True), dict(max_new=9, stream=torch.cuda.Stream())):
        out, lse = call(leaf, **kw)
        torch.cuda.synchronize()
        assert torch.equal(out, plain) and (lse is None) == ("want_lse" not in kw)
        with pytest.raises(RuntimeError, match="misa_attention_tree has no backward pass"):
            out.float().sum().backward()
        if lse is not None:
            assert torch.equal(lse, rl)
            out, lse = call(leaf, **kw)
            with pytest.raises(RuntimeError, match="misa_attention_tree has no backward pass"):
                lse[4:].sum().backward()


def test_without_gradients_nothing_is_said():
    plain, rl = call(None, want_lse=True)
    with torch.no_grad():
        out, lse = call("q", want_lse=True)
    assert torch.equal(out, plain) and not out.requires_grad and not lse.requires_grad
    given = torch.zeros_like(plain)   # the caller's own tensors stay as they are
    o, l = call("q", out=given, want_lse=True)
    assert o is given and not given.requires_grad and torch.equal(given, plain) and not l.requires_grad
    given = torch.zeros_like(rl)
    o, l = call("q", lse=given)
    assert l is given and not given.requires_grad and torch.equal(l, rl) and o.requires_grad and torch.equal(o, plain)
