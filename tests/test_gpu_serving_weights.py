"""Attention whose softmax weights enter the product with the values in two bf16 parts: at most 32 rows of a kv head in
a sequence, or in a selected token's group.  The keys come in pairs of nearly equal scores and opposite values, so that the outputs are small
beside their terms and a weight's rounding shows."""
import pytest
import torch

import long_context_sparse_block_amd as misa
import serving_helpers as ref
from gpu_helpers import say

PARTS = 2.0 ** -16    # half a bf16 step of what half a bf16 step left of a weight


def paired(seed, lens, new, heads, kv_heads, dim, page, fp8):
    """A ragged batch, tokens 2 i and 2 i + 1 of a sequence with keys that differ in one element and values v and -v."""
    p = ref.Paged(seed, lens, new, heads, kv_heads, dim, page, fp8)
    for b, n in enumerate(lens):
        first, second = torch.arange(0, n - n % 2, 2), torch.arange(1, n, 2)
        (fp, fr), (sp, sr) = ((p.table[b].long()[t // page], t % page) for t in (first, second))
        for which in (0, 1):
            src = p.pages[which][fp, fr].clone()
            if fp8:
                src = src ^ 0x80 if which else src
                if not which:   # the code next to it (a sixteenth to an eighth of the element), none of them NaN
                    src[..., 5] ^= torch.where((src[..., 5] & 0x7F) == 0x7E, 3, 1).to(torch.uint8)
                p.scale[which][sp, sr] = p.scale[which][fp, fr]
                p.vals[which][sp, sr] = src.view(torch.float8_e4m3fn).double() * p.scale[which][sp, sr].double()[..., None]
            else:
                src = -src if which else src
                src[..., 5] *= 1 if which else 1.0625
                p.vals[which][sp, sr] = src.double()
            p.pages[which][sp, sr] = src
    return p


def exact(p, idx=None, parts=None):
    """out in 64 bits, and its bound where weights have two bf16 parts.  parts: the weights' rounding, to plant a loss.
    (The terms are those of serving_helpers.attention, with 2^-16 in the place of a weight's 2^-8.)"""
    scale = p.dim ** -0.5
    G = p.heads // p.kv_heads
    out = torch.zeros((p.tokens, p.heads, p.dim), dtype=torch.float64)
    tol = torch.zeros_like(out)
    for t in range(p.tokens):
        b = p.seq_of(t)
        toks = torch.arange(p.pos(t) + 1)
        if idx is not None:
            toks = idx[t].long()
            toks = toks[(toks >= 0) & (toks <= p.pos(t))]
        k, v = p.rows(0, b, toks), p.rows(1, b, toks)
        for h in range(p.heads):
            q, kh, vh = p.q[t, h].double(), k[:, h // G], v[:, h // G]
            s = kh @ q * scale
            w = torch.exp(s - s.max())
            e = (p.dim + 8) * ref.F32_HALF * float((kh.abs() @ q.abs()).max() * scale) + 8 * ref.F32_HALF * (1 + float(s.abs().max()))
            o = (parts(w) if parts else w) @ vh / w.sum()
            A = (w @ vh.abs()) / w.sum()
            out[t, h] = o
            tol[t, h] = ref.BF16_HALF * o.abs() + (PARTS + 2 * e + len(toks) * ref.F32_HALF) * A * 1.01
    return out, tol


CASES = {   # lens, new, heads, kv_heads, dim, page, fp8, topk (0: dense)
    "decode": ([64, 130, 700], [1, 1, 1], 8, 2, 128, 16, False, 0),
    "decode_e4m3": ([64, 130, 700], [1, 2, 1], 8, 2, 128, 16, True, 0),
    "decode_32_rows": ([200, 31], [1, 1], 32, 1, 64, 64, False, 0),
    "decode_32_rows_e4m3": ([200, 31], [2, 1], 16, 1, 64, 64, True, 0),
    "selected": ([300], [3], 8, 2, 64, 16, False, 80),
    "selected_17_rows": ([300], [3], 17, 1, 64, 64, False, 90),
    "selected_e4m3": ([2600], [2], 32, 1, 128, 64, True, 2048),
}


def case(name):
    *shape, topk = CASES[name]
    p = paired(len(name), *shape)
    return p, p.select(topk) if topk else None


@pytest.mark.parametrize("name", CASES)
def test_the_bound_tells_one_part_from_two(name):
    """On the CPU: weights rounded to bf16 once are past it, in two parts within."""
    p, idx = case(name)
    want, tol = exact(p, idx)
    once = exact(p, idx, lambda w: w.bfloat16().double())[0]
    twice = exact(p, idx, lambda w: w.bfloat16().double() + (w - w.bfloat16().double()).bfloat16().double())[0]
    assert bool(((once - want).abs() > tol).any()) and bool(((twice - want).abs() <= tol).all())


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_weights_in_two_parts(name):
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the -m gpu tests need an MI355X")
    say("two parts", name)
    p, idx = case(name)
    want, tol = exact(p, idx)
    if idx is None:
        out = misa.misa_attention_paged(**p.gpu(), max_new=2)[0]
    else:
        out = misa.misa_attention_selected(**p.gpu(), idx=idx.cuda())[0]
    over = float(((out.double().cpu() - want).abs() / tol).max())
    print("largest error over its bound", over)
    assert over <= 1
