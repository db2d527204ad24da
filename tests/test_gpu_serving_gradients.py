"""Gradients through misa_rope: what autograd gives is the transposed rotation of the output's gradient."""
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


def inputs(T, H, D, rot, dt, seed=0):
    g = torch.Generator().manual_seed(seed)
    x, gy = (torch.randn((T, H, D), generator=g).to(dt) for _ in range(2))
    pos = torch.randint(0, 1 << 20, (T,), generator=g).to(torch.int32)
    f, m = misa.rope_inv_freq(rot, scaling="yarn", factor=8.0)
    return x, gy, pos, f, m


def bound(x, y, m):
    """Half a step of the type at y; cos and sin good to 2^-22 and three fp32 roundings of terms within m (|a| + |b|); what
    fp16 loses below its normal range."""
    return (torch.finfo(x.dtype).eps / 2 * y.abs() + (2.0 ** -22 + 3 * ref.F32_HALF) * 2 * x.double().abs().amax() * m
            + (2.0 ** -25 if x.dtype == torch.float16 else 0))


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("T,H,D,rot,start,layout,dt", [
    (1, 1, 64, 64, 0, "half", torch.float32), (33, 3, 192, 64, 128, "interleaved", torch.float32),
    (17, 5, 80, 20, 60, "half", torch.float16), (300, 2, 128, 64, 0, "half", torch.bfloat16)])
def test_gradient_of_rope(T, H, D, rot, start, layout, dt, backward):
    say("rope gradient", T, H, D, rot, start, layout, dt, backward)
    x, gy, pos, f, m = inputs(T, H, D, rot, dt)
    leaf = x.cuda().requires_grad_()
    kw = dict(layout=layout, rot_start=start, mscale=m, backward=backward)
    y = misa.misa_rope(leaf, pos.cuda(), f, **kw)
    with torch.no_grad():
        plain = misa.misa_rope(leaf, pos.cuda(), f, **kw)
    assert torch.equal(y, plain) and not plain.requires_grad
    got, = torch.autograd.grad(y, leaf, gy.cuda())
    want = ref.rope(gy, pos, f.cpu(), layout, start, m, not backward)
    assert got.dtype == dt and float(((got.double().cpu() - want).abs() - bound(gy, want, m)).max()) <= 0


def test_gradients_that_come_expanded_or_strided():
    x, gy, pos, f, m = inputs(9, 4, 128, 64, torch.float32, 1)
    for loss in (lambda y: y.sum(), lambda y: (y.transpose(0, 2) * gy.cuda().transpose(0, 2)).sum(), lambda y: y[2:5, 1].sum()):
        leaf = x.cuda().requires_grad_()
        y = misa.misa_rope(leaf, pos.cuda(), f, mscale=m)
        loss(y).backward()
        at = y.detach().cpu().double().requires_grad_()
        g, = torch.autograd.grad(loss(at.cuda()), at)
        want = ref.rope(g, pos, f.cpu(), "half", 0, m, True)
        assert float(((leaf.grad.double().cpu() - want).abs() - bound(g.float(), want, m)).max()) <= 0


def test_heads_that_share_an_input_sum_their_gradients():
    x, gy, pos, f, m = inputs(9, 4, 128, 128, torch.float32, 2)
    leaf = x[:, :1].cuda().requires_grad_()
    misa.misa_rope(leaf.expand(9, 4, 128), pos.cuda(), f, mscale=m).backward(gy.cuda())
    want = ref.rope(gy, pos, f.cpu(), "half", 0, m, True).sum(1, keepdim=True)
    # four heads' bounds, and three fp32 sums of at most four heads' gradients
    most = 4 * bound(gy, gy.double().abs().amax() * 2 * m, m) + 3 * ref.F32_HALF * 8 * m * gy.abs().amax()
    assert float((leaf.grad.double().cpu() - want).abs().max()) <= float(most)


def test_second_derivatives_rotate_forward_again():
    x, gy, pos, f, m = inputs(5, 2, 64, 64, torch.float32, 3)
    leaf, g = x.cuda().requires_grad_(), gy.cuda().requires_grad_()
    y = misa.misa_rope(leaf, pos.cuda(), f, mscale=m)
    gx, = torch.autograd.grad(y, leaf, g, create_graph=True)
    gg, = torch.autograd.grad(gx, g, x.cuda())
    want = ref.rope(x, pos, f.cpu(), "half", 0, m)
    assert float(((gg.double().cpu() - want).abs() - bound(x, want, m)).max()) <= 0


def test_gradient_on_a_stream_of_the_callers():
    x, gy, pos, f, m = inputs(700, 8, 128, 128, torch.bfloat16, 4)
    leaf, g, p = x.cuda().requires_grad_(), gy.cuda(), pos.cuda()
    base, = torch.autograd.grad(misa.misa_rope(leaf, p, f, mscale=m), leaf, g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got, = torch.autograd.grad(misa.misa_rope(leaf, p, f, mscale=m, stream=side), leaf, g)
    torch.cuda.synchronize()
    assert torch.equal(got, base)


def test_outputs_of_the_callers_take_no_gradient():
    x, gy, pos, f, m = inputs(5, 2, 64, 64, torch.float32, 5)
    leaf = x.cuda().requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        misa.misa_rope(leaf, pos.cuda(), f, out=torch.empty_like(x.cuda()))
    with torch.no_grad():
        misa.misa_rope(leaf, pos.cuda(), f, out=torch.empty_like(x.cuda()))


def test_rotation_and_gradient_captured():
    x, gy, pos, f, m = inputs(700, 4, 128, 64, torch.bfloat16, 6)
    p = pos.cuda()
    jobs = [(x.cuda() * s, gy.cuda() * s) for s in (1, 2, 3)]

    def step(a, g):
        leaf = a.detach().requires_grad_()
        y = misa.misa_rope(leaf, p, f, mscale=m)
        return y.detach(), torch.autograd.grad(y, leaf, g)[0]
    base = [step(*j) for j in jobs]
    a, g = (t.clone() for t in jobs[0])
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(a, g)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            out = step(a, g)
    torch.cuda.synchronize()
    for rep in range(6):
        j = rep % 3
        a.copy_(jobs[j][0])
        g.copy_(jobs[j][1])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, want, again in zip(out, base[j], step(*jobs[j])):
            assert torch.equal(got, want) and torch.equal(again, want), rep
