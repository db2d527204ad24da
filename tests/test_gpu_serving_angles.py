"""The angles of fp32 rotations: cosine and sine of the fp64 angle, rounded to fp32 once."""
import pytest
import torch

import long_context_sparse_block_amd as misa
from gpu_helpers import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the -m gpu tests need an MI355X")
    misa.load()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dim", [128, 66])
@pytest.mark.parametrize("backward", [False, True])
def test_fp32_rotations_round_their_angles_functions_once(layout, dim, backward):
    """y = a c - b s with c and s good to half a step of fp32, one rounded product and one rounded sum: half a step each
    of |a c|, |b s|, |b s| and |y|.  The fp64 angles of positions up to 2^20 are good to 2^-31 on either side."""
    say("angles", layout, dim, backward)
    T, H = 4000, 3
    g = torch.Generator().manual_seed(dim)
    x = torch.randn((T, H, dim), generator=g)
    pos = torch.randint(0, 1 << 20, (T,), generator=g).to(torch.int32)
    f, m = misa.rope_inv_freq(dim, scaling="yarn", factor=8.0)
    got = misa.misa_rope(x.cuda(), pos.cuda(), f, layout=layout, mscale=m, backward=backward).double().cpu()
    ang = pos.double()[:, None] * f.cpu()[None]
    c, s = (m * torch.cos(ang))[:, None], (m * torch.sin(ang) * (-1 if backward else 1))[:, None]
    half = dim // 2
    pair = (lambda t: (t[..., :half], t[..., half:])) if layout == "half" else (lambda t: (t[..., 0::2], t[..., 1::2]))
    a, b = pair(x.double())
    step = 2.0 ** -24
    for got_y, y, u, v in zip(pair(got), (a * c - b * s, a * s + b * c), ((a * c).abs(), (a * s).abs()),
                              ((b * s).abs(), (b * c).abs())):
        bound = step * (u + 2 * v + y.abs()) * 1.0001 + 2 * 2.0 ** -31 * m * (a.abs() + b.abs())
        over = float(((got_y - y).abs() / bound).max())
        print("largest error over its bound", over)
        assert over <= 1
