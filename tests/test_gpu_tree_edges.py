"""Narrow paths of drafted trees, and workspaces of the caller's, on the GPU, against 64-bit forms."""
import pytest
import torch

import long_context_sparse_block_amd as misa
import tree_helpers as th
from test_gpu_tree import starts

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
