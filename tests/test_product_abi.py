"""The e4m3 products on the CPU: their kernels' source, and workspaces."""
import pathlib
import re

import long_context_sparse_block_amd as misa
from long_context_sparse_block_amd import _lib
from test_tree_abi import at

CSRC = pathlib.Path(misa.__file__).parent / "csrc"


def test_no_assembly_writes_a_register_behind_the_compilers_back():
    """m0 is the compiler's own: a statement that sets it cannot name it as clobbered, so it takes it as an input."""
    blocks = [(p.name, b) for p in CSRC.glob("*.h*") for b in re.findall(r"asm\s+volatile\s*\((.*?)\);", p.read_text(), re.S)]
    assert any("lds" in b for _, b in blocks)
    for name, b in blocks:
        assert not re.search(r"\bs_\w+\s+m0\b", b), (name, b)
        if re.search(r"\boffen lds\b", b):
            assert '"{m0}"' in b, (name, b)


def test_workspaces_of_products_in_parts():
    """Sizes whose blocks are made in parts need a workspace: too small, missing or off its alignment it is refused."""
    lib = _lib.load()
    for m, n, k in ((64, 128, 8192), (64, 1024, 16384), (500, 1003, 5008), (120, 500, 4112)):
        need = misa.misa_matmul_q8_workspace_bytes(m, n, k)
        # whole parts: at least two, each a row of columns (rounded up to four) in fp32 for every row
        part = 4 * m * (-(-n // 4) * 4)
        assert need >= 2 * part and need % part == 0, (m, n, k, need)

        def call(nb=need, work=at(5)):
            return lib.misa_matmul_q8(m, n, k, at(0), k, at(1), at(2), k, at(3), at(4), n, work, nb, None)
        assert call(nb=need - 1) == -3 and call(nb=0) == -3
        assert call(work=None) == -3 and call(work=at(5, 4)) == -3
        assert call(nb=need - 1, work=None) == -3
    for m, n, k in ((1, 8192, 4096), (8192, 8192, 4096), (0, 128, 8192)):   # whole: no workspace
        assert misa.misa_matmul_q8_workspace_bytes(m, n, k) == 0
