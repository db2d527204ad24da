"""The e4m3 products on the CPU: their kernels' source, and workspaces."""
import pathlib
import re

import long_context_sparse_block_amd as misa

CSRC = pathlib.Path(misa.__file__).parent / "csrc"


def test_no_assembly_writes_a_register_behind_the_compilers_back():
    """m0 is the compiler's own: a statement that sets it cannot name it as clobbered, so it takes it as an input."""
    blocks = [(p.name, b) for p in CSRC.glob("*.h*") for b in re.findall(r"asm\s+volatile\s*\((.*?)\);", p.read_text(), re.S)]
    assert any("lds" in b for _, b in blocks)
    for name, b in blocks:
        assert not re.search(r"\bs_\w+\s+m0\b", b), (name, b)
        if re.search(r"\boffen lds\b", b):
            assert '"{m0}"' in b, (name, b)
