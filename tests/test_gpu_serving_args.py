"""Arguments of the paged serving calls, and what the wrappers around them do, on the GPU."""
import pytest
import torch

import long_context_sparse_block_amd as misa
from long_context_sparse_block_amd import serving

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the -m gpu tests need an MI355X")
    misa.load()


def test_a_workspace_that_does_not_fit_is_out_of_memory():
    x = torch.zeros(1, device="cuda")
    with pytest.raises(torch.OutOfMemoryError):
        serving._scratch(1 << 46, x)
    assert serving._scratch(64, x)[0].numel() == 64
