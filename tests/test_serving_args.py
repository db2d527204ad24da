"""Arguments of the paged serving calls that the built checks (_tensor_args) and the wrappers around them have to turn
into Python errors, on the CPU.  Fake tensors stand for GPU ones: they have a device, sizes and strides and no memory."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Each call below meets a tensor whose sizes, strides or pointer torch refuses with a C++ exception.  Tried in a process
# of its own: one that passes a C function's border ends it.
CALLS = {
    "dense": "serving._dense(x, torch.float32, (3, 2, 64), 'x', 0)",
    "rows": "serving._rows(x, (torch.float32,), 'x', 0)",
    "rows_shape": "serving._rows(x, (torch.float32,), 'x', 0, (3, 2, 64))",
    "pool": "serving._pool(x.to(torch.bfloat16), 1, 64, 'x', 0)",
    "scratch": "serving._scratch(-5, x)",
}
TENSORS = {
    "vmap": "torch.func.vmap(call)(torch.empty((2, 3, 2, 64), device='cuda'))",
    "sparse": "call(torch.sparse_coo_tensor(torch.zeros((3, 1), dtype=torch.int64, device='cuda'), "
              "torch.zeros(1, device='cuda'), (3, 2, 64)))",
    "symbolic": "call(torch.empty((sizes.create_unbacked_symint(), 2, 64), device='cuda'))",
}
PROGRAM = """
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from torch.fx.experimental.symbolic_shapes import ShapeEnv
from long_context_sparse_block_amd import serving
sizes = ShapeEnv()
mode = FakeTensorMode(shape_env=sizes, allow_non_fake_inputs=True)
def call(x):
    return {call}
with mode:
    try:
        print("returned", {tensor})
    except Exception as e:
        print("raised", type(e).__name__, str(e)[:200])
"""


@pytest.mark.parametrize("tensor", TENSORS)
@pytest.mark.parametrize("call", CALLS)
def test_errors_of_torch_stay_errors(call, tensor):
    r = subprocess.run([sys.executable, "-W", "ignore", "-c", PROGRAM.format(call=CALLS[call], tensor=TENSORS[tensor])],
                       cwd=ROOT, capture_output=True, text=True, timeout=120)
    print(r.stdout, r.stderr[-500:])
    assert r.returncode == 0
    assert r.stdout.startswith("raised")


BROKEN = """
import sys
class Finder:
    def find_spec(self, name, path=None, target=None):
        if name.endswith("._tensor_args"):
            raise {error}
sys.meta_path.insert(0, Finder())
import torch
from long_context_sparse_block_amd import build, serving   # (building again stays possible)
try:
    serving._dense(None, torch.float32, (3,), "x", 0)
except Exception as e:
    print(type(e).__name__, serving._dense is serving._dense_py, e)
"""


def test_built_checks_that_do_not_load_are_an_error():
    """A library that is there but fails to load (built against another torch, say) is not passed over; one that is not
    built leaves the Python checks."""
    def run(error):
        r = subprocess.run([sys.executable, "-c", BROKEN.format(error=error)], cwd=ROOT, capture_output=True, text=True,
                           timeout=120)
        assert r.returncode == 0, r.stderr[-2000:]
        return r.stdout
    assert run("ModuleNotFoundError('none', name=name)").startswith("ValueError True x is required")
    out = run("ImportError('undefined symbol: _Znwm')")
    assert out.startswith("RuntimeError False") and "undefined symbol" in out and "build" in out


def attention_bytes(n_seq, tokens, max_new, heads=32, kv_heads=8, dim=128, fp8=False, width=256, page=64):
    import long_context_sparse_block_amd as misa
    shape = misa.AttnShape(n_seq, heads, kv_heads, dim, tokens, heads * dim, dim, max_new, 1.0)
    return misa.misa_attention_paged_workspace_bytes(
        shape, misa.KvPages(None, None, None, None, None, width, n_seq * width, page, int(fp8)))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("fp8", [False, True])
def test_workspace_follows_the_rows_that_exist(dim, fp8):
    """Parts are kept for at most two workgroups to each that the GPU holds (768 or 512 of up to 128 rows, 1024 of 32),
    whatever max_new says: 768 x 2 x 128 rows and 1024 x 2 x 32 of dim fp32 values and two more."""
    most = (2 * (768 if dim == 64 else 512) * 128 + 2 * 1024 * 32) * (dim + 2) * 4 + (1 << 20)
    for n in (1, 2, 9, 64, 256, 1024, 4096):
        for new in (1, 2, 7):
            for max_new in (0, new):
                assert attention_bytes(n, n * new, max_new, dim=dim, fp8=fp8) <= most, (n, new, max_new)
    # few decodes: no more than 96 splits of the rows there are
    for n in (1, 2, 3, 9):
        assert attention_bytes(n, n, 0, dim=dim, fp8=fp8) <= 96 * n * 32 * (dim + 2) * 4 + (1 << 16)


# name, bytes of each array of a misa_plan_pages call of 4 sequences, 8 free pages, 10 table columns and 16 tokens
PLAN_ARRAYS = [("cached", 16), ("new", 16), ("free", 32), ("table", 160), ("qs", 20), ("kv", 16), ("slots", 128), ("pos", 64),
               ("taken", 4)]
PLAN_INPUTS = ("cached", "new", "free")


def plan_status(**at):
    """Status of a call whose arrays lie apart, but for those given (addresses, never read)."""
    import ctypes

    import long_context_sparse_block_amd as misa
    where = {name: 0x100000 + 0x1000 * i for i, (name, _) in enumerate(PLAN_ARRAYS)}
    where.update(at)
    p = {name: ctypes.c_void_p(a) for name, a in where.items()}
    return misa.load().misa_plan_pages(4, p["cached"], p["new"], 64, p["free"], 8, p["table"], 10, p["qs"], p["kv"], p["slots"],
                                       p["pos"], 16, p["taken"], None)


def test_plan_refuses_outputs_over_its_arrays():
    """Workgroups read the lengths and the free list while others write: the next step's cached_lens may not be the
    kv_lens that the same call fills."""
    for i, (a, bytes_a) in enumerate(PLAN_ARRAYS):
        for b, bytes_b in PLAN_ARRAYS[i + 1:]:
            if a in PLAN_INPUTS and b in PLAN_INPUTS:
                continue   # (two inputs may be one array)
            for apart in (0, bytes_a - 4, 4 - bytes_b):   # the same array, the last four bytes of either
                assert plan_status(**{a: 0x800000, b: 0x800000 + apart}) == -1, (a, b, apart)


def test_a_stream_of_another_gpu_is_refused(monkeypatch):
    """Work goes to the stream that the caller names, or nowhere."""
    import torch
    from torch._subclasses.fake_tensor import FakeTensorMode

    import long_context_sparse_block_amd as misa

    class Stream:
        device_index = 1
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    with FakeTensorMode():
        x = torch.empty((3, 2, 64), dtype=torch.bfloat16, device="cuda")   # on GPU 0
        n = torch.empty((3,), dtype=torch.int32, device="cuda")
    at = dict(stream=Stream())
    for call in (lambda: misa.misa_rope(x, n, None, **at), lambda: misa.misa_write_pages(x, n, x, **at),
                 lambda: misa.misa_plan_pages(n, n, n, n, 16, 3, **at),
                 lambda: misa.misa_attention_paged(x, x, x, n, n, n, **at),
                 lambda: misa.misa_attention_selected(x, x, x, n, n, n, n, **at)):
        with pytest.raises(ValueError, match="stream.*cuda:1.*cuda:0"):
            call()
    with pytest.raises(ValueError, match="stream"):
        misa.misa_rope(x, n, None, stream=7)


def test_attention_grids_past_their_bound_are_refused():
    """More than 2^23 workgroups: unsupported, and no workspace is asked for."""
    import ctypes

    import long_context_sparse_block_amd as misa
    lib, at = misa.load(), ctypes.c_void_p(0x100000)   # (never read)
    ref = ctypes.byref
    pages = misa.KvPages(0x100000, 0x100000, None, None, 0x100000, 8, 20, 64, 0)
    for n_seq, heads, kv, tokens, topk in ((2, 32, 8, (1 << 20) + 1, 64), (2, 1024, 1, (1 << 20) + 1, 2048),
                                           (65535, 1024, 1024, 65535, 0), (1, 1024, 1, (1 << 20) + 64, 0)):
        shape = misa.AttnShape(n_seq, heads, kv, 128, tokens, 0, 0, 0, 1.0)
        if topk:
            st = lib.misa_attention_selected(ref(shape), ref(pages), at, at, at, at, topk, at, None, at, 1 << 40, None)
            need = misa.misa_attention_selected_workspace_bytes(shape, pages, topk)
        else:
            st = lib.misa_attention_paged(ref(shape), ref(pages), at, at, at, at, None, at, 1 << 40, None)
            need = misa.misa_attention_paged_workspace_bytes(shape, pages)
        assert st == -2 and need == 0, (n_seq, heads, kv, tokens, topk)


@pytest.mark.parametrize("dim,fp8,heads,groups", [(128, False, 32, 1), (64, False, 32, 2), (128, True, 32, 2), (128, True, 256, 1),
                                                  (64, True, 32, 3), (64, True, 256, 2)])
def test_decodes_split_for_the_workgroups_a_cu_holds(dim, fp8, heads, groups):
    """Two splits to each workgroup that the GPU holds: 256 CUs of `groups` (e4m3 with 32 rows of 128: one)."""
    rows, kv = heads // 8, 8
    for n in (1, 3, 17, 32, 50, 64, 65, 100, 128, 200):
        units = n * kv
        splits = 1 if units >= 512 * groups else min(-(-512 * groups // units), 64, 128 // 4)
        part = splits * units * rows * 4
        want = 0 if splits == 1 else sum(-(-x // 256) * 256 for x in (part * dim, part * 2, 16 * n))
        assert attention_bytes(n, n, 1, heads=heads, kv_heads=kv, dim=dim, fp8=fp8) == want, n


def test_missing_arguments_are_named():
    import torch
    from torch._subclasses.fake_tensor import FakeTensorMode

    import long_context_sparse_block_amd as misa
    with FakeTensorMode():
        n = torch.empty((3,), dtype=torch.int32, device="cuda")
        table = torch.empty((3, 4), dtype=torch.int32, device="cuda")
        x = torch.empty((3, 2, 64), dtype=torch.bfloat16, device="cuda")
        pages = torch.empty((5, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
        plan = [n, n, n, table]
        for i, name in enumerate(("cached_lens", "new_lens", "free_pages", "block_table")):
            with pytest.raises(ValueError, match=f"^{name} is required$"):
                misa.misa_plan_pages(*plan[:i], None, *plan[i + 1:], 16, 3)
        for i, name in enumerate(("q", "k_pages", "v_pages", "block_table")):
            args = [x, pages, pages, table]
            args[i] = None
            with pytest.raises(ValueError, match=f"^{name} is required$"):
                misa.misa_attention_paged(*args, n, n)
        with pytest.raises(ValueError, match="^inv_freq is required$"):
            misa.misa_rope(x, n, None)
