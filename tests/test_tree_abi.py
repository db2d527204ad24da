"""The drafted trees' calls and the e4m3 products on the CPU: every refusal of the C ABI happens on the host before
anything is enqueued, and the Python wrappers check their arguments."""
import ctypes
import subprocess
import sys

import pytest
import torch

import long_context_sparse_block_amd as misa
from long_context_sparse_block_amd import _lib
from test_serving_abi import attn, pool
from tree_helpers import ancestors, pack, unpack

REF = ctypes.byref
STEP = 1 << 40   # buffers that do not overlap


def at(i, off=0):
    return ctypes.c_void_p((i + 1) * STEP + off)   # never dereferenced


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def test_plan_refusals(lib):
    def call(n=4, up=at(0), qs=at(1), kv=at(2), tokens=16, words=2, mask=at(3), pos=at(4)):
        return lib.misa_plan_tree(n, up, qs, kv, tokens, words, mask, pos, None)
    for bad in (dict(n=0), dict(tokens=-1), dict(words=0), dict(up=None), dict(qs=None), dict(kv=None), dict(mask=None),
                dict(pos=None), dict(mask=at(0, 60)), dict(pos=at(1, 16)), dict(pos=at(2)), dict(pos=at(3, 124))):
        assert call(**bad) == -1, bad
    for big in (dict(n=65536), dict(tokens=(1 << 26) + 1), dict(words=1025)):
        assert call(**big) == -2, big
    assert call(tokens=0) == 0 and call(tokens=0, up=None, mask=None, pos=None) == 0


def test_tree_attention_refusals(lib):
    def call(s=attn(), p=pool(max_pages=4096), q=at(0), qs=at(1), kv=at(2), mask=at(3), words=1, out=at(4), ws=at(5), nb=1 << 40):
        return lib.misa_attention_tree(None if s is None else REF(s), None if p is None else REF(p), q, qs, kv, mask, words,
                                       out, None, ws, nb, None)
    assert call(s=None) == -1 and call(p=None) == -1
    for bad in (dict(mask=None), dict(words=0), dict(q=None), dict(q=at(0, 4)), dict(qs=None), dict(kv=None), dict(out=None),
                dict(s=attn(n_heads=7)), dict(s=attn(max_new=-1)), dict(p=pool(page_keys=0)), dict(p=pool(kdtype=1))):
        assert call(**bad) == -1, bad
    for bad in (dict(words=1025), dict(s=attn(head_dim=96)), dict(p=pool(n_pages=1 << 25))):
        assert call(**bad) == -2, bad
    long = pool(max_pages=4096)
    need = misa.misa_attention_tree_workspace_bytes(attn(), long)
    assert need == misa.misa_attention_paged_workspace_bytes(attn(), long) > 0
    assert call(nb=need - 1) == -3 and call(ws=None) == -3 and call(ws=at(5, 4)) == -3
    assert call(s=attn(n_tokens=0)) == 0
    assert misa.misa_attention_tree_workspace_bytes(attn(n_heads=7), pool()) == 0


def test_keep_refusals(lib):
    def call(n=3, path=at(0), most=4, qs=at(1), kv=at(2), table=at(3), width=8, H=2, D=64, k=at(4), v=at(5), kd=1, ks=at(6),
             vs=at(7), pages=20, page=16, kept=at(8)):
        return lib.misa_keep_path(n, path, most, qs, kv, table, width, H, D, k, v, kd, ks, vs, pages, page, kept, None)
    for bad in (dict(n=0), dict(most=0), dict(width=0), dict(H=0), dict(D=0), dict(kd=2), dict(path=None), dict(qs=None),
                dict(kv=None), dict(table=None), dict(kept=None), dict(k=None), dict(k=at(4, 4)), dict(v=at(5, 8)),
                dict(ks=None), dict(vs=None), dict(pages=0), dict(page=0), dict(kept=at(2)), dict(kept=at(0, 40)),
                dict(kept=at(1, 12)), dict(kept=at(3, 92)), dict(kept=at(4)), dict(v=at(4)), dict(ks=at(5)), dict(vs=at(6)),
                dict(k=at(3, 16))):
        assert call(**bad) == -1, bad
    for bad in (dict(n=65536), dict(most=(1 << 20) + 1), dict(width=1 << 31), dict(D=12), dict(D=520), dict(H=1 << 15),
                dict(pages=1 << 27)):
        assert call(**bad) == -2, bad


def test_quantize_refusals(lib):
    def call(x=at(0), dt=0, rows=5, cols=256, st=256, br=1, codes=at(1), scale=at(2)):
        return lib.misa_quantize_blocks(x, dt, rows, cols, st, br, codes, scale, None)
    for bad in (dict(rows=-1), dict(cols=0), dict(st=-8), dict(dt=3), dict(br=0), dict(br=64), dict(x=None), dict(x=at(0, 8)),
                dict(codes=None), dict(codes=at(1, 8)), dict(scale=None), dict(st=260), dict(dt=2, st=258),
                dict(codes=at(0, 16)), dict(scale=at(0)), dict(scale=at(1, 64))):
        assert call(**bad) == -1, bad
    for bad in (dict(cols=264), dict(cols=8), dict(cols=(1 << 20) + 16), dict(rows=(1 << 26) + 1),
                dict(rows=1 << 20, cols=1 << 15, st=1 << 15)):
        assert call(**bad) == -2, bad
    assert call(rows=0) == 0


def test_product_refusals(lib):
    def call(m=5, n=300, k=256, x=at(0), xst=256, xs=at(1), w=at(2), wst=256, ws=at(3), out=at(4), ost=300, work=at(5),
             nb=1 << 40):
        return lib.misa_matmul_q8(m, n, k, x, xst, xs, w, wst, ws, out, ost, work, nb, None)
    for bad in (dict(m=-1), dict(n=0), dict(k=0), dict(x=None), dict(x=at(0, 8)), dict(w=None), dict(w=at(2, 4)),
                dict(xs=None), dict(ws=None), dict(out=None), dict(xst=-16), dict(xst=264), dict(wst=8), dict(ost=299),
                dict(out=at(0, 1024)), dict(out=at(1)), dict(out=at(2)), dict(out=at(3, 4))):
        assert call(**bad) == -1, bad
    for bad in (dict(k=24), dict(k=(1 << 20) + 16), dict(n=(1 << 26) + 1), dict(m=(1 << 26) + 1), dict(m=1 << 26, n=1 << 26),
                dict(xst=1 << 41), dict(wst=1 << 41), dict(ost=1 << 41)):
        assert call(**bad) == -2, bad
    assert call(m=0) == 0
    assert misa.misa_matmul_q8_workspace_bytes(5, 300, 24) == 0
    # sizes that split the blocks need a workspace, and it is checked
    need = misa.misa_matmul_q8_workspace_bytes(5, 128, 8192)
    if need:
        big = dict(n=128, k=8192, xst=8192, wst=8192, ost=128)
        assert call(**big, nb=need - 1) == -3 and call(**big, work=None) == -3 and call(**big, work=at(5, 4)) == -3


def test_wrappers_take_gpu_tensors_only():
    i = torch.zeros(4, dtype=torch.int32)
    pages = torch.zeros((2, 4, 2, 64), dtype=torch.bfloat16)
    x = torch.zeros((3, 128), dtype=torch.bfloat16)
    c, s = torch.zeros((3, 128), dtype=torch.uint8), torch.zeros((3, 1))
    for call in (lambda: misa.misa_plan_tree(i, i, i, 1), lambda: misa.misa_quantize_blocks(x),
                 lambda: misa.misa_matmul_q8(c, s, c, s), lambda: misa.misa_keep_path(i.view(1, 4), i, i, i.view(1, 4), pages),
                 lambda: misa.misa_attention_tree(torch.zeros((4, 2, 64), dtype=torch.bfloat16), pages, pages, i.view(1, 4),
                                                  i, i, i.view(4, 1))):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_matrix_arguments():
    from long_context_sparse_block_amd import _tensor_args, serving
    assert serving._matrix is _tensor_args.matrix
    for check in (serving._matrix, serving._matrix_py):
        with pytest.raises(ValueError, match="^x is required$"):
            check(None, (torch.float32,), "x", 0, None)
        with pytest.raises(ValueError, match="^x must be a GPU tensor$"):
            check(torch.zeros(3, 2), (torch.float32,), "x", 0, None)
    with pytest.raises(TypeError):
        serving._matrix(1)


def test_helpers_agree_on_a_tree_by_hand():
    sees = ancestors([-1, 0, 0, 1, 3, 7, -5])   # 5's parent is not before it, 6's is none
    assert [[j for j in range(7) if r[j]] for r in sees] == [[0], [0, 1], [0, 2], [0, 1, 3], [0, 1, 3, 4], [5], [6]]
    assert pack(sees, 1).flatten().tolist() == [1, 3, 5, 11, 27, 32, 64]
    assert (unpack(pack(sees, 2))[:, :7].numpy() == sees).all()
    assert pack(ancestors([i - 1 for i in range(33)]), 2)[32].tolist() == [-1, 1]


@pytest.mark.parametrize("tensor", ["vmap", "sparse", "symbolic"])
@pytest.mark.parametrize("call", ["serving._matrix(x.select(1, 0), (torch.float32,), 'x', 0)",
                                  "serving._fresh((-5, 2), torch.float32, x)"])
def test_errors_of_torch_stay_errors(call, tensor):
    """As tests/test_serving_args.py has it for the other checks: a C++ exception that passes their border would end the
    process."""
    from test_serving_args import PROGRAM, ROOT, TENSORS
    r = subprocess.run([sys.executable, "-W", "ignore", "-c", PROGRAM.format(call=call, tensor=TENSORS[tensor])], cwd=ROOT,
                       capture_output=True, text=True, timeout=120)
    print(r.stdout, r.stderr[-500:])
    assert r.returncode == 0
    assert r.stdout.startswith("raised")


def test_the_calls_without_ctypes(lib):
    """The wrappers' calls turn their arguments into C's themselves: the same status as through ctypes, and an error for
    what is no such argument."""
    from long_context_sparse_block_amd import _tensor_args, serving
    names = ("misa_plan_pages", "misa_rope", "misa_write_pages", "misa_attention_paged", "misa_attention_selected",
             "misa_plan_tree", "misa_attention_tree", "misa_keep_path", "misa_quantize_blocks", "misa_matmul_q8")
    for name in names:
        call, n = serving._entry(name), len(getattr(lib, name).argtypes)
        assert call is getattr(_tensor_args, name)
        zeros = [None if t is ctypes.c_void_p else 0 for t in getattr(lib, name).argtypes]
        assert call(*zeros) == getattr(lib, name)(*zeros) == -1, name
        for args in (zeros[:-1], zeros + [0]):
            with pytest.raises(TypeError, match=str(n)):
                call(*args)
    quantize, matmul = serving._entry("misa_quantize_blocks"), serving._entry("misa_matmul_q8")
    good = [at(1).value, 0, 4, 256, 256, 128, at(2).value, at(3).value, None]
    for i, bad, status in ((1, 7, -1), (2, -1, -1), (3, 24, -2), (4, 4, -1), (5, 2, -1), (6, at(2, 8).value, -1), (2, 1 << 40, -2)):
        args = good[:i] + [bad] + good[i + 1:]
        assert quantize(*args) == lib.misa_quantize_blocks(*args) == status, (i, bad)
    for i, bad, error in ((1, 1 << 31, OverflowError), (5, -(1 << 31) - 1, OverflowError),
                          (2, 1 << 63, OverflowError), (2, 1.5, TypeError), (0, "x", TypeError), (0, 1.5, TypeError)):
        with pytest.raises(error):
            quantize(*good[:i], bad, *good[i + 1:])
    with pytest.raises((OverflowError, TypeError)):
        matmul(*[1] * 12, -1, None)
    with pytest.raises(ValueError, match="no serving call"):
        _tensor_args.bind("misa_topk", 0)
