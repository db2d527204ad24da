"""The paged serving operators on the CPU: every refusal of the C ABI happens on
the host before anything is enqueued, the Python wrappers check their
arguments, and the rotary frequencies follow their formulas."""
import ctypes
import math

import pytest
import torch

import long_context_sparse_block_amd as misa
from long_context_sparse_block_amd import _lib, serving

FAKE = ctypes.c_void_p(0x10000)   # never dereferenced
ODD = ctypes.c_void_p(0x10004)
REF = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def test_plan_refusals(lib):
    def call(n=4, cached=FAKE, new=FAKE, page=64, free=FAKE, n_free=8, table=FAKE, width=10, qs=FAKE, kv=FAKE, slots=FAKE,
             pos=FAKE, tokens=16, taken=FAKE):
        return lib.misa_plan_pages(n, cached, new, page, free, n_free, table, width, qs, kv, slots, pos, tokens, taken, None)
    for bad in (dict(n=0), dict(page=0), dict(width=0), dict(n_free=-1), dict(tokens=-1), dict(cached=None),
                dict(new=None), dict(table=None), dict(qs=None), dict(kv=None), dict(taken=None), dict(free=None),
                dict(slots=None), dict(pos=None)):
        assert call(**bad) == -1, bad
    for big in (dict(n=65536), dict(tokens=(1 << 26) + 1), dict(width=1 << 31)):
        assert call(**big) == -2, big


def spec(**kw):
    base = dict(inv_freq=0x10000, positions=0x10000, rotary_dim=64, rot_start=0, layout=0, backward=0, mscale=1.0)
    base.update(kw)
    return serving.RopeSpec(*[base[f] for f, _ in serving.RopeSpec._fields_])


BAD_SPECS = [dict(inv_freq=None), dict(positions=None), dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=1026),
             dict(rotary_dim=130), dict(rot_start=-2), dict(rot_start=65), dict(layout=2), dict(mscale=math.nan)]


def test_rope_refusals(lib):
    def call(s=spec(), x=FAKE, dt=0, T=5, H=2, D=128, xst=256, xsh=128, out=ODD, ost=256, osh=128):
        return lib.misa_rope(None if s is None else REF(s), x, dt, T, H, D, xst, xsh, out, ost, osh, None)
    assert call(s=None) == -1
    for kw in BAD_SPECS:
        assert call(s=spec(**kw)) == -1, kw
    for bad in (dict(x=None), dict(out=None), dict(dt=3), dict(T=-1), dict(H=0), dict(D=0), dict(xst=-1),
                dict(ost=255), dict(osh=127), dict(ost=0), dict(x=ODD, xst=512)):
        assert call(**bad) == -1, bad
    assert call(T=(1 << 26) + 1) == -2
    assert call(H=1 << 14, D=128, osh=128, ost=1 << 21) == -2
    assert call(T=0) == 0


def test_write_refusals(lib):
    def call(T=5, H=2, D=128, k=FAKE, kst=256, ksh=128, v=None, vst=0, vsh=0, slots=FAKE, s=None, kp=FAKE, vp=None, kd=0,
             ks=None, vs=None, pages=4, page=16):
        return lib.misa_write_pages(T, H, D, k, kst, ksh, v, vst, vsh, slots, None if s is None else REF(s), kp, vp, kd,
                                    ks, vs, pages, page, None)
    for bad in (dict(T=-1), dict(H=0), dict(D=0), dict(k=None), dict(k=ODD), dict(slots=None), dict(kp=None), dict(kp=ODD),
                dict(kd=2), dict(kd=1), dict(kst=4), dict(ksh=-8), dict(v=FAKE), dict(vp=FAKE), dict(v=FAKE, vp=FAKE, vst=3),
                dict(v=FAKE, vp=FAKE, kd=1, ks=FAKE), dict(pages=0), dict(page=0), dict(s=spec(backward=1))):
        assert call(**bad) == -1, bad
    for kw in BAD_SPECS:
        assert call(s=spec(**kw)) == -1, kw
    for big in (dict(D=12), dict(D=520), dict(T=(1 << 26) + 1), dict(pages=1 << 27), dict(H=1 << 14)):
        assert call(**big) == -2, big
    assert call(T=0) == 0


def attn(**kw):
    base = dict(n_seq=2, n_heads=8, n_kv_heads=2, head_dim=128, n_tokens=4, q_stride_token=1024, q_stride_head=128,
                max_new=0, scale=0.1)
    base.update(kw)
    return serving.AttnShape(*[base[f] for f, _ in serving.AttnShape._fields_])


def pool(**kw):
    base = dict(k=0x10000, v=0x10000, k_scale=None, v_scale=None, block_table=0x10000, max_pages=8, n_pages=20,
                page_keys=64, kdtype=0)
    base.update(kw)
    return serving.KvPages(*[base[f] for f, _ in serving.KvPages._fields_])


@pytest.mark.parametrize("selected", [False, True])
def test_attention_refusals(lib, selected):
    def call(s=attn(), p=pool(), q=FAKE, qs=FAKE, kv=FAKE, idx=FAKE, topk=64, out=FAKE, ws=FAKE, nb=1 << 40):
        a = [None if s is None else REF(s), None if p is None else REF(p), q, qs, kv]
        if selected:
            a += [idx, topk]
        f = lib.misa_attention_selected if selected else lib.misa_attention_paged
        return f(*a, out, None, ws, nb, None)
    assert call(s=None) == -1 and call(p=None) == -1
    for kw in (dict(n_seq=0), dict(n_heads=0), dict(n_kv_heads=0), dict(n_heads=7), dict(n_tokens=-1), dict(max_new=-1),
               dict(scale=math.nan), dict(scale=math.inf), dict(q_stride_token=4), dict(q_stride_head=-8)):
        assert call(s=attn(**kw)) == -1, kw
    for kw in (dict(head_dim=96), dict(n_seq=65536), dict(n_heads=2048), dict(n_tokens=(1 << 26) + 1)):
        assert call(s=attn(**kw)) == -2, kw
    for kw in (dict(k=None), dict(v=None), dict(k=0x10004), dict(v=0x10008), dict(block_table=None), dict(max_pages=0),
               dict(n_pages=0), dict(page_keys=0), dict(kdtype=2), dict(kdtype=1), dict(kdtype=1, k_scale=0x10000)):
        assert call(p=pool(**kw)) == -1, kw
    for kw in (dict(n_pages=1 << 25), dict(max_pages=1 << 25)):
        assert call(p=pool(**kw)) == -2, kw
    for bad in (dict(q=None), dict(q=ODD), dict(qs=None), dict(kv=None), dict(out=None), dict(out=ODD)):
        assert call(**bad) == -1, bad
    if selected:
        for bad in (dict(idx=None), dict(topk=0), dict(topk=misa.MAX_TOPK + 1)):
            assert call(**bad) == -1, bad
        need = lib.misa_attention_selected_workspace_bytes(REF(attn()), REF(pool()), 64)
    else:
        need = lib.misa_attention_paged_workspace_bytes(REF(attn()), REF(pool()))
    if need:
        assert call(nb=need - 1) == -3 and call(ws=None) == -3 and call(ws=ODD) == -3
    assert call(s=attn(n_tokens=0)) == 0


def test_workspace_queries_of_invalid_shapes(lib):
    assert misa.misa_attention_paged_workspace_bytes(attn(n_heads=7), pool()) == 0
    assert misa.misa_attention_selected_workspace_bytes(attn(), pool(), 0) == 0
    assert misa.misa_attention_selected_workspace_bytes(attn(), pool(page_keys=0), 64) == 0


def test_wrappers_take_gpu_tensors_only():
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    pos = torch.zeros(3, dtype=torch.int32)
    f, _ = misa.rope_inv_freq(64, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        misa.misa_rope(x, pos, f)
    with pytest.raises(ValueError, match="GPU"):
        misa.misa_write_pages(x, torch.zeros(3, dtype=torch.int64), torch.zeros((2, 4, 2, 64), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="GPU"):
        misa.misa_plan_pages(pos, pos, pos, torch.zeros((3, 4), dtype=torch.int32), 16, 8)
    with pytest.raises(ValueError, match="GPU"):
        misa.misa_attention_paged(x, torch.zeros((2, 4, 2, 64), dtype=torch.bfloat16),
                                  torch.zeros((2, 4, 2, 64), dtype=torch.bfloat16), torch.zeros((1, 1), dtype=torch.int32),
                                  torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


def test_rope_frequencies():
    f, m = misa.rope_inv_freq(8, base=10000.0, device="cpu")
    assert f.dtype == torch.float64 and m == 1.0
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-14, atol=0)
    lin, m = misa.rope_inv_freq(8, scaling="linear", factor=4.0, device="cpu")
    assert torch.allclose(lin, f / 4, rtol=1e-14, atol=0) and m == 1.0
    # ntk: the lowest frequency is stretched by the factor, the highest stays
    ntk, m = misa.rope_inv_freq(128, scaling="ntk", factor=4.0, device="cpu")
    base, _ = misa.rope_inv_freq(128, device="cpu")
    assert ntk[0] == 1.0 and m == 1.0 and math.isclose(float(ntk[-1]), float(base[-1]) / 4, rel_tol=1e-12)
    # yarn: pairs that turn more than 32 times in 4096 positions stay, those that turn less than once are divided
    y, m = misa.rope_inv_freq(128, scaling="yarn", factor=40.0, device="cpu")
    turns = 4096 * base / (2 * math.pi)
    ratio = y / base
    assert math.isclose(m, 0.1 * math.log(40.0) + 1)
    assert bool((ratio[turns > 40] == 1).all())
    assert torch.allclose(ratio[turns < 0.8], torch.full_like(ratio[turns < 0.8], 1 / 40), rtol=1e-12, atol=0)
    # (equal ratios may differ by the fp64 roundings of a quotient, a product and a sum)
    assert bool((ratio[1:] <= ratio[:-1] * (1 + 4 * 2.0 ** -53)).all())
    assert misa.rope_inv_freq(64, scaling="yarn", factor=1.0, device="cpu")[1] == 1.0
    for bad in (dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=8, scaling="other"),
                dict(rotary_dim=8, factor=0.0), dict(rotary_dim=2, scaling="ntk", factor=2.0)):
        with pytest.raises(ValueError):
            misa.rope_inv_freq(device="cpu", **bad)


def test_argument_checks_are_the_built_ones():
    from long_context_sparse_block_amd import _tensor_args, serving
    assert serving._dense is _tensor_args.dense and serving._rows is _tensor_args.rows
    for check in (serving._dense, serving._dense_py):
        with pytest.raises(ValueError, match="^x is required$"):
            check(None, torch.float32, (3,), "x", 0)
        with pytest.raises(ValueError, match="^x must be a GPU tensor$"):
            check(torch.zeros(3), torch.float32, (3,), "x", 0)
    for check in (serving._rows, serving._rows_py):
        with pytest.raises(ValueError, match="^x is required$"):
            check(None, (torch.float32,), "x", 0)
        with pytest.raises(ValueError, match="^x must be a GPU tensor$"):
            check(torch.zeros(3, 2, 4), (torch.float32,), "x", 0, None)
    with pytest.raises(TypeError):
        serving._dense(1)
    with pytest.raises(ValueError):
        serving._dense(7, torch.float32, (3,), "x", 0)
