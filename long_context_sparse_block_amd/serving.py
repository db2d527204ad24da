"""The paged serving step around the indexer (C ABI in include/misa.h): page
planning from request lengths, rotary positions, the write of new keys and
values into their pages, attention over the pages, over the tokens that the
indexer picked or of trees of drafted tokens, those trees' plan and the move of
an accepted path's rows, and e4m3 projections with a scale for each block of 128.

As in _lib: argument marshalling only, raw device pointers and the current HIP
stream (of the tensors' own device) go to the library, and there is no
fallback.  misa_rope takes part in autograd; the other calls serve, and their
outputs have no gradient (misa_attention_tree's say so when asked for one).
"""
from __future__ import annotations

import ctypes
import math
import struct
from typing import NamedTuple

import torch

from ._lib import MISA_K_FP8_E4M3, _check, _kdtype, _need, load

MISA_T_BF16, MISA_T_FP16, MISA_T_FP32 = 0, 1, 2
_DTYPES = {torch.bfloat16: MISA_T_BF16, torch.float16: MISA_T_FP16, torch.float32: MISA_T_FP32}
_BF16 = (torch.bfloat16,)
_CODES = (torch.uint8, torch.float8_e4m3fn)
_LAYOUTS = {"half": 0, "interleaved": 1}


class RopeSpec(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("rotary_dim", ctypes.c_int32),
                ("rot_start", ctypes.c_int32), ("layout", ctypes.c_int32), ("backward", ctypes.c_int32),
                ("mscale", ctypes.c_double)]


class KvPages(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("max_pages", ctypes.c_int64),
                ("n_pages", ctypes.c_int64), ("page_keys", ctypes.c_int32), ("kdtype", ctypes.c_int32)]


class AttnShape(ctypes.Structure):
    _fields_ = [("n_seq", ctypes.c_int32), ("n_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("n_tokens", ctypes.c_int64), ("q_stride_token", ctypes.c_int64),
                ("q_stride_head", ctypes.c_int64), ("max_new", ctypes.c_int32), ("scale", ctypes.c_float)]


class PagePlan(NamedTuple):
    """What misa_plan_pages writes (misa.h)."""
    q_start: torch.Tensor     # int32 [n_seq + 1]
    kv_lens: torch.Tensor     # int32 [n_seq]
    slots: torch.Tensor       # int64 [n_tokens]
    positions: torch.Tensor   # int32 [n_tokens]
    n_taken: torch.Tensor     # int32 [1]


class TreePlan(NamedTuple):
    """What misa_plan_tree writes (misa.h)."""
    mask: torch.Tensor        # int32 [n_tokens, words]: ancestor bits
    positions: torch.Tensor   # int32 [n_tokens]


# The C structures as bytes (native layout: the ctypes classes above); packing
# is several times cheaper than filling a ctypes object, which counts where a
# whole call takes a few microseconds.
_PACK_ROPE = struct.Struct("@PPiiiid")
_PACK_PAGES = struct.Struct("@PPPPPqqii")
_PACK_ATTN = struct.Struct("@iiiiqqqif")
assert _PACK_ROPE.size == ctypes.sizeof(RopeSpec) and _PACK_PAGES.size == ctypes.sizeof(KvPages)
assert _PACK_ATTN.size == ctypes.sizeof(AttnShape)

_raw_stream = torch._C._cuda_getCurrentRawStream   # the current stream's handle, without a Stream object


def _dev(t, name):
    """Index of the GPU t is on."""
    if t is None:
        raise ValueError(f"{name} is required")
    d = t.get_device()
    if d < 0:
        raise ValueError(f"{name} must be a GPU tensor")
    return d


def _dense_py(t, dtype, shape, name, dev):
    """Pointer of a dense tensor of this type and shape on GPU `dev`."""
    if t is None or t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _need(t, dtype, shape, name)
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    return t.data_ptr()


def _rows_py(t, dtypes, name, dev, shape=None):
    """Pointer, token and head strides of a [tokens, heads, head_dim] tensor whose
    last dimension is dense."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}" if t.is_cuda else f"{name} must be a GPU tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected one of {tuple(dtypes)}")
    if t.dim() != 3 or (shape is not None and t.shape != shape):
        want = "[tokens, heads, head_dim]" if shape is None else tuple(shape)
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {want}")
    T, H, D = t.shape
    st, sh, sd = t.stride()
    if sd != 1 and D > 1:
        raise ValueError(f"{name}: the last dimension must be dense")
    # the strides of dimensions of one element mean nothing
    return t.data_ptr(), (st if T > 1 else 0), (sh if H > 1 else 0)


def _matrix_py(t, dtypes, name, dev, shape=None):
    """Pointer and row stride of a [rows, columns] tensor whose last dimension is dense."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}" if t.is_cuda else f"{name} must be a GPU tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected one of {tuple(dtypes)}")
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {'[rows, columns]' if shape is None else tuple(shape)}")
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"{name}: the last dimension must be dense")
    return t.data_ptr(), (t.stride(0) if t.shape[0] > 1 else 0)


def _pool_py(pages, heads, head_dim, name, dev):
    """Pointer, kdtype, n_pages, page_keys of a page pool [n_pages, page_keys, heads,
    head_dim] (or [n_pages, page_keys, head_dim] of one head) on GPU `dev`."""
    if pages is None:
        raise ValueError(f"{name} is required")
    if not pages.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if pages.get_device() != dev:
        raise ValueError(f"{name} is on {pages.device}, expected cuda:{dev}")
    if pages.dtype not in (torch.bfloat16, torch.uint8, torch.float8_e4m3fn):
        raise ValueError(f"{name}: dtype {pages.dtype} (expected bfloat16 or float8_e4m3fn/uint8 codes)")
    shape = tuple(pages.shape)
    if shape[2:] != (heads, head_dim) and not (heads == 1 and shape[2:] == (head_dim,)):
        raise ValueError(f"{name}: shape {shape}, expected (n_pages, page_keys, {heads}, {head_dim})")
    if not pages.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return pages.data_ptr(), _kdtype(pages), shape[0], shape[1]


def _scratch_py(nbytes, like):
    t = torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    return t, t.data_ptr()


def _fresh_py(shape, dtype, like):
    """A dense uninitialised tensor on like's device, and its pointer."""
    t = torch.empty(shape, dtype=dtype, device=like.device)
    return t, t.data_ptr()


try:   # the same in C++ (csrc/tensor_args.cpp): a quarter of the time
    from ._tensor_args import dense as _dense, fresh as _fresh, matrix as _matrix, pool as _pool, rows as _rows, scratch as _scratch
    from . import _tensor_args as _cpp
except ModuleNotFoundError:   # not built yet
    _cpp = None
    _dense, _fresh, _matrix, _pool, _rows, _scratch = _dense_py, _fresh_py, _matrix_py, _pool_py, _rows_py, _scratch_py
except ImportError as e:   # built against another torch, say: every call raises, importing and building again do not
    def _dense(*args, why=str(e)):
        raise RuntimeError(f"_tensor_args does not load ({why}): build it again with "
                           "`python -m long_context_sparse_block_amd.build`")
    _cpp, _fresh, _matrix, _pool, _rows, _scratch = None, *[_dense] * 5


def _on(stream, t, name, f, *args):
    """f(*args) with `stream`, of tensor t's GPU, as the current one: what f
    allocates is then `stream`'s own memory, which no work of another stream may
    still be using."""
    if not isinstance(stream, torch.cuda.Stream):
        raise ValueError(f"stream: {stream!r}, expected a torch.cuda.Stream")
    if stream.device_index != _dev(t, name):
        raise ValueError(f"stream is on cuda:{stream.device_index}, {name} on {t.device}")
    with torch.cuda.stream(stream):
        return f(*args)


_entries = {}   # what calls an entry point: C++, or ctypes where that is not built


def _entry(name):
    fn = getattr(load(), name)
    if _cpp is not None:
        _cpp.bind(name, ctypes.cast(fn, ctypes.c_void_p).value)
        fn = getattr(_cpp, name)
    _entries[name] = fn
    return fn


def _call(name, dev, *args):
    """The entry point's call with args and the current stream's handle, on GPU `dev`."""
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return _call(name, dev, *args)
    st = (_entries.get(name) or _entry(name))(*args, _raw_stream(dev))
    if st != 0:
        _check(st, name)


def misa_plan_pages(cached_lens, new_lens, free_pages, block_table, page_keys: int, n_tokens: int,
                    plan: PagePlan | None = None, stream=None) -> PagePlan:
    """Pages for the new tokens of every sequence: writes the new entries of
    block_table [n_seq, max_pages] (int32, in place) from free_pages (int32) and
    returns the PagePlan (plan: its tensors, made new unless given, and none of
    them among this call's inputs).  n_tokens: length of the slot map (at least the sum of
    new_lens; entries behind the last token get slot -1)."""
    if stream is not None:
        return _on(stream, cached_lens, "cached_lens", misa_plan_pages, cached_lens, new_lens, free_pages, block_table,
                   page_keys, n_tokens, plan)
    dev = _dev(cached_lens, "cached_lens")
    _dev(free_pages, "free_pages"), _dev(block_table, "block_table")
    n = cached_lens.shape[0]
    i32 = torch.int32
    if plan is None:
        slots = torch.empty(n_tokens, dtype=torch.int64, device=cached_lens.device)
        rest = torch.empty(2 * n + 2 + n_tokens, dtype=i32, device=cached_lens.device)
        q_start, kv_lens, positions, n_taken = torch.unsafe_split_with_sizes(rest, (n + 1, n, n_tokens, 1))
        plan = PagePlan(q_start, kv_lens, slots, positions, n_taken)
        at = rest.data_ptr()
        outs = (at, at + 4 * (n + 1), slots.data_ptr(), at + 4 * (2 * n + 1), n_tokens, at + 4 * (2 * n + 1 + n_tokens))
    else:
        outs = (_dense(plan.q_start, i32, (n + 1,), "q_start", dev), _dense(plan.kv_lens, i32, (n,), "kv_lens", dev),
                _dense(plan.slots, torch.int64, (n_tokens,), "slots", dev),
                _dense(plan.positions, i32, (n_tokens,), "positions", dev), n_tokens,
                _dense(plan.n_taken, i32, (1,), "n_taken", dev))
    n_free, width = free_pages.shape[0], block_table.shape[-1]
    _call("misa_plan_pages", dev, n, _dense(cached_lens, i32, (n,), "cached_lens", dev),
          _dense(new_lens, i32, (n,), "new_lens", dev), page_keys, _dense(free_pages, i32, (n_free,), "free_pages", dev),
          n_free, _dense(block_table, i32, (n, width), "block_table", dev), width, *outs)
    return plan


def rope_inv_freq(rotary_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                  original_max: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda"):
    """Rotary frequencies (fp64 [rotary_dim / 2], radians a position) and the
    mscale that goes with them.  With f_j = base ** (-2 j / rotary_dim):
      None      f_j, mscale 1
      "linear"  f_j / factor (positions divided by factor), mscale 1
      "ntk"     the base raised to base * factor ** (rotary_dim / (rotary_dim - 2)),
                which stretches the lowest frequency by factor and leaves the highest
      "yarn"    f_j where pair j turns more than beta_fast times within original_max
                positions, f_j / factor where fewer than beta_slow, a linear ramp over j
                between; mscale 0.1 ln(factor) + 1, on queries and keys alike.
                A model that scales its attention's logits by the square of that
                instead (its configuration then gives the same factor for all
                dimensions) takes the frequencies with mscale 1, and
                scale = mscale ** 2 / sqrt(head_dim) in the attention calls.
    """
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError(f"rotary_dim: {rotary_dim}, expected a positive even number")
    if not factor > 0 or not base > 0:
        raise ValueError("base and factor must be positive")
    j = torch.arange(0, rotary_dim, 2, dtype=torch.float64)
    mscale = 1.0
    if scaling == "ntk":
        if rotary_dim == 2:
            raise ValueError("ntk scaling needs rotary_dim > 2")
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = float(base) ** (-j / rotary_dim)
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        def pair_of(turns):   # the (real) pair index that turns so often within original_max positions
            return rotary_dim * math.log(original_max / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo = max(math.floor(pair_of(beta_fast)), 0)
        hi = min(math.ceil(pair_of(beta_slow)), rotary_dim - 1)
        ramp = ((torch.arange(rotary_dim // 2, dtype=torch.float64) - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f * (1 - ramp) + f / factor * ramp
        mscale = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError(f"scaling: {scaling!r}, expected None, 'linear', 'ntk' or 'yarn'")
    return f.to(device), mscale


def _rope_spec(positions, inv_freq, layout, rot_start, mscale, backward, n_tokens, dev):
    if layout not in _LAYOUTS:
        raise ValueError(f"layout: {layout!r}, expected 'half' or 'interleaved'")
    _dev(inv_freq, "inv_freq")
    half = inv_freq.shape[0]
    return _PACK_ROPE.pack(_dense(inv_freq, torch.float64, (half,), "inv_freq", dev),
                           _dense(positions, torch.int32, (n_tokens,), "positions", dev), 2 * half, rot_start,
                           _LAYOUTS[layout], 1 if backward else 0, mscale)


class _Rope(torch.autograd.Function):
    """misa_rope of an x that requires a gradient, which is the other rotation of
    the output's."""

    @staticmethod
    def forward(ctx, x, positions, inv_freq, layout, rot_start, mscale, backward):
        ctx.save_for_backward(positions, inv_freq)
        ctx.how = layout, rot_start, mscale
        ctx.turned_back = backward
        return misa_rope(x, positions, inv_freq, layout, rot_start, mscale, backward)

    @staticmethod
    def backward(ctx, g):
        positions, inv_freq = ctx.saved_tensors
        if g.stride(-1) != 1:   # (expanded, say)
            g = g.contiguous()
        return (misa_rope(g, positions, inv_freq, *ctx.how, not ctx.turned_back),) + (None,) * 6


def misa_rope(x, positions, inv_freq, layout: str = "half", rot_start: int = 0, mscale: float = 1.0,
              backward: bool = False, out=None, stream=None):
    """Rotary positions of x [tokens, heads, head_dim] (bf16, fp16 or fp32; any
    token and head strides).  inv_freq, mscale: as rope_inv_freq gives them; the
    rotary part is elements rot_start .. rot_start + 2 len(inv_freq) - 1 of a
    head.  backward: the gradient with respect to x of x -> misa_rope(x, ...),
    given the gradient of its output.  out may be x (in place).
    Where x requires a gradient the result carries it (positions and inv_freq are
    read again then, and have none themselves); a given out cannot."""
    if stream is not None:
        return _on(stream, x, "x", misa_rope, x, positions, inv_freq, layout, rot_start, mscale, backward, out)
    dev = _dev(x, "x")
    if x.requires_grad and torch.is_grad_enabled():
        if out is not None:
            raise ValueError("out takes no gradient: x requires one")
        return _Rope.apply(x, positions, inv_freq, layout, rot_start, mscale, backward)
    xp, xst, xsh = _rows(x, _DTYPES, "x", dev)
    T, H, D = x.shape
    if out is None:
        out = torch.empty((T, H, D), dtype=x.dtype, device=x.device)
    op, ost, osh = _rows(out, (x.dtype,), "out", dev, x.shape)
    spec = _rope_spec(positions, inv_freq, layout, rot_start, mscale, backward, T, dev)
    if T > 0:
        _call("misa_rope", dev, spec, xp, _DTYPES[x.dtype], T, H, D, xst, xsh, op, ost, osh)
    return out


def _pool_scale(scale, n_pages, page_keys, heads, name, dev):
    want = (n_pages, page_keys, heads)
    if scale is not None and heads == 1 and scale.dim() == 2:
        want = (n_pages, page_keys)
    return _dense(scale, torch.float32, want, name, dev)


def misa_write_pages(k, slots, k_pages, k_scale_pages=None, v=None, v_pages=None, v_scale_pages=None, positions=None,
                     inv_freq=None, layout: str = "half", rot_start: int = 0, mscale: float = 1.0, stream=None):
    """Rows k (and v) [tokens, heads, head_dim] (bf16) into their slots of the page
    pools [n_pages, page_keys, heads, head_dim] (bf16, or e4m3 codes with scale
    pools [n_pages, page_keys, heads]); with one head the pools may leave the
    head dimension out, as misa_indexer_paged takes them.  Given positions and
    inv_freq, k is rotated first (misa_rope).  Slots outside the pool are
    skipped."""
    if stream is not None:
        return _on(stream, k, "k", misa_write_pages, k, slots, k_pages, k_scale_pages, v, v_pages, v_scale_pages,
                   positions, inv_freq, layout, rot_start, mscale)
    dev = _dev(k, "k")
    kp, kst, ksh = _rows(k, _BF16, "k", dev)
    T, H, D = k.shape
    kpool, kd, n_pages, page_keys = _pool(k_pages, H, D, "k_pages", dev)
    sp = _dense(slots, torch.int64, (T,), "slots", dev)
    if (v is None) != (v_pages is None):
        raise ValueError("v and v_pages go together")
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq go together")
    vp = vst = vsh = vpool = ks = vs = spec = None
    if v is not None:
        vp, vst, vsh = _rows(v, _BF16, "v", dev, k.shape)
        vpool, *like = _pool(v_pages, H, D, "v_pages", dev)
        if like != [kd, n_pages, page_keys]:
            raise ValueError("v_pages must match k_pages")
    if kd == MISA_K_FP8_E4M3:
        ks = _pool_scale(k_scale_pages, n_pages, page_keys, H, "k_scale_pages", dev)
        if v is not None:
            vs = _pool_scale(v_scale_pages, n_pages, page_keys, H, "v_scale_pages", dev)
    if inv_freq is not None:
        spec = _rope_spec(positions, inv_freq, layout, rot_start, mscale, False, T, dev)
    if T > 0:
        _call("misa_write_pages", dev, T, H, D, kp, kst, ksh, vp, vst or 0, vsh or 0, sp,
              spec, kpool, vpool, kd, ks, vs, n_pages, page_keys)


def misa_attention_paged_workspace_bytes(shape: AttnShape, pages: KvPages) -> int:
    return int(load().misa_attention_paged_workspace_bytes(ctypes.byref(shape), ctypes.byref(pages)))


def misa_attention_selected_workspace_bytes(shape: AttnShape, pages: KvPages, topk: int) -> int:
    return int(load().misa_attention_selected_workspace_bytes(ctypes.byref(shape), ctypes.byref(pages), int(topk)))


def _attention(name, q, k_pages, v_pages, block_table, q_start, kv_lens, idx, k_scale, v_scale, scale, max_new, out, lse,
               want_lse, ws, stream):
    """idx: the selected tokens, or a tree's mask, by the call's name."""
    if stream is not None:
        return _on(stream, q, "q", _attention, name, q, k_pages, v_pages, block_table, q_start, kv_lens, idx, k_scale,
                   v_scale, scale, max_new, out, lse, want_lse, ws, None)
    dev = _dev(q, "q")
    qp, qst, qsh = _rows(q, _BF16, "q", dev)
    T, H, D = q.shape
    KH = k_pages.shape[2] if k_pages is not None and k_pages.dim() == 4 else 1
    kpool, kd, n_pages, page_keys = _pool(k_pages, KH, D, "k_pages", dev)
    vpool, *like = _pool(v_pages, KH, D, "v_pages", dev)
    if like != [kd, n_pages, page_keys]:
        raise ValueError("v_pages must match k_pages")
    ks = vs = 0
    if kd == MISA_K_FP8_E4M3:
        ks = _pool_scale(k_scale, n_pages, page_keys, KH, "k_scale_pages", dev)
        vs = _pool_scale(v_scale, n_pages, page_keys, KH, "v_scale_pages", dev)
    _dev(block_table, "block_table")
    n_seq, width = block_table.shape[0], block_table.shape[-1]
    i32 = torch.int32
    shape = _PACK_ATTN.pack(n_seq, H, KH, D, T, qst, qsh, max_new, D ** -0.5 if scale is None else scale)
    pages = _PACK_PAGES.pack(kpool, vpool, ks, vs, _dense(block_table, i32, (n_seq, width), "block_table", dev), width,
                             n_pages, page_keys, kd)
    args = [shape, pages, qp, _dense(q_start, i32, (n_seq + 1,), "q_start", dev),
            _dense(kv_lens, i32, (n_seq,), "kv_lens", dev)]
    lib = load()
    if name == "misa_attention_selected":
        _dev(idx, "idx")
        topk = idx.shape[-1]
        if idx.dim() == 3 and idx.shape[0] * idx.shape[1] == T and idx.is_contiguous():
            idx = idx.view(T, topk)
        args += [_dense(idx, i32, (T, topk), "idx", dev), topk]
    elif name == "misa_attention_tree":
        _dev(idx, "mask")
        words = idx.shape[-1]
        args += [_dense(idx, i32, (T, words), "mask", dev), words]
    if out is None:
        out = torch.empty((T, H, D), dtype=torch.bfloat16, device=q.device)
    args.append(_dense(out, torch.bfloat16, (T, H, D), "out", dev))
    if lse is None and want_lse:
        lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    args.append(None if lse is None else _dense(lse, torch.float32, (T, H), "lse", dev))
    if T == 0:
        return out, lse
    if ws is None:
        if name == "misa_attention_selected":
            need = lib.misa_attention_selected_workspace_bytes(shape, pages, topk)
        elif name == "misa_attention_tree":
            need = lib.misa_attention_tree_workspace_bytes(shape, pages)
        else:
            need = lib.misa_attention_paged_workspace_bytes(shape, pages)
        ws, at = _scratch(need, q) if need else (None, None)   # (ws stays until the call has been made)
        _call(name, dev, *args, at, need)
    else:
        if ws.get_device() != dev or not ws.is_contiguous():
            raise ValueError(f"ws must be a dense tensor on cuda:{dev}")
        _call(name, dev, *args, ws.data_ptr(), ws.numel() * ws.element_size())
    return out, lse


def misa_attention_paged(q, k_pages, v_pages, block_table, q_start, kv_lens, k_scale_pages=None, v_scale_pages=None,
                         scale=None, max_new: int = 0, out=None, lse=None, want_lse=False, ws=None, stream=None):
    """Causal attention of a ragged batch's new tokens q [tokens, heads, head_dim]
    (bf16) over its paged keys and values (pools [n_pages, page_keys, kv_heads,
    head_dim], bf16 or e4m3 codes with scale pools).  q_start int32 [n_seq + 1]
    and kv_lens int32 [n_seq] as misa_plan_pages gives them; max_new: a bound on
    the new tokens of any sequence, when the caller knows one (1 for a decode
    batch; without it the call prepares for any mix, see misa_attn_shape).
    scale: on q . k, 1 / sqrt(head_dim) unless given.  Returns (out [tokens,
    heads, head_dim] bf16, lse [tokens, heads] fp32 or None); rows from
    q_start[-1] on are left as they were."""
    return _attention("misa_attention_paged", q, k_pages, v_pages, block_table, q_start, kv_lens, None, k_scale_pages,
                      v_scale_pages, scale, max_new, out, lse, want_lse, ws, stream)


def misa_attention_selected(q, k_pages, v_pages, block_table, q_start, kv_lens, idx, k_scale_pages=None,
                            v_scale_pages=None, scale=None, max_new: int = 0, out=None, lse=None, want_lse=False,
                            ws=None, stream=None):
    """misa_attention_paged over the tokens that the indexer picked: token t reads
    tokens idx[t] (int32 [tokens, topk], or an indexer's [n_seq, M, topk]) of its
    sequence; negative entries and ones behind the token's position are absent."""
    return _attention("misa_attention_selected", q, k_pages, v_pages, block_table, q_start, kv_lens, idx, k_scale_pages,
                      v_scale_pages, scale, max_new, out, lse, want_lse, ws, stream)


def misa_plan_tree(parents, q_start, kv_lens, words: int, plan: TreePlan | None = None, stream=None) -> TreePlan:
    """The trees of drafted tokens that a step verifies: parents int32 [tokens] names
    each new token's parent among its sequence's new tokens (the last cached token:
    -1), q_start and kv_lens as misa_plan_pages gives them.  Returns the TreePlan:
    ancestor bits for misa_attention_tree, words * 32 of them at least as many as a
    sequence has new tokens, and the positions that misa_rope and misa_write_pages
    turn the tokens by (their slots are misa_plan_pages').  plan: its tensors, made
    new unless given, and none of them among this call's inputs."""
    if stream is not None:
        return _on(stream, parents, "parents", misa_plan_tree, parents, q_start, kv_lens, words, plan)
    dev = _dev(parents, "parents")
    _dev(kv_lens, "kv_lens")
    T, n = parents.shape[0], kv_lens.shape[0]
    i32 = torch.int32
    args = (n, _dense(parents, i32, (T,), "parents", dev), _dense(q_start, i32, (n + 1,), "q_start", dev),
            _dense(kv_lens, i32, (n,), "kv_lens", dev), T, words)
    if plan is None:
        mask, mp = _fresh((T, max(words, 0)), i32, parents)
        positions, pp = _fresh((T,), i32, parents)
        plan = TreePlan(mask, positions)
    else:
        mp = _dense(plan.mask, i32, (T, words), "mask", dev)
        pp = _dense(plan.positions, i32, (T,), "positions", dev)
    if T > 0:
        _call("misa_plan_tree", dev, *args, mp, pp)
    return plan


def _wants_grad(t):
    return t is not None and t.requires_grad


class _NoBackward(torch.autograd.Function):
    """A call without a backward pass, of inputs that require a gradient: its outputs require one too, and asking them
    for it is an error, where outputs cut off the graph would lose it without a word."""

    @staticmethod
    def forward(ctx, name, call, *inputs):
        ctx.call_name = name
        return call()

    @staticmethod
    def backward(ctx, *g):
        raise RuntimeError(f"{ctx.call_name} has no backward pass: detach its inputs, or call it under torch.no_grad()")


def misa_attention_tree(q, k_pages, v_pages, block_table, q_start, kv_lens, mask, k_scale_pages=None,
                        v_scale_pages=None, scale=None, max_new: int = 0, out=None, lse=None, want_lse=False, ws=None,
                        stream=None):
    """misa_attention_paged of trees of drafted tokens: a sequence's new token i sees
    its cached tokens and those new tokens j whose bit j its mask row has
    (int32 [tokens, words], as misa_plan_tree gives it or any other).  There is no
    backward pass: where q, keys or values require a gradient, asking a new out or
    lse for one raises (a given one has none)."""
    if out is None and torch.is_grad_enabled() and (_wants_grad(q) or _wants_grad(k_pages) or _wants_grad(v_pages)):
        def call():
            o, l = misa_attention_tree(q, k_pages, v_pages, block_table, q_start, kv_lens, mask, k_scale_pages,
                                       v_scale_pages, scale, max_new, None, lse, want_lse, ws, stream)
            return o, (l if lse is None else None)
        o, l = _NoBackward.apply("misa_attention_tree", call, q, k_pages, v_pages)
        return o, (l if lse is None else lse)
    return _attention("misa_attention_tree", q, k_pages, v_pages, block_table, q_start, kv_lens, mask, k_scale_pages,
                      v_scale_pages, scale, max_new, out, lse, want_lse, ws, stream)


def misa_attention_tree_workspace_bytes(shape: AttnShape, pages: KvPages) -> int:
    return int(load().misa_attention_tree_workspace_bytes(ctypes.byref(shape), ctypes.byref(pages)))


def misa_keep_path(path, q_start, kv_lens, block_table, k_pages, k_scale_pages=None, v_pages=None, v_scale_pages=None,
                   kept_lens=None, stream=None):
    """Moves an accepted path's keys (and values) to the places behind the cached
    prefix, in the pages: path int32 [n_seq, most] names each sequence's kept new
    tokens in rising order, ended by -1 (or the row's end).  Returns kept_lens int32
    [n_seq], the sequences' lengths now, the next step's cached_lens (made new unless
    given; not kv_lens itself).  One call for each layer's pages, and for the index
    keys'."""
    if stream is not None:
        return _on(stream, path, "path", misa_keep_path, path, q_start, kv_lens, block_table, k_pages, k_scale_pages,
                   v_pages, v_scale_pages, kept_lens)
    dev = _dev(path, "path")
    _dev(block_table, "block_table"), _dev(k_pages, "k_pages")
    H, D = (k_pages.shape[2] if k_pages.dim() == 4 else 1), k_pages.shape[-1]
    kpool, kd, n_pages, page_keys = _pool(k_pages, H, D, "k_pages", dev)
    vpool = ks = vs = None
    if v_pages is not None:
        vpool, *like = _pool(v_pages, H, D, "v_pages", dev)
        if like != [kd, n_pages, page_keys]:
            raise ValueError("v_pages must match k_pages")
    if kd == MISA_K_FP8_E4M3:
        ks = _pool_scale(k_scale_pages, n_pages, page_keys, H, "k_scale_pages", dev)
        if v_pages is not None:
            vs = _pool_scale(v_scale_pages, n_pages, page_keys, H, "v_scale_pages", dev)
    n, most, width = path.shape[0], path.shape[-1], block_table.shape[-1]
    i32 = torch.int32
    if kept_lens is None:
        kept_lens, kp = _fresh((n,), i32, path)
    else:
        kp = _dense(kept_lens, i32, (n,), "kept_lens", dev)
    _call("misa_keep_path", dev, n, _dense(path, i32, (n, most), "path", dev), most,
          _dense(q_start, i32, (n + 1,), "q_start", dev), _dense(kv_lens, i32, (n,), "kv_lens", dev),
          _dense(block_table, i32, (n, width), "block_table", dev), width, H, D, kpool, vpool, kd, ks, vs, n_pages,
          page_keys, kp)
    return kept_lens


def misa_quantize_blocks(x, block_rows: int = 1, codes=None, scale=None, stream=None):
    """e4m3 codes (uint8) of x [rows, columns] (bf16, fp16 or fp32; any row stride that
    keeps rows 16-byte aligned; columns a multiple of 16) and the fp32 scales of its
    blocks of block_rows x 128, [ceil(rows / block_rows), ceil(columns / 128)]:
    block_rows = 1 for activations, 128 for weights.  Codes are whole numbers: no
    gradient passes them, nor the scales."""
    if stream is not None:
        return _on(stream, x, "x", misa_quantize_blocks, x, block_rows, codes, scale)
    dev = _dev(x, "x")
    at, st = _matrix(x, _DTYPES, "x", dev)
    R, K = x.shape
    if block_rows not in (1, 128):
        raise ValueError(f"block_rows: {block_rows}, expected 1 or 128")
    blocks = (-(-R // block_rows), -(-K // 128))
    if codes is None:
        codes, cp = _fresh((R, K), torch.uint8, x)
    else:
        cp = _dense(codes, codes.dtype if codes.dtype in _CODES else torch.uint8, (R, K), "codes", dev)
    if scale is None:
        scale, sp = _fresh(blocks, torch.float32, x)
    else:
        sp = _dense(scale, torch.float32, blocks, "scale", dev)
    if R > 0:
        _call("misa_quantize_blocks", dev, at, _DTYPES[x.dtype], R, K, st, block_rows, cp, sp)
    return codes, scale


def misa_matmul_q8_workspace_bytes(m: int, n: int, k: int) -> int:
    return int(load().misa_matmul_q8_workspace_bytes(m, n, k))


def misa_matmul_q8(x, x_scale, w, w_scale, out=None, ws=None, stream=None):
    """x w^T in bf16 of e4m3 codes x [m, k] with a scale for each 1 x 128 block and w [n, k] with one for each
    128 x 128 (misa_quantize_blocks; uint8 or float8_e4m3fn, rows 16-byte aligned, k a
    multiple of 16).  out: bf16 [m, n], its last dimension dense; it has no gradient."""
    if stream is not None:
        return _on(stream, x, "x", misa_matmul_q8, x, x_scale, w, w_scale, out, ws)
    dev = _dev(x, "x")
    xp, xst = _matrix(x, _CODES, "x", dev)
    wp, wst = _matrix(w, _CODES, "w", dev)
    (M, K), N = x.shape, w.shape[0]
    if w.shape[1] != K:
        raise ValueError(f"w: shape {tuple(w.shape)}, expected ({N}, {K})")
    across = (K + 127) // 128
    if out is None:
        out, op = _fresh((M, N), torch.bfloat16, x)
        ost = N
    else:
        op, ost = _matrix(out, _BF16, "out", dev, (M, N))
    args = (M, N, K, xp, xst, _dense(x_scale, torch.float32, (M, across), "x_scale", dev), wp, wst,
            _dense(w_scale, torch.float32, ((N + 127) // 128, across), "w_scale", dev), op, ost)
    if M == 0:
        return out
    lib = load()
    if ws is None:
        need = lib.misa_matmul_q8_workspace_bytes(M, N, K)
        ws, at = _scratch(need, x) if need else (None, None)   # (ws stays until the call has been made)
    else:
        if ws.get_device() != dev or not ws.is_contiguous():
            raise ValueError(f"ws must be a dense tensor on cuda:{dev}")
        at, need = ws.data_ptr(), ws.numel() * ws.element_size()
    _call("misa_matmul_q8", dev, *args, at, need)
    return out
