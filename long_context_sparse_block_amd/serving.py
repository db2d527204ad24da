"""The paged serving step around the indexer (C ABI in include/misa.h): page
planning from request lengths, rotary positions, the write of new keys and
values into their pages, and attention over the pages or over the tokens that
the indexer picked.

As in _lib: argument marshalling only, raw device pointers and the current HIP
stream (of the tensors' own device) go to the library, and there is no
fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import NamedTuple

import torch

from ._lib import MISA_K_BF16, MISA_K_FP8_E4M3, _check, _kdtype, _need, _ptr, load

MISA_T_BF16, MISA_T_FP16, MISA_T_FP32 = 0, 1, 2
_DTYPES = {torch.bfloat16: MISA_T_BF16, torch.float16: MISA_T_FP16, torch.float32: MISA_T_FP32}
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


def _on(t, stream):
    """The device guard for t's device and the stream handle of a call on it."""
    dev = t.device
    guard = contextlib.nullcontext() if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)
    s = torch.cuda.current_stream(dev) if stream is None else stream
    return guard, ctypes.c_void_p(s.cuda_stream)


def _same_device(first, **others):
    for name, t in others.items():
        if t is not None and t.device != first.device:
            raise ValueError(f"{name} is on {t.device}, expected {first.device}")


def _rows(t, dtypes, name, shape=None):
    """A [tokens, heads, head_dim] tensor whose last dimension is dense; its token and head strides."""
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected one of {tuple(dtypes)}")
    if t.dim() != 3 or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {'[tokens, heads, head_dim]' if shape is None else tuple(shape)}")
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"{name}: the last dimension must be dense")
    # the strides of dimensions of one element mean nothing
    return (t.stride(0) if t.shape[0] > 1 else 0), (t.stride(1) if t.shape[1] > 1 else 0)


def misa_plan_pages(cached_lens, new_lens, free_pages, block_table, page_keys: int, n_tokens: int,
                    plan: PagePlan | None = None, stream=None) -> PagePlan:
    """Pages for the new tokens of every sequence: writes the new entries of
    block_table [n_seq, max_pages] (int32, in place) from free_pages (int32) and
    returns the PagePlan.  n_tokens: length of the slot map (at least the sum of
    new_lens; entries behind the last token get slot -1)."""
    n = int(cached_lens.shape[0])
    _need(cached_lens, torch.int32, (n,), "cached_lens")
    _need(new_lens, torch.int32, (n,), "new_lens")
    _need(free_pages, torch.int32, (free_pages.shape[0],), "free_pages")
    _need(block_table, torch.int32, (n, block_table.shape[-1]), "block_table")
    dev = cached_lens.device
    if plan is None:
        plan = PagePlan(torch.empty(n + 1, dtype=torch.int32, device=dev),
                        torch.empty(n, dtype=torch.int32, device=dev),
                        torch.empty(n_tokens, dtype=torch.int64, device=dev),
                        torch.empty(n_tokens, dtype=torch.int32, device=dev),
                        torch.empty(1, dtype=torch.int32, device=dev))
    else:
        _need(plan.q_start, torch.int32, (n + 1,), "q_start")
        _need(plan.kv_lens, torch.int32, (n,), "kv_lens")
        _need(plan.slots, torch.int64, (n_tokens,), "slots")
        _need(plan.positions, torch.int32, (n_tokens,), "positions")
        _need(plan.n_taken, torch.int32, (1,), "n_taken")
    _same_device(cached_lens, new_lens=new_lens, free_pages=free_pages, block_table=block_table, q_start=plan.q_start,
                 kv_lens=plan.kv_lens, slots=plan.slots, positions=plan.positions, n_taken=plan.n_taken)
    guard, s = _on(cached_lens, stream)
    with guard:
        st = load().misa_plan_pages(n, _ptr(cached_lens), _ptr(new_lens), int(page_keys), _ptr(free_pages),
                                    int(free_pages.shape[0]), _ptr(block_table), int(block_table.shape[1]),
                                    _ptr(plan.q_start), _ptr(plan.kv_lens), _ptr(plan.slots), _ptr(plan.positions),
                                    int(n_tokens), _ptr(plan.n_taken), s)
    _check(st, "misa_plan_pages")
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
                between; mscale 0.1 ln(factor) + 1
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


def _rope_spec(positions, inv_freq, layout, rot_start, mscale, backward, n_tokens, like):
    if layout not in _LAYOUTS:
        raise ValueError(f"layout: {layout!r}, expected 'half' or 'interleaved'")
    _need(positions, torch.int32, (n_tokens,), "positions")
    _need(inv_freq, torch.float64, (inv_freq.shape[0],), "inv_freq")
    _same_device(like, positions=positions, inv_freq=inv_freq)
    return RopeSpec(inv_freq.data_ptr(), positions.data_ptr(), 2 * int(inv_freq.shape[0]), int(rot_start),
                    _LAYOUTS[layout], int(bool(backward)), float(mscale))


def misa_rope(x, positions, inv_freq, layout: str = "half", rot_start: int = 0, mscale: float = 1.0,
              backward: bool = False, out=None, stream=None):
    """Rotary positions of x [tokens, heads, head_dim] (bf16, fp16 or fp32; any
    token and head strides).  inv_freq, mscale: as rope_inv_freq gives them; the
    rotary part is elements rot_start .. rot_start + 2 len(inv_freq) - 1 of a
    head.  backward: the gradient with respect to x of x -> misa_rope(x, ...),
    given the gradient of its output.  out may be x (in place)."""
    xst, xsh = _rows(x, _DTYPES, "x")
    T, H, D = x.shape
    if out is None:
        out = torch.empty((T, H, D), dtype=x.dtype, device=x.device)
    ost, osh = _rows(out, (x.dtype,), "out", x.shape)
    _same_device(x, out=out)
    spec = _rope_spec(positions, inv_freq, layout, rot_start, mscale, backward, T, x)
    if T == 0:
        return out
    guard, s = _on(x, stream)
    with guard:
        st = load().misa_rope(ctypes.byref(spec), _ptr(x), _DTYPES[x.dtype], T, H, D, xst, xsh, _ptr(out), ost, osh, s)
    _check(st, "misa_rope")
    return out


def _pool(pages, heads, head_dim, name):
    """kdtype, n_pages, page_keys of a page pool [n_pages, page_keys, heads, head_dim]
    (or [n_pages, page_keys, head_dim] of one head)."""
    if pages is None:
        raise ValueError(f"{name} is required")
    kd = _kdtype(pages)
    n_pages, page_keys = int(pages.shape[0]), int(pages.shape[1])
    if pages.dim() == 3 and heads == 1:
        _need(pages, pages.dtype, (n_pages, page_keys, head_dim), name)
    else:
        _need(pages, pages.dtype, (n_pages, page_keys, heads, head_dim), name)
    return kd, n_pages, page_keys


def _pool_scale(scale, n_pages, page_keys, heads, name):
    if scale is not None and scale.dim() == 2 and heads == 1:
        _need(scale, torch.float32, (n_pages, page_keys), name)
    else:
        _need(scale, torch.float32, (n_pages, page_keys, heads), name)


def misa_write_pages(k, slots, k_pages, k_scale_pages=None, v=None, v_pages=None, v_scale_pages=None, positions=None,
                     inv_freq=None, layout: str = "half", rot_start: int = 0, mscale: float = 1.0, stream=None):
    """Rows k (and v) [tokens, heads, head_dim] (bf16) into their slots of the page
    pools [n_pages, page_keys, heads, head_dim] (bf16, or e4m3 codes with scale
    pools [n_pages, page_keys, heads]); with one head the pools may leave the
    head dimension out, as misa_indexer_paged takes them.  Given positions and
    inv_freq, k is rotated first (misa_rope).  Slots outside the pool are
    skipped."""
    kst, ksh = _rows(k, (torch.bfloat16,), "k")
    T, H, D = k.shape
    kd, n_pages, page_keys = _pool(k_pages, H, D, "k_pages")
    _need(slots, torch.int64, (T,), "slots")
    vst = vsh = 0
    if (v is None) != (v_pages is None):
        raise ValueError("v and v_pages go together")
    if v is not None:
        vst, vsh = _rows(v, (torch.bfloat16,), "v", k.shape)
        if _pool(v_pages, H, D, "v_pages") != (kd, n_pages, page_keys):
            raise ValueError("v_pages must match k_pages")
    if kd == MISA_K_FP8_E4M3:
        _pool_scale(k_scale_pages, n_pages, page_keys, H, "k_scale_pages")
        if v is not None:
            _pool_scale(v_scale_pages, n_pages, page_keys, H, "v_scale_pages")
    _same_device(k, slots=slots, k_pages=k_pages, k_scale_pages=k_scale_pages, v=v, v_pages=v_pages,
                 v_scale_pages=v_scale_pages)
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq go together")
    spec = None
    if inv_freq is not None:
        spec = ctypes.byref(_rope_spec(positions, inv_freq, layout, rot_start, mscale, False, T, k))
    if T == 0:
        return
    guard, s = _on(k, stream)
    with guard:
        st = load().misa_write_pages(T, H, D, _ptr(k), kst, ksh, _ptr(v), vst, vsh, _ptr(slots), spec, _ptr(k_pages),
                                     _ptr(v_pages), kd, _ptr(k_scale_pages), _ptr(v_scale_pages), n_pages, page_keys,
                                     s)
    _check(st, "misa_write_pages")


def _attn_structs(q, k_pages, v_pages, block_table, n_kv_heads, k_scale, v_scale, scale, max_new):
    qst, qsh = _rows(q, (torch.bfloat16,), "q")
    T, H, D = q.shape
    kd, n_pages, page_keys = _pool(k_pages, n_kv_heads, D, "k_pages")
    if _pool(v_pages, n_kv_heads, D, "v_pages") != (kd, n_pages, page_keys):
        raise ValueError("v_pages must match k_pages")
    if kd == MISA_K_FP8_E4M3:
        _pool_scale(k_scale, n_pages, page_keys, n_kv_heads, "k_scale_pages")
        _pool_scale(v_scale, n_pages, page_keys, n_kv_heads, "v_scale_pages")
    n_seq = int(block_table.shape[0])
    _need(block_table, torch.int32, (n_seq, block_table.shape[-1]), "block_table")
    shape = AttnShape(n_seq, H, n_kv_heads, D, T, qst, qsh, int(max_new),
                      1.0 / math.sqrt(D) if scale is None else float(scale))
    pages = KvPages(k_pages.data_ptr(), v_pages.data_ptr(), k_scale.data_ptr() if kd == MISA_K_FP8_E4M3 else None,
                    v_scale.data_ptr() if kd == MISA_K_FP8_E4M3 else None, block_table.data_ptr(),
                    int(block_table.shape[1]), n_pages, page_keys, kd)
    return shape, pages


def misa_attention_paged_workspace_bytes(shape: AttnShape, pages: KvPages) -> int:
    return int(load().misa_attention_paged_workspace_bytes(ctypes.byref(shape), ctypes.byref(pages)))


def misa_attention_selected_workspace_bytes(shape: AttnShape, pages: KvPages, topk: int) -> int:
    return int(load().misa_attention_selected_workspace_bytes(ctypes.byref(shape), ctypes.byref(pages), int(topk)))


def _attention(name, q, k_pages, v_pages, block_table, q_start, kv_lens, idx, k_scale, v_scale, scale, max_new, out, lse,
               want_lse, ws, stream):
    if k_pages is None:
        raise ValueError("k_pages is required")
    n_kv = int(k_pages.shape[2]) if k_pages.dim() == 4 else 1
    shape, pages = _attn_structs(q, k_pages, v_pages, block_table, n_kv, k_scale, v_scale, scale, max_new)
    T, H, D = q.shape
    _need(q_start, torch.int32, (shape.n_seq + 1,), "q_start")
    _need(kv_lens, torch.int32, (shape.n_seq,), "kv_lens")
    topk = 0
    if name == "misa_attention_selected":
        if idx is None:
            raise ValueError("idx is required")
        topk = int(idx.shape[-1])
        idx = idx.reshape(T, topk) if idx.dim() == 3 and idx.is_contiguous() and idx.shape[0] * idx.shape[1] == T else idx
        _need(idx, torch.int32, (T, topk), "idx")
    if out is None:
        out = torch.empty((T, H, D), dtype=torch.bfloat16, device=q.device)
    _need(out, torch.bfloat16, (T, H, D), "out")
    if lse is None and want_lse:
        lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, torch.float32, (T, H), "lse")
    _same_device(q, k_pages=k_pages, v_pages=v_pages, block_table=block_table, q_start=q_start, kv_lens=kv_lens, idx=idx,
                 k_scale_pages=k_scale, v_scale_pages=v_scale, out=out, lse=lse, ws=ws)
    lib = load()
    sp, pp = ctypes.byref(shape), ctypes.byref(pages)
    if T == 0:
        return out, lse
    guard, s = _on(q, stream)
    with guard:
        if ws is None:
            need = (lib.misa_attention_selected_workspace_bytes(sp, pp, topk) if idx is not None
                    else lib.misa_attention_paged_workspace_bytes(sp, pp))
            if need:
                ws = torch.empty(need, dtype=torch.uint8, device=q.device)
                if stream is not None:   # the block may be reused once `stream` has passed this call
                    ws.record_stream(stream)
        nb = 0 if ws is None else ws.numel() * ws.element_size()
        if idx is not None:
            st = lib.misa_attention_selected(sp, pp, _ptr(q), _ptr(q_start), _ptr(kv_lens), _ptr(idx), topk, _ptr(out),
                                             _ptr(lse), _ptr(ws), nb, s)
        else:
            st = lib.misa_attention_paged(sp, pp, _ptr(q), _ptr(q_start), _ptr(kv_lens), _ptr(out), _ptr(lse),
                                          _ptr(ws), nb, s)
    _check(st, name)
    return out, lse


def misa_attention_paged(q, k_pages, v_pages, block_table, q_start, kv_lens, k_scale_pages=None, v_scale_pages=None,
                         scale=None, max_new: int = 0, out=None, lse=None, want_lse=False, ws=None, stream=None):
    """Causal attention of a ragged batch's new tokens q [tokens, heads, head_dim]
    (bf16) over its paged keys and values (pools [n_pages, page_keys, kv_heads,
    head_dim], bf16 or e4m3 codes with scale pools).  q_start int32 [n_seq + 1]
    and kv_lens int32 [n_seq] as misa_plan_pages gives them; max_new: a bound on
    the new tokens of any sequence, when the caller knows one (1 for a decode
    batch).  scale: on q . k, 1 / sqrt(head_dim) unless given.  Returns (out
    [tokens, heads, head_dim] bf16, lse [tokens, heads] fp32 or None); rows from
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
