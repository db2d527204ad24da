"""Plain 64-bit forms of the drafted trees' operators and of e4m3 products, on the
CPU, and the bounds their kernels are held to."""
import math

import numpy as np
import torch

from serving_helpers import BF16_HALF, F32_HALF

FP8 = torch.float8_e4m3fn


def random_parents(g, m, kind="tree"):
    """Parents of one sequence's m new tokens."""
    if kind == "chain":
        return [i - 1 for i in range(m)]
    if kind == "star":
        return [-1] + [0] * (m - 1) if m else []
    if kind == "forest":   # nobody has a parent
        return [-1] * m
    up = [-1]
    for i in range(1, m):
        up.append(i - 1 - int(torch.randint(0, min(i, 6), (1,), generator=g)))
    return up[:m]


def ancestors(parents):
    """bool [m, m]: token j is an ancestor of token i, or i itself.  A parent that is not before its child is none."""
    m = len(parents)
    sees = np.zeros((m, m), dtype=bool)
    for i in range(m):
        p = parents[i]
        if 0 <= p < i:
            sees[i] = sees[p]
        sees[i, i] = True
    return sees


def pack(sees, words):
    """Rows of bits as int32 words."""
    m, width = sees.shape[0], 32 * words
    full = np.zeros((m, width), dtype=bool)
    n = min(width, sees.shape[1])
    full[:, :n] = sees[:, :n]
    bits = (full.reshape(m, words, 32).astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(2).astype(np.uint32)
    return torch.from_numpy(bits.view(np.int32).reshape(m, words).copy())


def plan(parents, q_start, kv_lens, n_tokens, words):
    """misa_plan_tree of all sequences (parents: the whole list of n_tokens)."""
    mask = torch.zeros((n_tokens, words), dtype=torch.int32)
    pos = torch.full((n_tokens,), -1, dtype=torch.int32)
    for b in range(len(kv_lens)):
        t0, t1 = q_start[b], q_start[b + 1]
        if t1 > t0:
            sees = ancestors([int(p) for p in parents[t0:t1]])
            mask[t0:t1] = pack(sees, words)
            pos[t0:t1] = torch.from_numpy(sees.sum(1).astype(np.int32) - 1 + kv_lens[b] - (t1 - t0))
    return mask, pos


def unpack(mask):
    """int32 [T, words] -> bool [T, 32 words]"""
    m = mask.numpy().view(np.uint32)
    return torch.from_numpy(((m[:, :, None] >> np.arange(32, dtype=np.uint32)) & 1).astype(bool).reshape(m.shape[0], -1))


def attention(p, mask, scale=None):
    """out, lse (fp64) of a serving_helpers.Paged batch under the mask, and the bounds on the kernel's errors of both.

    The kernel rounds out (half a bf16 step of it) and each softmax weight (half a bf16 step of w_s |v_s|, so 2^-8 A
    with A = sum_s p_s |v_s|); a score's fp32 error e (a dot product of D fp32 products, its scaling, the subtraction and
    exp2, each good to a few 2^-24 of |score| + 1) moves a weight by the factor 1 + e and, through the sum, every weight
    by the same: 2 e A.  Sums over n keys in fp32 add n 2^-24 of A; the log-sum moves by e + n 2^-24 and its own
    rounding."""
    scale = 1 / math.sqrt(p.dim) if scale is None else scale
    T, G = p.tokens, p.heads // p.kv_heads
    out = torch.zeros((T, p.heads, p.dim), dtype=torch.float64)
    lse = torch.full((T, p.heads), -math.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    bits = unpack(mask[:T])
    for b in range(len(p.kv_lens)):
        t0, t1, n = int(p.q_start[b]), int(p.q_start[b + 1]), int(p.kv_lens[b])
        m = t1 - t0
        if m == 0 or n == 0:
            continue
        seen = torch.zeros((m, n), dtype=torch.bool)
        seen[:, :n - m] = True
        w = min(m, bits.shape[1])
        seen[:, n - m:n - m + w] = bits[t0:t1, :w]
        k, v = p.rows(0, b, torch.arange(n)), p.rows(1, b, torch.arange(n))
        q = p.q[t0:t1].double()
        for h in range(p.heads):
            kh, vh = k[:, h // G], v[:, h // G]
            s = ((q[:, h] @ kh.T) * scale).masked_fill(~seen, -math.inf)
            mag = (q[:, h].abs() @ kh.abs().T) * abs(scale)
            l = torch.logsumexp(s, 1)
            wt = torch.exp(s - torch.where(l > -math.inf, l, 0.0)[:, None])
            A, o = wt @ vh.abs(), wt @ vh
            e = ((p.dim + 8) * F32_HALF * mag.masked_fill(~seen, 0).amax(1)
                 + 8 * F32_HALF * (1 + s.masked_fill(~seen, 0).abs().amax(1)))
            out[t0:t1, h], lse[t0:t1, h] = o, l
            tol[t0:t1, h] = BF16_HALF * o.abs() + (BF16_HALF + 2 * e + n * F32_HALF)[:, None] * A * 1.01
            ltol[t0:t1, h] = e + n * F32_HALF + 4 * F32_HALF * l.abs().nan_to_num(0, 0, 0)
    return out, lse, tol, ltol


def check_attention(p, got, lse, mask, scale=None):
    ref, rl, tol, ltol = attention(p, mask, scale)
    got, lse = got.double().cpu(), lse.double().cpu()
    assert torch.isfinite(got[:p.tokens]).all()
    over = (got[:p.tokens] - ref).abs() - tol
    assert float(over.max() if over.numel() else -1) <= 0, f"out over its bound by {float(over.max()):.3e}"
    empty = rl == -math.inf
    assert torch.equal(lse[:p.tokens] == -math.inf, empty)
    d = (lse[:p.tokens] - rl)[~empty].abs() - ltol[~empty]
    assert float(d.max() if d.numel() else -1) <= 0, f"lse over its bound by {float(d.max()):.3e}"


def keep(path, q_start, kv_lens, table, page, pools):
    """misa_keep_path in Python: the pools' rows after it (new tensors), and the kept lengths."""
    flat = [x.clone().view(-1, *x.shape[2:]) for x in pools]
    n_slots, kept = flat[0].shape[0], []
    for b, nodes in enumerate(path.tolist()):
        m = int(q_start[b + 1]) - int(q_start[b])
        first, c, last = int(kv_lens[b]) - m, 0, -1

        def slot(t):
            if t < 0 or t // page >= table.shape[1]:
                return -1
            e = int(table[b, t // page])
            return e * page + t % page if 0 <= e < n_slots // page else -1
        for node in nodes:
            if node <= last or node >= m:
                break
            s, d = slot(first + node), slot(first + c)
            if s >= 0 and d >= 0:
                for x in flat:
                    x[d] = x[s].clone()
            last, c = node, c + 1
        kept.append(max(0, first + c))
    return [x.view(y.shape) for x, y in zip(flat, pools)], kept


def quantize(x, block_rows):
    """Codes (bytes) and scales by the definition: fp32 quotients of values held exactly, so plain fp32 divisions."""
    r, k = x.shape
    up, across = -(-r // block_rows), -(-k // 128)
    y = torch.zeros((up * block_rows, across * 128), dtype=torch.float32)
    y[:r, :k] = x.float()
    y = y.view(up, block_rows, across, 128)
    amax = y.abs().nan_to_num(nan=0.0, posinf=math.inf).amax((1, 3))
    scale = torch.where(amax > 0, (amax / torch.full_like(amax, 448)).clamp(min=2.0 ** -126), 1.0)
    q = y / scale[:, None, :, None]
    codes = q.to(FP8).view(torch.uint8)
    codes = torch.where(torch.isnan(q), torch.full_like(codes, 0x7F) | ((codes & 0x80)), codes)
    return codes.view(up * block_rows, across * 128)[:r, :k].contiguous(), scale


def values(codes, scale, block_rows):
    """fp64 values of codes."""
    r, k = codes.shape
    s = scale.double().repeat_interleave(block_rows, 0)[:r].repeat_interleave(128, 1)[:, :k]
    return codes.contiguous().view(torch.uint8).view(FP8).double() * s


def product(x8, xs, w8, ws):
    """out (fp64) and the bound on the kernel's error.  The matrix unit sums eight neighbouring products at a time, each
    cut (towards 0) at 2^-13 of the power of two in the largest of the eight, which itself keeps all its 8 bits: 7 x
    2^-13 of the largest, at most, for each eight (measured: +1, -1 in another eight and 2^-13 beside the first leave
    2^-13, with 2^-14 nothing).  Beside that the sums of the eights, the product of two scales and the scaled addition of
    each block in fp32, (16 + blocks + 3) 2^-24 of the sum of |x w|, and half a bf16 step of the result."""
    x, w = values(x8, xs, 1), values(w8, ws, 128)
    ref, mag = x @ w.T, x.abs() @ w.abs().T
    m, k = x.shape
    if m * k * w.shape[0] <= 1 << 27:
        top = torch.zeros_like(ref)
        for g in range(0, k, 8):
            most = torch.zeros_like(ref, dtype=torch.float32)
            for i in range(g, g + 8):
                torch.maximum(most, x[:, i, None].abs().float() * w[None, :, i].abs().float(), out=most)
            top += most.double()
        top *= 1 + 2.0 ** -20
    else:
        top = mag   # (the largest of eight is at most their sum)
    tol = BF16_HALF * ref.abs() + (7 * 2.0 ** -13 * top + (xs.shape[1] + 19) * F32_HALF * mag) * 1.01
    return ref, tol


def check_product(got, x8, xs, w8, ws):
    ref, tol = product(x8, xs, w8, ws)
    over = (got.double().cpu() - ref).abs() - tol
    assert torch.isfinite(got).all()
    assert float(over.max()) <= 0, f"over its bound by {float(over.max()):.3e}"
