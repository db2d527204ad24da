"""Plain fp64 forms of the paged serving operators, on the CPU, and the bounds
their kernels are held to."""
import math

import numpy as np
import torch

BF16_HALF = 2.0 ** -8    # half a step of bf16, relative
F32_HALF = 2.0 ** -24


def plan(cached, new, free, table, page, n_tokens):
    """misa_plan_pages in Python integers."""
    cached, new = [max(int(c), 0) for c in cached], [max(int(m), 0) for m in new]
    table = [list(map(int, r)) for r in table]
    width = len(table[0])
    q_start, slots, pos, used = [0], [], [], 0
    for b, (c, m) in enumerate(zip(cached, new)):
        q_start.append(q_start[-1] + m)
        have, end = min(-(-c // page), width), min(-(-(c + m) // page), width)
        for j in range(have, end):
            table[b][j] = int(free[used]) if used < len(free) else -1
            used += 1
        for p in range(c, c + m):
            if len(slots) >= n_tokens:
                break
            e = table[b][p // page] if p // page < width else -1
            slots.append(e * page + p % page if e >= 0 else -1)
            pos.append(p)
    slots += [-1] * (n_tokens - len(slots))
    pos += [-1] * (n_tokens - len(pos))
    return dict(table=table, q_start=q_start, kv_lens=[c + m for c, m in zip(cached, new)], slots=slots, positions=pos,
                n_taken=[used])


def rope(x, pos, f, layout, start, mscale, backward=False):
    """fp64 rotation, element by element of the pair list."""
    y = x.double().clone()
    half = f.numel()
    ang = pos.double()[:, None] * f.double()[None]
    c, s = torch.cos(ang) * mscale, torch.sin(ang) * mscale * (-1 if backward else 1)
    for j in range(half):
        ia, ib = (start + j, start + j + half) if layout == "half" else (start + 2 * j, start + 2 * j + 1)
        a, b = x[..., ia].double(), x[..., ib].double()
        y[..., ia] = a * c[:, None, j] - b * s[:, None, j]
        y[..., ib] = a * s[:, None, j] + b * c[:, None, j]
    return y


class Paged:
    """A ragged batch over a shuffled page pool.  Pages nobody owns, and rows behind a sequence's end, hold NaN."""

    def __init__(self, seed, kv_lens, new, heads, kv_heads, dim, page, fp8=False, spare=3, width=None, pad_rows=0):
        g = torch.Generator().manual_seed(seed)
        n = len(kv_lens)
        self.page, self.heads, self.kv_heads, self.dim, self.fp8 = page, heads, kv_heads, dim, fp8
        need = [-(-l // page) for l in kv_lens]
        self.width = max(need + [1]) if width is None else width
        n_pages = sum(need) + spare
        ids = torch.randperm(n_pages, generator=g).tolist()
        self.table = torch.zeros((n, self.width), dtype=torch.int32)   # entries behind the end: some page (0)
        shape = (n_pages, page, kv_heads, dim)
        rows = [torch.randn(shape, generator=g) for _ in range(2)]
        live = torch.zeros((n_pages, page), dtype=torch.bool)
        for b, l in enumerate(kv_lens):
            for j in range(need[b]):
                p = ids.pop()
                self.table[b, j] = p
                live[p, :min(page, l - j * page)] = True
        self.live = live
        if fp8:
            self.scale = [x.abs().amax(-1) / 448 for x in rows]
            self.codes = [(x / s[..., None]).to(torch.float8_e4m3fn) for x, s in zip(rows, self.scale)]
            self.vals = [c.double() * s.double()[..., None] for c, s in zip(self.codes, self.scale)]
            for s in self.scale:
                s[~live] = float("nan")
            self.pages = [c.view(torch.uint8).clone() for c in self.codes]
            for c in self.pages:
                c[~live] = 0x7F   # e4m3fn NaN
        else:
            self.scale = [None, None]
            self.pages = [x.bfloat16() for x in rows]
            self.vals = [x.double() for x in self.pages]
            for x in self.pages:
                x[~live] = float("nan")
        self.kv_lens = torch.tensor(kv_lens, dtype=torch.int32)
        self.q_start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
        self.tokens = int(self.q_start[-1])
        self.q = (2 * torch.randn((self.tokens + pad_rows, heads, dim), generator=g)).bfloat16()
        self.gen = g

    def seq_of(self, t):
        return int(torch.searchsorted(self.q_start[1:].contiguous(), t, right=True))

    def pos(self, t):
        b = self.seq_of(t)
        return int(self.kv_lens[b]) - int(self.q_start[b + 1]) + t

    def select(self, topk, holes=0.0):
        """Random distinct tokens of each query's prefix, -1 behind them (and, with holes, among them)."""
        idx = torch.full((self.q.shape[0], topk), -1, dtype=torch.int32)
        for t in range(self.tokens):
            n = self.pos(t) + 1
            if n <= 0:
                continue
            pick = torch.randperm(n, generator=self.gen)[:topk].to(torch.int32)
            idx[t, :len(pick)] = pick
        if holes:
            idx[torch.rand(idx.shape, generator=self.gen) < holes] = -1
        return idx

    def rows(self, which, b, toks):
        """fp64 [len(toks), kv_heads, dim]"""
        toks = torch.as_tensor(toks, dtype=torch.long)
        return self.vals[which][self.table[b].long()[toks // self.page], toks % self.page]

    def gpu(self):
        d = dict(q=self.q, k_pages=self.pages[0], v_pages=self.pages[1], block_table=self.table, q_start=self.q_start,
                 kv_lens=self.kv_lens, k_scale_pages=self.scale[0], v_scale_pages=self.scale[1])
        return {k: None if v is None else v.cuda() for k, v in d.items()}


def attention(p: Paged, idx=None, scale=None):
    """out, lse (fp64), and the bounds on the kernel's errors of both.

    The kernel rounds out (half a bf16 step of it) and each softmax weight (half a bf16 step of w_s |v_s|, so
    2^-8 A with A = sum_s p_s |v_s|); a score's fp32 error e (a dot product of D fp32 products, its scaling, the
    subtraction and exp2, each good to a few 2^-24 of |score| + 1) moves a weight by the factor 1 + e and, through
    the sum, every weight by the same: 2 e A.  Sums over n keys in fp32 add n 2^-24 of A; the log-sum moves by
    e + n 2^-24 and its own rounding."""
    scale = 1 / math.sqrt(p.dim) if scale is None else scale
    T, G = p.tokens, p.heads // p.kv_heads
    out = torch.zeros((T, p.heads, p.dim), dtype=torch.float64)
    lse = torch.full((T, p.heads), -math.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    groups = {}
    if idx is None:
        for b in range(len(p.kv_lens)):
            t0, t1, n = int(p.q_start[b]), int(p.q_start[b + 1]), int(p.kv_lens[b])
            if t1 > t0 and n > 0:
                groups[b] = (list(range(t0, t1)), torch.arange(n))
    work = groups.items() if idx is None else [((t, p.seq_of(t)), ([t], None)) for t in range(T)]
    for key, (ts, toks) in work:
        b = key if idx is None else key[1]
        if idx is not None:
            toks = idx[ts[0]].long()
            toks = toks[(toks >= 0) & (toks <= p.pos(ts[0]))]
        if len(toks) == 0:
            continue
        k, v = p.rows(0, b, toks), p.rows(1, b, toks)
        pos = torch.tensor([p.pos(t) for t in ts])
        seen = toks[None, :] <= pos[:, None]
        q = p.q[ts].double()
        for h in range(p.heads):
            kh, vh = k[:, h // G], v[:, h // G]
            s = (q[:, h] @ kh.T) * scale
            mag = (q[:, h].abs() @ kh.abs().T) * abs(scale)
            s = s.masked_fill(~seen, -math.inf)
            l = torch.logsumexp(s, 1)
            w = torch.exp(s - torch.where(l > -math.inf, l, 0.0)[:, None])
            A = w @ vh.abs()
            o = w @ vh
            n = len(toks)
            e = ((p.dim + 8) * F32_HALF * mag.masked_fill(~seen, 0).amax(1) + 8 * F32_HALF * (1 + s.masked_fill(~seen, 0).abs().amax(1)))
            out[ts, h], lse[ts, h] = o, l
            tol[ts, h] = BF16_HALF * o.abs() + (BF16_HALF + 2 * e + n * F32_HALF)[:, None] * A * 1.01
            ltol[ts, h] = e + n * F32_HALF + 4 * F32_HALF * l.abs().nan_to_num(0, 0, 0)
    return out, lse, tol, ltol


def check_attention(p, got, lse, idx=None, scale=None):
    ref, rl, tol, ltol = attention(p, idx, scale)
    got, lse = got.double().cpu(), lse.double().cpu()
    assert torch.isfinite(got[:p.tokens]).all()
    over = (got[:p.tokens] - ref).abs() - tol
    assert float(over.max() if over.numel() else -1) <= 0, f"out over its bound by {float(over.max()):.3e}"
    empty = rl == -math.inf
    assert torch.equal(lse[:p.tokens] == -math.inf, empty)
    d = (lse[:p.tokens] - rl)[~empty].abs() - ltol[~empty]
    assert float(d.max() if d.numel() else -1) <= 0, f"lse over its bound by {float(d.max()):.3e}"
