"""GPU parity of the paged serving operators against plain fp64 forms: page
planning, rotary positions, page writes, attention over the pages and over
selected tokens, and a serving step that runs them around misa_indexer_paged."""
import math

import pytest
import torch

import long_context_sparse_block_amd as misa
import serving_helpers as ref
from gpu_helpers import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the -m gpu tests need an MI355X")
    misa.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- page planning

PLANS = [   # cached, new, page, spare table columns, free pages held back, slots past the end
    ([0], [1], 64, 0, 0, 0),
    ([63, 64, 65, 0], [1, 1, 1, 0], 64, 1, 0, 3),
    ([5, 0, 131071, 17], [300, 0, 1, 16], 16, 2, 0, 100),
    ([0, 0, 0], [0, 0, 0], 64, 0, 0, 5),            # nothing new
    ([10, 20], [40, 50], 1, 0, 0, 0),               # pages of one token
    ([10, 20, 30], [100, 100, 100], 7, 3, 12, 9),   # the free list runs out
    ([10, 20], [100, 100], 16, -4, 0, 0),           # tokens past the table
    ([-5, 3], [4, -2], 4, 1, 0, 2),                 # negative lengths count as 0
    ([100, 7], [50, 60], 32, 0, 0, -30),            # a slot map shorter than the tokens
]


def run_plan(cached, new, page, spare, hold, extra, seed=0):
    n = len(cached)
    cc, nn = [max(c, 0) for c in cached], [max(m, 0) for m in new]
    width = max(1, max(-(-(c + m) // page) for c, m in zip(cc, nn)) + spare)
    g = torch.Generator().manual_seed(seed)
    ids = torch.randperm(n * width + 10, generator=g).to(torch.int32)
    table = torch.full((n, width), -7, dtype=torch.int32)
    at = 0
    for b, c in enumerate(cc):
        h = min(-(-c // page), width)
        table[b, :h] = ids[at:at + h]
        at += h
    need = sum(min(-(-(c + m) // page), width) - min(-(-c // page), width) for c, m in zip(cc, nn))
    free = ids[at:at + max(0, need - hold)]
    T = max(0, sum(nn) + extra)
    want = ref.plan(cached, new, free, table, page, T)
    t = table.cuda()
    got = misa.misa_plan_pages(i32(cached), i32(new), free.cuda(), t, page, T)
    torch.cuda.synchronize()
    assert t.tolist() == want["table"]
    assert got.q_start.tolist() == want["q_start"] and got.kv_lens.tolist() == want["kv_lens"]
    assert got.positions.tolist() == want["positions"] and got.slots.tolist() == want["slots"]
    assert got.n_taken.tolist() == want["n_taken"]


@pytest.mark.parametrize("case", PLANS, ids=range(len(PLANS)))
def test_plan_pages(case):
    say("plan", case)
    run_plan(*case)


@pytest.mark.parametrize("n,page,hi", [(255, 16, 40), (256, 64, 300), (257, 64, 5), (3001, 8, 30), (64, 128, 1)])
def test_plan_many_sequences(n, page, hi):
    say("plan", n, page, hi)
    g = torch.Generator().manual_seed(n)
    cached = torch.randint(0, 500, (n,), generator=g).tolist()
    new = torch.randint(0, hi + 1, (n,), generator=g).tolist()
    run_plan(cached, new, page, 1, 0, 37, seed=n)


def test_plan_slots_pass_32_bits():
    # page ids near 2^31 / page_keys x page_keys rows: slots past 2^31
    table = torch.full((1, 3), 2_000_000_000, dtype=torch.int32, device="cuda")
    got = misa.misa_plan_pages(i32([100]), i32([60]), i32([2_100_000_000]), table, 128, 60)
    torch.cuda.synchronize()
    assert got.slots.tolist() == [(2_000_000_000 if p < 128 else 2_100_000_000) * 128 + p % 128 for p in range(100, 160)]


# ---------------------------------------------------------------- rotary positions

ROPES = [   # tokens, heads, dim, rot, start, layout, dtype
    (1, 1, 128, 128, 0, "half", torch.bfloat16),
    (70, 64, 128, 64, 0, "half", torch.bfloat16),
    (33, 3, 192, 64, 128, "interleaved", torch.float32),
    (17, 5, 80, 20, 0, "half", torch.float16),          # a quarter of the head: the single-element path
    (9, 2, 80, 20, 60, "interleaved", torch.bfloat16),
    (300, 2, 64, 64, 0, "interleaved", torch.float16),
    (5, 7, 66, 2, 11, "half", torch.float32),           # one pair at an odd offset
    (2, 130, 256, 256, 0, "half", torch.float32),
    (1500, 1, 576, 64, 512, "interleaved", torch.bfloat16),
]


def rope_bound(x, y, start, rot, mscale):
    """One rounding to the output type; cos and sin good to 2^-22 (angle and function) and three fp32 roundings
    of terms no larger than mscale (|a| + |b|)."""
    half = torch.finfo(x.dtype).eps / 2
    big = 2 * x.double().abs().amax() * mscale
    return half * y.abs() + (2.0 ** -22 + 3 * ref.F32_HALF) * big + (2.0 ** -25 if x.dtype == torch.float16 else 0)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("case", ROPES, ids=range(len(ROPES)))
def test_rope(case, backward):
    T, H, D, rot, start, layout, dt = case
    say("rope", case, backward)
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, H, D), generator=g).to(dt)
    pos = torch.randint(0, 1 << 20, (T,), generator=g).to(torch.int32)
    f, m = misa.rope_inv_freq(rot, scaling="yarn", factor=8.0)
    y = misa.misa_rope(x.cuda(), pos.cuda(), f, layout=layout, rot_start=start, mscale=m, backward=backward)
    want = ref.rope(x, pos, f.cpu(), layout, start, m, backward)
    got = y.double().cpu()
    assert y.dtype == dt and float(((got - want).abs() - rope_bound(x, want, start, rot, m)).max()) <= 0
    keep = torch.ones(D, dtype=torch.bool)
    keep[start:start + rot] = False
    assert torch.equal(y.cpu()[..., keep], x[..., keep])
    z = x.cuda()   # in place
    r = misa.misa_rope(z, pos.cuda(), f, layout=layout, rot_start=start, mscale=m, backward=backward, out=z)
    assert r is z and torch.equal(z, y)


def test_rope_strided_and_ragged_ends():
    # q and k as slices of one projection [T, (8 + 2) * 128], written into a slice of another
    g = torch.Generator().manual_seed(3)
    T = 41
    qkv = torch.randn((T, 10, 128), generator=g).bfloat16().cuda()
    pos = torch.arange(T, dtype=torch.int32).cuda()
    f, m = misa.rope_inv_freq(128)
    dst = torch.full((T, 12, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    misa.misa_rope(qkv[:, 1:9], pos, f, out=dst[:, 2:10])
    assert torch.equal(dst[:, 2:10], misa.misa_rope(qkv[:, 1:9].contiguous(), pos, f))
    assert bool((dst[:, :2] == 5).all()) and bool((dst[:, 10:] == 5).all())
    # head-major storage, and an offset that is not 16-byte aligned
    hm = qkv.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(misa.misa_rope(hm, pos, f), misa.misa_rope(qkv, pos, f))
    odd = torch.randn((T, 3, 129), generator=g).bfloat16().cuda()[:, :, 1:]
    assert torch.equal(misa.misa_rope(odd, pos, f), misa.misa_rope(odd.contiguous(), pos, f))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_gradient_against_differences(layout):
    # the map is linear: a difference quotient of any step is exact but for rounding, so <g, d/dx rope(x) u> =
    # <rope_backward(g), u> for random u, g, to fp32 rounding of sums of 2 T H D products
    g0 = torch.Generator().manual_seed(9)
    T, H, D = 13, 3, 96
    x, u, g = (torch.randn((T, H, D), generator=g0).cuda() for _ in range(3))
    pos = torch.randint(0, 100000, (T,), generator=g0).to(torch.int32).cuda()
    f, m = misa.rope_inv_freq(32, scaling="yarn", factor=4.0)
    kw = dict(layout=layout, rot_start=16, mscale=m)
    h = 0.5
    diff = (misa.misa_rope(x + h * u, pos, f, **kw).double() - misa.misa_rope(x - h * u, pos, f, **kw).double()) / (2 * h)
    back = misa.misa_rope(g, pos, f, backward=True, **kw).double()
    lhs, rhs = float((g.double() * diff).sum()), float((back * u.double()).sum())
    scale = float((g.double().abs() * diff.abs()).sum())
    assert abs(lhs - rhs) <= 2.0 ** -20 * scale


# ---------------------------------------------------------------- page writes

WRITES = [   # tokens, heads, dim, page, fp8, values, rot, start, layout
    (1, 1, 128, 64, True, False, 64, 0, "half"),
    (200, 1, 128, 64, True, False, 64, 64, "interleaved"),
    (77, 8, 128, 16, False, True, 128, 0, "half"),
    (50, 3, 64, 10, True, True, 0, 0, "half"),
    (33, 2, 80, 7, True, True, 20, 3, "half"),
    (19, 5, 512, 4, False, False, 64, 448, "interleaved"),
]


@pytest.mark.parametrize("case", WRITES, ids=range(len(WRITES)))
def test_write_pages(case):
    T, H, D, page, fp8, values, rot, start, layout = case
    say("write", case)
    g = torch.Generator().manual_seed(T)
    n_pages = -(-T // page) + 2
    k, v = (torch.randn((T, H, D), generator=g).bfloat16() for _ in range(2))
    k[0] = 0   # a zero row: scale 1
    slots = torch.randperm(n_pages * page, generator=g)[:T]
    if T > 10:
        slots[3], slots[7] = -1, n_pages * page   # outside: skipped
    pos = torch.randint(0, 200000, (T,), generator=g).to(torch.int32)
    kind = torch.uint8 if fp8 else torch.bfloat16
    fill = 0x55 if fp8 else 3.0
    pools = [torch.full((n_pages, page, H, D), fill, dtype=kind, device="cuda") for _ in range(2)]
    scales = [torch.full((n_pages, page, H), -2.0, device="cuda") if fp8 else None for _ in range(2)]
    rope = {}
    if rot:
        f, m = misa.rope_inv_freq(rot, scaling="yarn", factor=2.0)
        rope = dict(positions=pos.cuda(), inv_freq=f, layout=layout, rot_start=start, mscale=m)
    misa.misa_write_pages(k.cuda(), slots.cuda(), pools[0], scales[0], v=v.cuda() if values else None,
                          v_pages=pools[1] if values else None, v_scale_pages=scales[1] if values else None, **rope)
    torch.cuda.synchronize()
    ok = (slots >= 0) & (slots < n_pages * page)
    for side, x in enumerate((k, v)):
        flat = pools[side].cpu().view(-1, H, D)
        untouched = torch.ones(n_pages * page, dtype=torch.bool)
        if side == 0 or values:
            untouched[slots[ok]] = False
        assert bool((flat[untouched].float() == fill).all())
        if side == 1 and not values:
            continue
        y = x.double()
        if side == 0 and rot:
            y = ref.rope(x, pos, f.cpu(), layout, start, m)
        y, got = y[ok], flat[slots[ok]]
        if not fp8:
            assert bool(((got.double() - y).abs() <= ref.BF16_HALF * y.abs() + 2.0 ** -40).all())
            continue
        sc = scales[side].cpu().view(-1, H)
        assert bool((sc[untouched] == -2.0).all())
        amax = y.abs().amax(-1)
        want = torch.where(amax > 0, amax / 448, 1.0)
        sc = sc[slots[ok]].double()
        # the scale: a rounding of the value and one of the quotient
        assert bool(((sc - want).abs() <= 2 * ref.F32_HALF * want * 1.01).all())
        # a code is the nearest to value / scale: half a step (2^-4 relative, 2^-10 below the normal range),
        # and two fp32 roundings that may carry a value over a border
        val = got.view(torch.float8_e4m3fn).double()
        r = y / sc[..., None]
        assert bool(((val - r).abs() <= 2.0 ** -4 * r.abs() * (1 + 2.0 ** -20) + 2.0 ** -10).all())


def test_write_pages_quantises_as_the_indexer_queries_do():
    g = torch.Generator().manual_seed(1)
    q = torch.randn((1, 50, 4, 128), generator=g).bfloat16().cuda()
    q8, qs = misa.misa_quantize_q(misa.make_shape(1, 50, 64, 0, 4, 16), q)
    pages = torch.zeros((13, 4, 4, 128), dtype=torch.uint8, device="cuda")
    sc = torch.zeros((13, 4, 4), device="cuda")
    misa.misa_write_pages(q[0], torch.arange(50, device="cuda"), pages, sc)
    assert torch.equal(pages.view(-1, 4, 128)[:50], q8[0]) and torch.equal(sc.view(-1, 4)[:50], qs[0])


# ---------------------------------------------------------------- attention

ATTN = {   # kv_lens, new, heads, kv_heads, dim, page, fp8
    "one_token": ([1], [1], 4, 1, 128, 64, False),
    "decode_small": ([5, 64, 65, 1, 0, 200], [1, 1, 1, 1, 1, 1], 8, 2, 128, 16, False),
    "decode_mha_d64": ([129, 700], [1, 1], 3, 3, 64, 64, False),
    "decode_group5_fp8": ([100, 1030, 31], [1, 1, 1], 20, 4, 64, 16, True),
    "decode_long": ([5003, 2111], [1, 1], 16, 2, 128, 64, False),
    "decode_long_fp8_mqa": ([4999], [1], 64, 1, 128, 128, True),
    "spec_tokens": ([300, 4, 77], [4, 4, 3], 8, 2, 128, 16, False),   # all of the second sequence is new
    "chunk": ([300], [130], 8, 2, 128, 64, False),
    "chunk_fp8_page1": ([150], [70], 4, 1, 128, 1, True),
    "chunk_page100_d64": ([517], [201], 6, 3, 64, 100, False),
    "whole_prompt": ([333], [333], 4, 4, 128, 48, False),
    "mixed": ([515, 1, 700, 40, 0, 260, 90], [130, 1, 1, 17, 0, 0, 90], 12, 4, 128, 16, False),
    "mixed_fp8": ([515, 1, 700, 40, 260], [130, 1, 5, 17, 257], 20, 4, 64, 16, True),
    "mqa_128_heads": ([210], [9], 128, 1, 64, 64, False),
    "group_33": ([140, 60], [3, 1], 66, 2, 128, 32, False),
    "longer_chunk": ([1400], [400], 4, 1, 128, 64, False),
}


def call(p, idx=None, **kw):
    d = p.gpu()
    if idx is None:
        return misa.misa_attention_paged(**d, want_lse=True, **kw)
    return misa.misa_attention_selected(**d, idx=idx.cuda(), want_lse=True, **kw)


@pytest.mark.parametrize("name", ATTN)
def test_attention_paged(name):
    lens, new, H, KH, D, page, fp8 = ATTN[name]
    say("attention", name)
    p = ref.Paged(len(name), lens, new, H, KH, D, page, fp8)
    out, lse = call(p)
    torch.cuda.synchronize()
    ref.check_attention(p, out, lse)
    # a true bound on the new tokens changes nothing, and neither does a second run
    again = call(p, max_new=max(new))
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


SELECTED = {   # kv_lens, new, heads, kv_heads, dim, page, fp8, topk, holes
    "decode": ([500, 90, 1, 0], [1, 1, 1, 1], 16, 2, 128, 64, False, 100, 0.0),
    "decode_mqa64_fp8": ([3000, 2500], [1, 1], 64, 1, 128, 64, True, 2048, 0.0),
    "chunk_holes": ([300], [50], 8, 1, 128, 16, False, 77, 0.3),
    "prompt_d64": ([130], [130], 12, 4, 64, 48, False, 64, 0.0),
    "prompt_fp8": ([70, 20], [70, 20], 5, 5, 64, 64, True, 33, 0.5),
    "group_128": ([900], [3], 128, 1, 128, 64, False, 513, 0.1),
    "one_pick": ([300], [20], 4, 4, 128, 64, False, 1, 0.0),
    "long_list": ([9000], [2], 8, 1, 128, 64, False, 8192, 0.0),
    "group_20": ([700], [9], 40, 2, 128, 32, True, 300, 0.0),
}


@pytest.mark.parametrize("name", SELECTED)
def test_attention_selected(name):
    lens, new, H, KH, D, page, fp8, topk, holes = SELECTED[name]
    say("selected", name)
    p = ref.Paged(len(name) + 50, lens, new, H, KH, D, page, fp8)
    idx = p.select(topk, holes)
    out, lse = call(p, idx)
    torch.cuda.synchronize()
    ref.check_attention(p, out, lse, idx)


def test_selected_entries_out_of_sight_are_absent():
    p = ref.Paged(5, [200, 40], [3, 2], 8, 2, 128, 16)
    idx = p.select(50)
    idx[0, :] = -1                      # a row that sees nothing
    idx[1, 5], idx[1, 6] = 10 ** 6, -9  # behind the end, negative
    idx[2, 0:4] = 7                     # the same token four times counts four times
    idx[4, 3] = 39                      # the last token: visible to token 4 (position 39)
    idx[3, 3] = 39                      # but not to token 3 (position 38)
    out, lse = call(p, idx)
    torch.cuda.synchronize()
    ref.check_attention(p, out, lse, idx)
    assert bool((out[0] == 0).all())


def test_selecting_the_whole_prefix_equals_attention():
    p = ref.Paged(6, [180, 60], [4, 1], 8, 2, 128, 16)
    idx = torch.full((5, 180), -1, dtype=torch.int32)
    for t in range(5):
        idx[t, :p.pos(t) + 1] = torch.arange(p.pos(t) + 1, dtype=torch.int32)
    a, b = call(p), call(p, idx)
    for o, l in (a, b):
        ref.check_attention(p, o, l)


def test_rows_behind_the_last_sequence_stay():
    for idx_k in (None, 20):
        p = ref.Paged(8, [100, 30], [7, 1], 8, 2, 64, 16, pad_rows=5)
        d = p.gpu()
        d["q"][p.tokens:] = float("nan")
        out = torch.full(d["q"].shape, 3.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full(out.shape[:2], 9.0, device="cuda")
        if idx_k is None:
            misa.misa_attention_paged(**d, out=out, lse=lse)
            ref.check_attention(p, out, lse)
        else:
            idx = p.select(idx_k)
            misa.misa_attention_selected(**d, idx=idx.cuda(), out=out, lse=lse)
            ref.check_attention(p, out, lse, idx)
        assert bool((out[p.tokens:] == 3).all()) and bool((lse[p.tokens:] == 9).all())


@pytest.mark.parametrize("scale", [0.01, -0.3, 3.0])
def test_scales_and_large_scores(scale):
    p = ref.Paged(11, [260], [40], 4, 2, 64, 16)
    p.q *= 8
    out, lse = misa.misa_attention_paged(**p.gpu(), scale=scale, want_lse=True)
    torch.cuda.synchronize()
    ref.check_attention(p, out, lse, scale=scale)


def test_strided_queries():
    p = ref.Paged(12, [150, 33], [20, 1], 8, 2, 128, 16)
    d = p.gpu()
    whole = torch.zeros((p.tokens, 12, 128), dtype=torch.bfloat16, device="cuda")
    whole[:, 3:11] = d["q"]
    base = misa.misa_attention_paged(**d)[0]
    d["q"] = whole[:, 3:11]
    assert torch.equal(misa.misa_attention_paged(**d)[0], base)
    d["q"] = whole[:, 3:11].transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(misa.misa_attention_paged(**d)[0], base)


def test_wide_table_and_another_stream():
    # a table far wider than the sequences, on a stream of the caller's
    p = ref.Paged(13, [150, 700], [1, 1], 8, 2, 128, 16, width=4000)
    d = p.gpu()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out, lse = misa.misa_attention_paged(**d, want_lse=True, stream=side)
    side.synchronize()
    ref.check_attention(p, out, lse)
    with torch.cuda.stream(side):
        out2, _ = misa.misa_attention_paged(**d)
    side.synchronize()
    assert torch.equal(out, out2)


# ---------------------------------------------------------------- together

def serving_step(s, fp8, step):
    """Plan, rotate, write, pick, attend: one step of a uniform batch; the state is in s."""
    n, m, page = s["n"], s["m"], s["page"]
    plan = misa.misa_plan_pages(s["cached"], s["new"], s["free"], s["table"], page, n * m, plan=s.get("plan"))
    f, ms = s["freq"]
    misa.misa_write_pages(s["ik"], plan.slots, s["ik_pages"], s["ik_scale"], positions=plan.positions, inv_freq=f,
                          mscale=ms)
    q = misa.misa_rope(s["q"], plan.positions, f, mscale=ms, out=s["q_rot"])
    iq = misa.misa_rope(s["iq"], plan.positions, f, mscale=ms, out=s["iq_rot"])
    misa.misa_write_pages(s["k"], plan.slots, s["k_pages"], s["k_scale"], v=s["v"], v_pages=s["v_pages"],
                          v_scale_pages=s["v_scale"], positions=plan.positions, inv_freq=f, mscale=ms)
    sh = misa.make_shape(n, m, s["total"], s["total"] - m, s["ih"], 64)
    idx, _ = misa.misa_indexer_paged(sh, iq.view(n, m, s["ih"], 128), s["w"], s["ik_pages"], s["table"], 4, s["topk"],
                                     misa.PooledCache(n, s["total"] // 64 + 1), scale_pages=s["ik_scale"],
                                     idx=s["idx"], ws=s["ws"])
    dense = misa.misa_attention_paged(q, s["k_pages"], s["v_pages"], s["table"], plan.q_start, plan.kv_lens,
                                      s["k_scale"], s["v_scale"], out=s["dense"])[0]
    picked = misa.misa_attention_selected(q, s["k_pages"], s["v_pages"], s["table"], plan.q_start, plan.kv_lens, idx,
                                          s["k_scale"], s["v_scale"], out=s["picked"])[0]
    return plan, idx, dense, picked


def serving_state(seed, n, m, total, fp8, topk, page=64):
    g = torch.Generator(device="cuda").manual_seed(seed)
    H, KH, D, ih = 8, 2, 128, 8
    width = -(-total // page)
    n_pages = n * width + 2
    ids = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    owned = -(-(total - m) // page)
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    table[:, :owned] = ids[:n * owned].view(n, owned)
    kind = torch.uint8 if fp8 else torch.bfloat16

    def pool(h):
        x = torch.randn((n_pages, page, h, D), generator=g, device="cuda")
        if not fp8:
            return x.bfloat16(), None
        sc = x.abs().amax(-1) / 448
        return (x / sc[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), sc

    def rand(h):
        return torch.randn((n * m, h, D), generator=g, device="cuda").bfloat16()
    s = dict(n=n, m=m, page=page, total=total, topk=topk, ih=ih, table=table, free=ids[n * owned:].contiguous(),
             cached=i32([total - m] * n), new=i32([m] * n), freq=misa.rope_inv_freq(64, scaling="yarn", factor=4.0),
             q=rand(H), k=rand(KH), v=rand(KH), ik=rand(1), iq=rand(ih), w=torch.rand((n, m, ih), generator=g, device="cuda"))
    s["k_pages"], s["k_scale"] = pool(KH)
    s["v_pages"], s["v_scale"] = pool(KH)
    ikp, iks = pool(1)
    s["ik_pages"], s["ik_scale"] = ikp[:, :, 0].contiguous(), None if iks is None else iks[:, :, 0].contiguous()
    for o in ("q", "iq"):
        s[o + "_rot"] = torch.empty_like(s[o])
    s["dense"], s["picked"] = torch.empty_like(s["q"]), torch.empty_like(s["q"])
    s["idx"] = torch.empty((n, m, topk), dtype=torch.int32, device="cuda")
    sh = misa.make_shape(n, m, total, total - m, ih, 64)
    s["ws"] = torch.empty(max(1, misa.misa_indexer_paged_workspace_bytes(sh, 1 if fp8 else 0, 4, topk)),
                          dtype=torch.uint8, device="cuda")
    return s


@pytest.mark.parametrize("fp8", [False, True])
def test_serving_step_together(fp8):
    """The step's outputs against fp64 over what the pages hold after the write."""
    say("serving step", fp8)
    n, m, total, topk = 3, 5, 333, 64
    s = serving_state(21, n, m, total, fp8, topk)
    plan, idx, dense, picked = serving_step(s, fp8, 0)
    torch.cuda.synchronize()
    p = ref.Paged(0, [total] * n, [m] * n, 8, 2, 128, 64, fp8, width=s["table"].shape[1])
    p.table, p.q = s["table"].cpu(), s["q_rot"].cpu()
    p.vals = []
    for k in ("k", "v"):
        x = s[k + "_pages"].cpu()
        p.vals.append(x.view(torch.float8_e4m3fn).double() * s[k + "_scale"].cpu().double()[..., None] if fp8 else x.double())
    for out, ix in ((dense, None), (picked, idx.view(n * m, topk).cpu())):
        r, _, tol, _ = ref.attention(p, ix)
        assert bool(((out.double().cpu() - r).abs() <= tol).all())
    assert bool((idx >= 0).all())


def test_serving_step_replays():
    """The whole step captured once and replayed with new inputs equals eager steps, the program's own work between."""
    say("serving step captured")
    mk = [serving_state(s, 3, 2, 700, True, 64) for s in (31, 32, 33)]
    s = serving_state(31, 3, 2, 700, True, 64)
    serving_step(s, True, 0)
    torch.cuda.synchronize()
    s["plan"] = misa.misa_plan_pages(s["cached"], s["new"], s["free"], s["table"], s["page"], s["n"] * s["m"])
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(g):
            serving_step(s, True, 0)
    torch.cuda.current_stream().wait_stream(side)
    keys = [k for k, v in s.items() if torch.is_tensor(v)]
    for rep in range(5):
        t = mk[rep % 3]
        for k in keys:
            if k not in ("ws", "dense", "picked", "idx", "q_rot", "iq_rot"):
                s[k].copy_(t[k])
        s["dense"].fill_(7)
        s["picked"].fill_(7)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        _, idx, dense, picked = serving_step(t, True, 0)
        torch.cuda.synchronize()
        assert torch.equal(s["idx"], idx) and torch.equal(s["dense"], dense) and torch.equal(s["picked"], picked), rep
