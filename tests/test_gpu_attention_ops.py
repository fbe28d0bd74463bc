"""Rotary positions, the 8-bit paged cache and attention over it on the GPU,
against the float64 forms of attention_ref (bounds derived there)."""
import math

import pytest
import torch

import attention_ref as ref
import nvfp4_block_scaled_20_b200 as nv
from gpu_helpers import DEV, require_gpu

pytestmark = pytest.mark.gpu

ERR_SHAPE = 2


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def starts_of(counts, first=0):
    s = [first]
    for n in counts:
        s.append(s[-1] + n)
    return s


def within(got, want, bound):
    d = (got.double() - want.to(got.device)).abs()
    bad = ~(d <= bound.to(got.device))
    assert not bad.any(), "worst excess %.3g at %s" % (
        (d - bound.to(got.device)).nan_to_num(nan=math.inf).max().item(), bad.nonzero()[0].tolist())


# ------------------------------------------------------------------- rope
ROPES = [  # tokens, heads of q and k, dim, sections, elements to the left of x in its storage
    (1, (24, 24), 128, (22, 21, 21), 0), (37, (3, 1), 128, (22, 21, 21), 0),
    (700, (16, 4), 128, (16, 24, 24), 0), (13, (5, 2), 64, (10, 0, 18), 0),
    (9, (2, 2), 64, (7, 5, 3), 2), (50, (1, 3), 96, (48,), 0), (3, (2, 1), 2, (1,), 0),
    (5, (70, 1), 512, (100, 100, 50, 6), 0), (21, (4, 4), 128, (20, 20, 20), 4),
    (6, (1, 1), 130, (65,), 0), (4, (2, 2), 64, (0, 0), 0)]


@pytest.mark.parametrize("tokens,heads,dim,sections,shift", ROPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("per_axis,inverse", [(True, False), (False, True)])
def test_rope(tokens, heads, dim, sections, shift, dtype, interleaved, per_axis, inverse):
    g = gen(1)
    hq, hk = heads
    flat = torch.randn(tokens * (hq + hk + 1) * dim + shift, generator=g, device=DEV).to(dtype)
    both = flat[shift:].view(tokens, hq + hk + 1, dim)
    xs = [both[:, :hq], both[:, hq:hq + hk]]
    pos = torch.randint(-300, 100000, (tokens, len(sections) + 1), generator=g, device=DEV,
                        dtype=torch.int32)
    before = flat.clone()
    outs = nv.rope(xs, pos, list(sections), theta=10000.0, interleaved=interleaved,
                   per_axis=per_axis, inverse=inverse)
    assert torch.equal(flat, before)
    for x, o in zip(xs, outs):
        want = ref.rope(x, pos, sections, 10000.0, interleaved, per_axis, inverse)
        within(o.cpu(), want, ref.rope_bound(x, sections, interleaved, want, dtype))
        rest = 2 * sum(sections)
        assert torch.equal(o[..., rest:], x[..., rest:])
    # in place
    nv.rope(xs, pos, list(sections), theta=10000.0, interleaved=interleaved, per_axis=per_axis,
            inverse=inverse, outs=xs)
    assert torch.equal(xs[0], outs[0]) and torch.equal(xs[1], outs[1])
    assert torch.equal(both[:, hq + hk:], before[shift:].view_as(both)[:, hq + hk:])


@pytest.mark.parametrize("interleaved", [True, False])
def test_rope_gradient(interleaved):
    """The inverse call is the gradient: against the formula (the transpose of
    the rotation) and against differences, which are exact for a linear map up
    to the rounding of the calls."""
    g = gen(2)
    kw = dict(theta=1e4, interleaved=interleaved)
    pos = torch.randint(0, 4000, (11, 3), generator=g, device=DEV, dtype=torch.int32)
    x, dy, v = (torch.randn(11, 4, 64, generator=g, device=DEV) for _ in range(3))
    dx = nv.rope([dy], pos, [12, 10, 10], inverse=True, **kw)[0].double()
    up = nv.rope([x + v], pos, [12, 10, 10], **kw)[0].double()
    down = nv.rope([x - v], pos, [12, 10, 10], **kw)[0].double()
    step = (((x + v).double() - (x - v).double()) * dx).sum()
    seen = ((up - down) * dy.double()).sum()
    # 4e-7 (|x0| + |x1|) per output, below 4e-6 per element of either side here
    assert abs(seen - step) <= 4e-6 * (dy.abs().sum() + 2 * v.abs().sum()).double()
    want = ref.rope(dy, pos, [12, 10, 10], 1e4, interleaved, True, True)
    within(dx.cpu(), want, ref.rope_bound(dy, [12, 10, 10], interleaved, want, torch.float32))


def test_rope_copies_what_is_not_turned_even_infinite():
    x = torch.full((2, 1, 16), math.inf, device=DEV)
    x[..., 12:] = torch.tensor([math.inf, math.nan, -0.0, 1e38], device=DEV)
    for inter in (True, False):
        o = nv.rope([x], i32([[1], [5]]), [6], interleaved=inter)[0]
        assert torch.equal(o[..., 12:].view(torch.int32), x[..., 12:].view(torch.int32))


# ------------------------------------------------------------------ cache
def new_cache(pages, heads, pt, d, seed=None):
    c = nv.kv8_cache(pages, heads, pt, d)
    if seed is not None:  # anything, NaN codes among it
        g = gen(seed)
        for t in (c.k_codes, c.v_codes):
            t.copy_(torch.randint(0, 256, t.shape, generator=g, device=DEV).to(torch.uint8))
        for t in (c.k_scales, c.v_scales):
            t.copy_(torch.exp2(torch.randint(-9, -3, t.shape, generator=g, device=DEV).float()))
    return c


def filled(pages, heads, pt, d, seed):
    """A cache of finite codes."""
    c = new_cache(pages, heads, pt, d, seed)
    for t in (c.k_codes, c.v_codes):
        t[(t & 0x7F) == 0x7F] = 0x33
    return c


def table_of(need, pages, seed, width=None):
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    width = width or max(need + [1])
    rows = []
    for n in need:
        rows.append([order.pop() for _ in range(n)] + [-1] * (width - n))
    return rows


def same_cache(c, k_codes, k_scales, v_codes, v_scales):
    for got, want in ((c.k_codes, k_codes), (c.v_codes, v_codes)):
        a, b = ref.values(got).cpu(), want
        assert torch.equal(a.isnan(), b.isnan())
        bad = (a.nan_to_num(7.0) != b.nan_to_num(7.0)).nonzero()
        assert bad.numel() == 0, (bad.shape, bad[0].tolist())
    assert torch.equal(c.k_scales.double().cpu(), k_scales)
    assert torch.equal(c.v_scales.double().cpu(), v_scales)


def mirror(c):
    return [ref.values(c.k_codes).cpu(), c.k_scales.double().cpu(), ref.values(c.v_codes).cpu(),
            c.v_scales.double().cpu()]


WRITES = [  # tokens before, rows
    ([0], [1]), ([0], [64]), ([63], [1]), ([64], [1]), ([5], [200]), ([31, 0, 100, 7], [1, 33, 0, 400]),
    ([130, 2], [3, 0]), ([17] * 9, [1] * 9)]


@pytest.mark.parametrize("before,new", WRITES)
@pytest.mark.parametrize("pt,d", [(32, 64), (64, 64), (128, 64), (32, 128), (64, 128), (128, 128)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_write_and_read(before, new, pt, d, dtype):
    heads = 3
    need = [-(-(a + n) // pt) for a, n in zip(before, new)]
    c = new_cache(sum(need) + 2, heads, pt, d, 3)
    table = table_of(need, sum(need) + 2, 4)
    starts = starts_of(new)
    g = gen(5)
    # two rows that belong to no sequence; k and v side by side; sizes over many powers of two
    x = torch.randn((starts[-1] + 2, 2 * heads, d), generator=g, device=DEV)
    x *= torch.exp2(torch.randint(-12, 6, x.shape[:2], generator=g, device=DEV).float())[..., None]
    x = x.to(dtype)
    k, v = x[:, :heads], x[:, heads:]
    want = mirror(c)
    ref.write(want[0], want[1], k, table, before, starts)
    ref.write(want[2], want[3], v, table, before, starts)
    ws = nv.workspace(0)
    args = (i32(table), i32(before), i32(starts))
    nv.kv8_write(c, k, v, *args, ws=ws, max_new=max(new))
    assert nv.device_error(ws) == 0
    same_cache(c, *want)
    # the same call again changes nothing
    nv.kv8_write(c, k, v, *args, ws=ws)
    same_cache(c, *want)
    # and back
    outs = [torch.full((starts[-1] + 2, heads, d), 7.0, dtype=dtype, device=DEV) for _ in "kv"]
    nv.kv8_read(c, *args, starts[-1] + 2, outs=outs, ws=ws, max_tokens=max(new))
    assert nv.device_error(ws) == 0
    for o, codes, scales in ((outs[0], c.k_codes, c.k_scales), (outs[1], c.v_codes, c.v_scales)):
        for s, n in enumerate(new):
            all_tokens = ref.tokens(codes, scales, i32(table[s]), before[s] + n)
            assert torch.equal(o[starts[s]:starts[s + 1]].double(), all_tokens[before[s]:])
        assert (o[starts[-1]:] == 7.0).all()


def test_write_values_that_are_not_ordinary():
    """Zero blocks, infinities, NaN, tiny and huge values, one type's extremes."""
    pt, d = 32, 64
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.zeros((pt * 8, 1, d), device=DEV)
        x[pt:2 * pt] = 1e-30
        x[2 * pt:3 * pt] = torch.finfo(dtype).max
        x[3 * pt, 0, :3] = torch.tensor([math.inf, -math.inf, math.nan])
        x[3 * pt, 0, 3] = 0.4
        x[4 * pt:5 * pt, 0, 0] = math.nan
        x[5 * pt:6 * pt, 0, :2] = torch.tensor([448.0, -449.0])
        x[6 * pt:7 * pt, 0, :3] = torch.tensor([1.75 * 2.0 ** -40 * 2 ** 8, 1e-12, -0.0])
        x[7 * pt:, 0] = torch.linspace(-500, 500, d)
        x = x.to(dtype)
        c = nv.kv8_cache(8, 1, pt, d)
        want = mirror(c)
        table = [list(range(8))]
        ref.write(want[0], want[1], x, table, [0], [0, pt * 8])
        ref.write(want[2], want[3], -x, table, [0], [0, pt * 8])
        nv.kv8_write(c, x, -x, i32(table), i32([0]), i32([0, pt * 8]))
        same_cache(c, *want)
        assert c.k_scales[0, 0] == 2.0 ** -40 and c.k_scales[2, 0] == 2.0 ** 40


def test_write_token_by_token_equals_the_running_maximum():
    """A page filled one token at a time: scales never shrink, and each code is
    off by at most half a step of a code at the page's last scale, once for each
    time the scale grew into its subnormal range."""
    pt, d, heads = 64, 128, 2
    g = gen(9)
    x = torch.randn((pt, heads, d), generator=g, device=DEV)
    x *= torch.exp2(torch.arange(pt, device=DEV).float() / 8)[:, None, None]
    x = x.bfloat16()
    c = nv.kv8_cache(3, heads, pt, d)
    want = mirror(c)
    ws = nv.workspace(0)
    for t in range(pt):
        ref.write(want[0], want[1], x[t:t + 1], [[1]], [t], [0, 1])
        ref.write(want[2], want[3], x[t:t + 1], [[1]], [t], [0, 1])
        nv.kv8_write(c, x[t:t + 1], x[t:t + 1], i32([[1]]), i32([t]), i32([0, 1]), ws=ws)
    same_cache(c, *want)
    k, _ = nv.kv8_read(c, i32([[1]]), i32([0]), i32([0, pt]), pt, out_dtype=torch.float32, ws=ws)
    grown = torch.log2(c.k_scales[1] / 2.0 ** -12).clamp(min=1)[None, :, None]
    step = x.double().abs() * 2.0 ** -4 + c.k_scales[1].double()[None, :, None] * 2.0 ** -10 * grown
    within(k, x.double(), step)


def bad_batches(pages):
    good = dict(table=[[0, 1], [2, 3]], lens=[10, 20], starts=[0, 4, 9])
    yield dict(good, table=[[0, 1], [-1, 3]]), [0]
    yield dict(good, table=[[pages, 1], [2, 3]]), [1]
    yield dict(good, lens=[-1, 20]), [1]
    yield dict(good, lens=[10, 2000]), [0]
    yield dict(good, starts=[4, 0, 5]), [1]
    yield dict(good, starts=[0, 4, 900]), [0]
    yield dict(good, starts=[-3, 0, 5]), [1]
    yield dict(good, starts=[0, 4, 20]), [0]  # more rows than max_rows


@pytest.mark.parametrize("case", range(8))
def test_bad_device_values_are_reported_and_skipped(case):
    """Sequences that do not fit are skipped with the error word set; the others
    are done as without them."""
    pages, heads, pt, d = 4, 2, 32, 64
    bad, fine = list(bad_batches(pages))[case]
    g = gen(11)
    x = torch.randn((20, heads, d), generator=g, device=DEV)
    for call in ("write", "read", "attend"):
        c = filled(pages, heads, pt, d, 12)
        want = mirror(c)
        ws = nv.workspace(0)
        args = (i32(bad["table"]), i32(bad["lens"]), i32(bad["starts"]))
        if call == "write":
            nv.kv8_write(c, x, -x, *args, max_new=6, ws=ws)
            for s in fine:
                a, b = bad["starts"][s], bad["starts"][s + 1]
                for w, y in ((want[:2], x), (want[2:], -x)):
                    ref.write(w[0], w[1], y[a:b], [bad["table"][s]], [bad["lens"][s]], [0, b - a])
            same_cache(c, *want)
        elif call == "read":
            outs = [torch.full((20, heads, d), 5.0, device=DEV) for _ in "kv"]
            nv.kv8_read(c, *args, 20, outs=outs, max_tokens=6, ws=ws)
            left = torch.ones(20, dtype=torch.bool)
            for s in fine:
                a, b, n = bad["starts"][s], bad["starts"][s + 1], bad["lens"][s]
                t = ref.tokens(c.k_codes, c.k_scales, i32(bad["table"][s]), n + b - a)[n:]
                assert torch.equal(outs[0][a:b].double(), t)
                left[a:b] = False
            assert (outs[0][left] == 5.0).all() and (outs[1][left] == 5.0).all()
        else:
            q = torch.randn((20, heads, d), generator=g, device=DEV).bfloat16()
            ws = nv.kv8_attention_workspace(c, args[0], args[2], heads, 6)
            out = torch.full_like(q, 5.0)
            nv.kv8_attention(q, c, *args, max_q=6, out=out, ws=ws)
            for s in fine:
                a, b = bad["starts"][s], bad["starts"][s + 1]
                check_sequence(out[a:b], None, q[a:b], c, i32(bad["table"][s]), bad["lens"][s])
        assert nv.device_error(ws) == ERR_SHAPE, call
        assert nv.device_error(ws) == 0


# -------------------------------------------------------------- attention
def check_sequence(out, lse, q, c, table_row, n, causal=False, window=-1, sink=0, scale=None):
    d = q.shape[2]
    k = ref.tokens(c.k_codes, c.k_scales, table_row, n)
    v = ref.tokens(c.v_codes, c.v_scales, table_row, n)
    ok = ref.seen(q.shape[0], n, causal, window, sink, q.device)
    any_sees = ok.any(0)
    k, v = k[:], v[:]
    k[~any_sees], v[~any_sees] = 0.0, 0.0
    pt = c.page_tokens
    pages = table_row.long()[torch.arange(max(n, 1), device=q.device) // pt]
    vs = c.v_scales[pages].double()
    codes = (v / vs[:n, :, None]).abs() if n else v
    want, wl, eo, el = ref.attention(q.double(), k, v, codes, vs, scale or d ** -0.5, ok)
    within(out, want, eo)
    if lse is not None:
        seen = ~torch.isinf(wl)
        assert torch.equal(torch.isinf(lse), ~seen)
        within(lse[seen], wl[seen], el[seen])


ATTENDS = [  # queries and cached tokens of each sequence
    ([1], [1]), ([1], [0]), ([1], [64]), ([1, 1, 1], [65, 2000, 31]), ([5, 1, 0, 3], [300, 1, 50, 3]),
    ([3], [1]), ([17], [17]), ([130, 7], [700, 129]), ([300], [1000])]
MASKS = [dict(causal=True), dict(causal=False), dict(causal=True, window=40, sink=5),
         dict(causal=False, window=100, sink=70), dict(causal=True, window=0)]


def attend_case(nq, lens, hq, hk, d, pt, mask, seed=20, lse=True, scale=None):
    need = [-(-n // pt) for n in lens]
    pages = sum(need) + 2
    c = filled(pages, hk, pt, d, seed)
    table = table_of(need, pages, seed + 1)
    # codes past the sequences' ends may be anything
    for s, n in enumerate(lens):
        if n % pt:
            c.k_codes[table[s][n // pt], :, n % pt:] = 0x7F
            c.v_codes[table[s][n // pt], :, n % pt:] = 0xFF
    starts = starts_of(nq)
    g = gen(seed + 2)
    q = (torch.randn((starts[-1] + 3, hq, d), generator=g, device=DEV) * 0.1).bfloat16()
    out = torch.full_like(q, 9.0)
    ls = torch.full((starts[-1] + 3, hq), 9.0, device=DEV) if lse else None
    t = i32(table)
    ws = nv.kv8_attention_workspace(c, t, i32(starts), hq, max(nq))
    nv.kv8_attention(q, c, t, i32(lens), i32(starts), max_q=max(nq), out=out, lse=ls, ws=ws,
                     scale=scale, **mask)
    assert nv.device_error(ws) == 0
    for s, n in enumerate(lens):
        a, b = starts[s], starts[s + 1]
        check_sequence(out[a:b], ls[a:b] if lse else None, q[a:b], c, t[s], n, scale=scale, **mask)
    assert (out[starts[-1]:] == 9.0).all()
    assert not lse or (ls[starts[-1]:] == 9.0).all()
    return c, q, t, i32(lens), i32(starts), ws, out, ls


@pytest.mark.parametrize("nq,lens", ATTENDS)
@pytest.mark.parametrize("pt,d", [(32, 64), (64, 64), (128, 64), (32, 128), (64, 128), (128, 128)])
@pytest.mark.parametrize("mask", range(len(MASKS)))
def test_attention(nq, lens, pt, d, mask):
    attend_case(nq, lens, 6, 2, d, pt, MASKS[mask])


@pytest.mark.parametrize("hq,hk", [(1, 1), (8, 8), (24, 1), (40, 2), (12, 4)])
def test_attention_heads(hq, hk):
    for nq, lens in (([1, 1], [100, 500]), ([9, 2], [200, 77]), ([150], [400])):
        attend_case(nq, lens, hq, hk, 128, 64, MASKS[0], seed=hq)
        attend_case(nq, lens, hq, hk, 64, 32, MASKS[1], seed=hq, lse=False, scale=0.37)


@pytest.mark.parametrize("nq", [1, 40, 600])
def test_attention_sharp_and_far_scores(nq):
    """Scores that span hundreds and rise along the keys, so that the running
    maximum keeps moving; V scales that differ by 2^30 between pages."""
    pt, d, hk, n = 64, 128, 2, 900
    c = filled(16, hk, pt, d, 31)
    c.v_scales.copy_(torch.exp2(torch.randint(-20, 11, c.v_scales.shape, generator=gen(32),
                                              device=DEV).float()))
    c.k_scales.fill_(2.0 ** -5)
    c.k_codes[..., 0] = 0x38  # 1.0
    t = torch.arange(15, device=DEV, dtype=torch.int32)[None].contiguous()
    for p in range(15):
        c.k_scales[p] = 2.0 ** (p // 2 - 5)
    g = gen(33)
    q = (torch.randn((nq, 2 * hk, d), generator=g, device=DEV)).bfloat16()
    q[:, 0] *= 1e-20
    q[:, 1, 0] = 300.0
    out = nv.kv8_attention(q, c, t, i32([n]), i32([0, nq]), causal=True)
    lse = torch.empty((nq, 2 * hk), device=DEV)
    again = nv.kv8_attention(q, c, t, i32([n]), i32([0, nq]), causal=True, lse=lse)
    assert torch.equal(out, again)
    check_sequence(out, lse, q, c, t[0], n, causal=True)


@pytest.mark.parametrize("pt,d", [(32, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("nq", [1, 9, 300])
def test_attention_single_keys_that_rise(pt, d, nq):
    """One key in 128 outweighs all before it by 2^20 and more, at places all over
    the steps, so that maxima jump in every part of a step; every query sees
    another number of them."""
    n = 1900
    c = filled(-(-n // pt) + 1, 1, pt, d, 35)
    c.k_codes.zero_()
    c.k_scales.fill_(1.0)
    t = torch.arange(-(-n // pt), device=DEV, dtype=torch.int32)[None].contiguous()
    codes = c.k_codes.view(torch.float8_e4m3fn)
    for s, at in enumerate((5, 40, 70, 95, 96, 101, 127, 120, 3, 99, 64, 111, 30, 126, 97)):
        key = 128 * s + at
        if key < n:
            codes[key // pt, 0, key % pt, 0] = float(16 * (s + 1))
    q = torch.zeros((nq, 2, d), device=DEV, dtype=torch.bfloat16)
    q[:, 0, 0] = 1.0
    q[:, 1, 0] = torch.linspace(-1, 3, nq, device=DEV).bfloat16()
    for mask in (dict(causal=False), dict(causal=True, window=500)):
        lse = torch.empty((nq, 2), device=DEV)
        out = nv.kv8_attention(q, c, t, i32([n]), i32([0, nq]), scale=1.0, lse=lse, **mask)
        check_sequence(out, lse, q, c, t[0], n, scale=1.0, **mask)


@pytest.mark.parametrize("nq", [3, 200])
def test_attention_nan_keys_reach_the_queries_that_see_them(nq):
    c = filled(8, 1, 64, 128, 36)
    t = torch.arange(8, device=DEV, dtype=torch.int32)[None].contiguous()
    n, at = 500, 500 - nq // 2
    q = torch.randn((nq, 1, 128), generator=gen(37), device=DEV).bfloat16()
    args = (t, i32([n]), i32([0, nq]))
    clean = nv.kv8_attention(q, c, *args, causal=True)
    c.k_codes[at // 64, 0, at % 64, 17] = 0x7F
    out = nv.kv8_attention(q, c, *args, causal=True)
    first = at - (n - nq)  # the first query that sees the key
    assert out[first:].isnan().all()
    assert torch.equal(out[:first], clean[:first])


def test_attention_long_cache_many_rows():
    """More steps than any ring holds, split and whole tiles in one call."""
    attend_case([700, 130], [4100, 3000], 16, 8, 128, 64, MASKS[1], seed=81)
    attend_case([520], [5000], 12, 12, 64, 32, MASKS[2], seed=82)
    attend_case([1500, 900, 1], [2000, 1024, 128], 8, 8, 128, 128, MASKS[0], seed=83)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,lens,hk", [
    ([1, 2], [9000, 130], 2),                       # many even shares
    ([2, 0, 1], [700, 65, 3], 2),                   # few of them
    ([1] * 40, [4200] + list(range(60, 99)), 8)])   # runs of fixed length
@pytest.mark.parametrize("mask", [0, 2])
def test_attention_few_rows_however_they_are_split(nq, lens, hk, d, mask):
    """Also where the page table is far wider than the sequences, with entries
    past them that name no page."""
    c, q, t, ln, starts, ws, out, ls = attend_case(nq, lens, 2 * hk, hk, d, 64, MASKS[mask], seed=91)
    wide = torch.full((t.shape[0], 420), c.k_codes.shape[0], dtype=torch.int32, device=DEV)
    wide[:, :t.shape[1]] = t
    w2 = nv.kv8_attention_workspace(c, wide, starts, 2 * hk, max(nq))
    other, l2 = torch.full_like(out, 9.0), torch.full_like(ls, 9.0)
    for _ in range(2):  # the same workspace twice
        nv.kv8_attention(q, c, wide, ln, starts, max_q=max(nq), out=other, lse=l2, ws=w2, **MASKS[mask])
        assert nv.device_error(w2) == 0
        for s, n in enumerate(lens):
            a, b = sum(nq[:s]), sum(nq[:s + 1])
            check_sequence(other[a:b], l2[a:b], q[a:b], c, t[s], n, **MASKS[mask])
        assert (other[sum(nq):] == 9.0).all() and (l2[sum(nq):] == 9.0).all()


def test_attention_nan_and_infinite_queries_stay_in_their_rows():
    c = filled(4, 1, 64, 64, 41)
    q = torch.randn((4, 2, 64), generator=gen(42), device=DEV).bfloat16()
    q[1, 0, 3] = math.nan
    q[2, 1, 5] = math.inf
    t = i32([[0, 1, 2]])
    out = nv.kv8_attention(q, c, t, i32([150]), i32([0, 4]))
    assert out[1, 0].isnan().all() and out[2, 1].isnan().all()
    keep = torch.ones((4, 2), dtype=torch.bool, device=DEV)
    keep[1, 0] = keep[2, 1] = False
    q2 = torch.where(keep[..., None], q, torch.zeros_like(q))
    assert torch.equal(out[keep], nv.kv8_attention(q2, c, t, i32([150]), i32([0, 4]))[keep])


def test_attention_hidden_tokens_may_hold_nan():
    """Tokens outside the window of every query, or behind the cache's end."""
    for nq, hq in ((1, 4), (5, 24), (200, 4)):
        c = filled(12, 4, 64, 128, 43)
        t = torch.arange(12, device=DEV, dtype=torch.int32)[None].contiguous()
        q = torch.randn((nq, hq, 128), generator=gen(44), device=DEV).bfloat16()
        kw = dict(causal=True, window=100, sink=10)
        args = (i32([700]), i32([0, nq]))
        a = nv.kv8_attention(q, c, t, *args, **kw)
        lo = 700 - nq - 100
        for pos in list(range(10, lo)) + list(range(700, 768)):
            c.k_codes[pos // 64, :, pos % 64] = 0x7F
            c.v_codes[pos // 64, :, pos % 64] = 0x7F
        assert torch.equal(a, nv.kv8_attention(q, c, t, *args, **kw))


def test_attention_strided_and_on_another_stream():
    c = filled(9, 2, 64, 128, 51)
    t, lens, starts = i32([[3, 1, 8], [0, 2, 5]]), i32([150, 90]), i32([0, 40, 43])
    qkv = torch.randn((43, 4 + 4, 128), generator=gen(52), device=DEV).bfloat16()
    q = qkv[:, :4]
    plain = nv.kv8_attention(q.contiguous(), c, t, lens, starts, causal=True)
    out = torch.full((43, 12, 128), 3.0, device=DEV).bfloat16()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    nv.kv8_attention(q, c, t, lens, starts, causal=True, out=out[:, 4:8], stream=side)
    side.synchronize()
    assert torch.equal(out[:, 4:8], plain)
    assert (out[:, :4] == 3.0).all() and (out[:, 8:] == 3.0).all()


@pytest.mark.parametrize("nq", [1, 40])
def test_attention_shared_pages_two_streams_and_replays(nq):
    """Sequences that share prefix pages, one of them the same page twice; two
    calls at once on their own workspaces; a captured call replayed with other
    lengths, some of them zero."""
    hk, hq, d, pt = 2, 6, 128, 64
    c = filled(12, hk, pt, d, 101)
    t = i32([[3, 1, 4, 0, 5, 9, 2, 6], [3, 1, 4, 8, 7, 7, 7, 10], [3, 1, 11, 11, 0, 0, 0, 0]])
    starts = i32([0, nq, 2 * nq, 3 * nq])
    q = (torch.randn((3 * nq, hq, d), generator=gen(102), device=DEV) * 0.1).bfloat16()

    def check(out, lens):
        for s, n in enumerate(lens):
            check_sequence(out[s * nq:(s + 1) * nq], None, q[s * nq:(s + 1) * nq], c, t[s], n, causal=True)

    first, second = [512, 500, 190], [70, 0, 256]
    want = []
    for lens in (first, second):
        want.append(nv.kv8_attention(q, c, t, i32(lens), starts, max_q=nq, causal=True))
        check(want[-1], lens)
    # two at once, each on its stream
    streams = [torch.cuda.Stream() for _ in "ab"]
    ws = [nv.kv8_attention_workspace(c, t, starts, hq, nq) for _ in "ab"]
    lens = [i32(first), i32(second)]
    outs = [[torch.empty_like(q) for _ in range(20)] for _ in "ab"]
    torch.cuda.synchronize()
    for k in range(20):
        for i in range(2):
            nv.kv8_attention(q, c, t, lens[i], starts, max_q=nq, causal=True, out=outs[i][k],
                             ws=ws[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])
    # captured once
    n, out = i32(first), torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.kv8_attention(q, c, t, n, starts, max_q=nq, causal=True, out=out, ws=ws[0])
    for i in (1, 0, 1):
        n.copy_(lens[i])
        graph.replay()
        assert torch.equal(out, want[i])
    assert nv.device_error(ws[0]) == 0 and nv.device_error(ws[1]) == 0


def test_offsets_past_32_bits():
    """Pages whose bytes lie past 2^32 of a long cache."""
    heads, pt, d = 16, 128, 128
    pages = (1 << 32) // (heads * pt * d) + 8
    codes = [torch.empty((pages, heads, pt, d), dtype=torch.uint8, device=DEV) for _ in "kv"]
    scales = [torch.ones((pages, heads), device=DEV) for _ in "kv"]
    c = nv.KV8Cache(codes[0], codes[1], scales[0], scales[1])
    t = i32([[pages - 2, 3, pages - 1]])
    x = torch.randn((300, heads, d), generator=gen(61), device=DEV).bfloat16()
    nv.kv8_write(c, x, x.flip(0), t, i32([0]), i32([0, 300]))
    k, v = nv.kv8_read(c, t, i32([0]), i32([0, 300]), 300, out_dtype=torch.float32)
    sub = nv.KV8Cache(*[a[[pages - 2, 3, pages - 1]].contiguous() for a in (*codes, *scales)])
    small = i32([[0, 1, 2]])
    k2, v2 = nv.kv8_read(sub, small, i32([0]), i32([0, 300]), 300, out_dtype=torch.float32)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    within(k, x.double(), x.double().abs() * 2.0 ** -4 + 2.0 ** -16)
    for nq in (1, 200):
        q = x[:nq]
        a = nv.kv8_attention(q, c, t, i32([300]), i32([0, nq]), causal=True)
        b = nv.kv8_attention(q, sub, small, i32([300]), i32([0, nq]), causal=True)
        assert torch.equal(a, b)
    check_sequence(a, None, q, sub, small[0], 300, causal=True)


def test_run_together_and_in_a_graph():
    """Rotary positions, a cache write and attention as a generation loop makes
    them, by chunks, eagerly and from a captured graph replayed on new inputs."""
    h, hk, d, pt, chunk = 8, 4, 128, 64, 90
    g = gen(71)
    t = i32([[5, 2, 7, 0, 1, 6, 3, 4]])
    ws = [nv.workspace(0)]
    starts = i32([0, chunk])

    def fresh():
        return nv.kv8_cache(8, hk, pt, d)

    def step(c, qkv, pos, before, after, ws_a):
        q, k = nv.rope([qkv[:, :h], qkv[:, h:h + hk]], pos, [22, 21, 21])
        nv.kv8_write(c, k, qkv[:, h + hk:], t, before, starts, ws=ws[0], max_new=chunk)
        return nv.kv8_attention(q, c, t, after, starts, max_q=chunk, causal=True, window=200,
                                sink=16, ws=ws_a), q

    inputs = [(torch.randn((chunk, h + 2 * hk, d), generator=g, device=DEV).bfloat16(),
               torch.randint(0, 50, (chunk, 3), generator=g, device=DEV, dtype=torch.int32))
              for _ in range(5)]
    c = fresh()
    ws_a = nv.kv8_attention_workspace(c, t, starts, h, chunk)
    eager = []
    for i, (x, pos) in enumerate(inputs):
        out, q = step(c, x, pos, i32([i * chunk]), i32([(i + 1) * chunk]), ws_a)
        check_sequence(out, None, q, c, t[0], (i + 1) * chunk, causal=True, window=200, sink=16)
        eager.append(out)
    kept = [x.clone() for x in (c.k_codes, c.v_codes, c.k_scales, c.v_scales)]
    # the same loop from one graph
    c = fresh()
    x, pos = torch.empty_like(inputs[0][0]), torch.empty_like(inputs[0][1])
    before, after = i32([0]), i32([chunk])
    x.copy_(inputs[0][0])
    pos.copy_(inputs[0][1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(fresh(), x, pos, before, after, ws_a)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = step(c, x, pos, before, after, ws_a)
    for i, (xi, pi) in enumerate(inputs):
        x.copy_(xi)
        pos.copy_(pi)
        before.fill_(i * chunk)
        after.fill_((i + 1) * chunk)
        graph.replay()
        assert torch.equal(out, eager[i]), i
    for a, b in zip((c.k_codes, c.v_codes, c.k_scales, c.v_scales), kept):
        assert torch.equal(a, b)
    assert nv.device_error(ws[0]) == 0 and nv.device_error(ws_a) == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,n", [(200, 0), (130, 0), (600, 60)])
def test_attention_rows_that_see_nothing_are_zero(nq, n, d):
    """Tiles without a single step, of an empty sequence and, causal, before the
    cache's first token: zeros and -infinity, whenever q arrives from memory."""
    heads = 24
    c = filled(4, heads, 64, d, 111)
    t = i32([[2, 1]] * 4)
    starts = i32([i * nq for i in range(5)])
    q = torch.randn((4 * nq, heads, d), generator=gen(112), device=DEV).bfloat16()
    out, lse = torch.empty_like(q), torch.empty((4 * nq, heads), device=DEV)
    ws = nv.kv8_attention_workspace(c, t, starts, heads, nq)
    flush = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    blind = torch.arange(4 * nq, device=DEV) % nq < nq - n  # at < 0
    for k in range(40):
        flush.fill_(k)
        out.fill_(9.0)
        lse.fill_(9.0)
        nv.kv8_attention(q, c, t, i32([n] * 4), starts, max_q=nq, causal=True, out=out, lse=lse, ws=ws)
        assert not out[blind].any()
        assert (lse[blind] == -math.inf).all() and torch.isfinite(lse[~blind]).all()
    for s in range(4 if n else 0):
        rows = slice(s * nq, (s + 1) * nq)
        check_sequence(out[rows], lse[rows], q[rows], c, t[s], n, causal=True)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 30, 2 ** 31 - 5])
@pytest.mark.parametrize("nq,n", [(3, 1), (5, 3), (700, 60), (90, 500)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_window_without_a_limit(window, nq, n, causal):
    """The widest windows, with queries before the cache's first token: as if
    there were none (causal, the last queries see what they see; else all)."""
    for d, heads in ((128, 2), (64, 1)):
        c, q, t, lens, starts, ws, out, lse = attend_case(
            [nq, 1], [n, 40], heads, heads, d, 64, dict(causal=causal, window=window, sink=2), seed=121)
        plain = nv.kv8_attention(q, c, t, lens, starts, max_q=nq, causal=causal, ws=ws)
        assert torch.equal(out[:nq + 1], plain[:nq + 1])


@pytest.mark.parametrize("call", ["token", "chunk", "read", "rope", "write"])
def test_what_a_call_allocates_belongs_to_its_stream(call):
    """A call on a stream of its own, without workspace and outputs, while either
    stream is behind the other: memory that the call takes or gives back is not
    used by the other stream's work meanwhile."""
    heads, d, n = 2, 128, 4000
    c = filled(64, heads, 64, d, 131)
    t = torch.arange(63, device=DEV, dtype=torch.int32)[None].contiguous()
    nq = dict(token=1, chunk=700).get(call, 500)
    x = torch.randn((nq, heads, d), generator=gen(132), device=DEV).bfloat16()
    lens, starts, zero, minus = i32([n]), i32([0, nq]), i32([0]), -x
    pos = torch.arange(nq, device=DEV, dtype=torch.int32)[:, None].contiguous()

    def go(stream=None):
        if call == "read":
            return nv.kv8_read(c, t, zero, starts, nq, stream=stream)[0]
        if call == "rope":
            return nv.rope([x], pos, [64], stream=stream)[0]
        if call == "write":
            nv.kv8_write(c, x, minus, t, zero, starts, stream=stream)
            return c.v_codes
        return nv.kv8_attention(x, c, t, lens, starts, stream=stream)

    want = go().clone()
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    size = max(want.numel() * want.element_size(),
               nv.kv8_attention_workspace(c, t, starts, heads, nq).numel())
    torch.cuda.synchronize()
    for _ in range(3):
        # the call's kernels come late: what this stream allocates now is not theirs
        with torch.cuda.stream(side):
            torch.cuda._sleep(30_000_000)
        got = go(side)
        mine = [torch.full((s,), 7, dtype=torch.uint8, device=DEV) for s in (size, size, 256, 512)]
        here.synchronize()
        side.synchronize()
        assert torch.equal(got, want)
        assert all((m == 7).all() for m in mine)
        # they come early: what this stream has yet to read is not overwritten
        mine = [torch.full((s,), 3, dtype=torch.uint8, device=DEV) for s in (size, size, 256, 512)]
        torch.cuda.synchronize()
        torch.cuda._sleep(30_000_000)
        sums = [m.clone() for m in mine]
        del mine
        got = go(side)
        side.synchronize()
        with torch.cuda.stream(side):
            assert torch.equal(got, want)
        here.synchronize()
        assert all((m == 3).all() for m in sums)


@pytest.mark.parametrize("nq,n,hq,hk,d,pt", [
    (1, 300, 4, 4, 128, 64), (5, 40, 6, 2, 64, 32), (7, 900, 8, 4, 128, 128), (4, 20000, 8, 2, 64, 64),
    (200, 700, 2, 1, 128, 64), (300, 300, 3, 3, 64, 32), (600, 2100, 4, 2, 128, 128),
    (40, 9000, 12, 2, 64, 64)])
@pytest.mark.parametrize("mask", [0, 1, 2, 3])
def test_attention_nan_values_stay_in_their_element_and_tile(nq, n, hq, hk, d, pt, mask):
    """A NaN among a token's values makes that element of the queries that see the
    token NaN.  Of the others only rows of a tile of 256 that holds a query which
    sees it may be NaN there; nothing else changes, other heads, elements and
    sequences included."""
    kw = MASKS[mask]
    pages = -(-n // pt) + 1
    c = filled(pages + 2, hk, pt, d, 151)
    order = torch.randperm(pages + 2, generator=gen(152), device=DEV).to(torch.int32)
    t = torch.stack([order[:pages], order[-2:].repeat(pages)[:pages]]).contiguous()
    q = torch.randn((nq + 2, hq, d), generator=gen(153), device=DEV).bfloat16()
    args = (t, i32([n, 30]), i32([0, nq, nq + 2]))
    lse = [torch.empty((nq + 2, hq), device=DEV) for _ in "ab"]
    clean = nv.kv8_attention(q, c, *args, max_q=nq + 1, lse=lse[0], **kw)
    must = torch.zeros((nq + 2, hq, d), dtype=torch.bool, device=DEV)
    may = torch.zeros_like(must)
    ok = ref.seen(nq, n, kw["causal"], kw.get("window", -1), kw.get("sink", 0), DEV)
    g = hq // hk
    tile = (torch.arange(nq, device=DEV)[:, None] * g + torch.arange(g, device=DEV)) // 256  # [nq, g]
    for i, (key, col) in enumerate([(0, 3), (3, 40), (n // 2, 17), (n - nq, 0), (n - nq // 2 - 1, d - 1),
                                    (n - 1, 33), (n - 1, 31), (max(0, n - 120), 5), (n - nq // 3 - 1, 62)]):
        head = i % hk
        c.v_codes[t[0, key // pt].long(), head, key % pt, col] = (0x7F, 0xFF)[i % 2]
        group = slice(head * g, (head + 1) * g)
        sees = ok[:, key]
        must[:nq, group, col] |= sees[:, None]
        may[:nq, group, col] |= torch.isin(tile, tile[sees])
    out = nv.kv8_attention(q, c, *args, max_q=nq + 1, lse=lse[1], **kw)
    assert out[must].isnan().all()
    assert torch.equal(out[~may], clean[~may])
    assert (out[may].isnan() | (out[may] == clean[may])).all()
    assert torch.equal(lse[0], lse[1])


@pytest.mark.parametrize("call", ["token", "chunk", "read", "rope"])
def test_outputs_dropped_while_the_callers_stream_still_reads_them(call):
    """Calls on a stream of their own, one after the other, whose outputs another
    stream reads late and that are dropped before: none gets the memory of one that
    has yet to be read."""
    heads, d, n = 2, 128, 900
    c = filled(16, heads, 64, d, 161)
    t = torch.arange(15, device=DEV, dtype=torch.int32)[None].contiguous()
    nq = 1 if call == "token" else 300
    xs = [torch.randn((nq, heads, d), generator=gen(162 + i), device=DEV).bfloat16() for i in range(4)]
    lens, starts, begins = i32([n]), i32([0, nq]), [i32([100 * i]) for i in range(4)]
    pos = torch.arange(nq, device=DEV, dtype=torch.int32)[:, None].contiguous()

    def go(i, stream=None):
        if call == "read":
            return nv.kv8_read(c, t, begins[i], starts, nq, stream=stream)
        if call == "rope":
            return nv.rope([xs[i]], pos, [64], stream=stream)
        return [nv.kv8_attention(xs[i], c, t, lens, starts, stream=stream)]

    want = [[o.clone() for o in go(i)] for i in range(4)]
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    torch.cuda.synchronize()
    late = []
    for i in range(4):
        outs = go(i, side)
        here.wait_stream(side)
        torch.cuda._sleep(5_000_000)
        late.append([o.clone() for o in outs])
        del outs
    torch.cuda.synchronize()
    for a, b in zip(late, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("nq,n,hq,hk", [(1, 1500, 4, 4), (5, 1000, 12, 2), (40, 2000, 4, 2), (300, 3000, 2, 1),
                                        (700, 9000, 4, 2)])
@pytest.mark.parametrize("pt,d", [(32, 64), (64, 64), (128, 64), (32, 128), (64, 128), (128, 128)])
@pytest.mark.parametrize("window,sink", [(100, 0), (333, 40), (0, 70)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_pages_out_of_the_window_may_be_gone(nq, n, hq, hk, pt, d, window, sink, causal):
    """Pages between the sink and the window of the first query may be freed: their
    entries name none, or one that is full of NaN, and no error is recorded."""
    mask = dict(causal=causal, window=window, sink=sink)
    pages = -(-n // pt)
    c = filled(pages + 1, hk, pt, d, 171)
    for codes in (c.k_codes, c.v_codes):
        codes[pages].fill_(0x7F)
    t = torch.randperm(pages, generator=gen(172), device=DEV).to(torch.int32)[None].contiguous()
    q = torch.randn((nq, hq, d), generator=gen(173), device=DEV).bfloat16()
    lens, starts = i32([n]), i32([0, nq])
    ws = nv.kv8_attention_workspace(c, t, starts, hq, nq)
    want = nv.kv8_attention(q, c, t, lens, starts, ws=ws, **mask)
    seen = ref.seen(nq, n, causal, window, sink, DEV).any(0)
    unseen = ~torch.nn.functional.pad(seen, (0, pages * pt - n)).view(pages, pt).any(1)
    assert unseen.any()
    for gone in (-1, pages, 2 ** 31 - 1, c.k_codes.shape[0]):
        less = torch.where(unseen[None], torch.full_like(t, gone), t)
        out = nv.kv8_attention(q, c, less, lens, starts, ws=ws, **mask)
        assert nv.device_error(ws) == 0
        assert torch.equal(out, want)


def test_no_sequences_no_rows_no_tokens():
    """Empty batches, and batches whose sequences have no rows, do nothing."""
    c = filled(4, 2, 64, 128, 181)
    kept = [x.clone() for x in (c.k_codes, c.v_codes, c.k_scales, c.v_scales)]
    x = torch.randn((0, 2, 128), device=DEV).bfloat16()
    for n in (0, 1, 3):
        t = torch.zeros((n, 2), dtype=torch.int32, device=DEV)
        lens, starts = i32([5] * n), i32([0] * (n + 1))
        ws = nv.kv8_attention_workspace(c, t, starts, 4, 1)
        nv.kv8_write(c, x, x, t, lens, starts, ws=ws)
        k, v = nv.kv8_read(c, t, lens, starts, 0, ws=ws)
        assert k.shape == v.shape == (0, 2, 128)
        q = torch.randn((0, 4, 128), device=DEV).bfloat16()
        assert nv.kv8_attention(q, c, t, lens, starts).shape == (0, 4, 128)
        # rows that belong to no sequence
        y = torch.randn((7, 2, 128), generator=gen(182), device=DEV).bfloat16()
        nv.kv8_write(c, y, y, t, lens, starts, ws=ws)
        outs = [torch.full_like(y, 4.0) for _ in "kv"]
        nv.kv8_read(c, t, lens, starts, 7, outs=outs, ws=ws)
        out = torch.full((7, 4, 128), 4.0, device=DEV).bfloat16()
        nv.kv8_attention(torch.zeros_like(out), c, t, lens, starts, max_q=7, out=out, lse=None)
        assert all((o == 4.0).all() for o in (*outs, out))
        assert nv.device_error(ws) == 0
    pos = torch.zeros((0, 3), dtype=torch.int32, device=DEV)
    assert nv.rope([x, x[:, :1]], pos, [22, 21, 21])[1].shape == (0, 1, 128)
    for a, b in zip(kept, (c.k_codes, c.v_codes, c.k_scales, c.v_scales)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("nq,n", [(1, 200), (1, 1500), (2, 9000), (40, 700), (600, 2500)])
def test_attention_in_place_of_q(nq, n):
    """out may be q itself: a tile reads its rows before it writes any of them."""
    hk, hq, d = 2, 6, 128
    pages = -(-n // 64)
    c = filled(pages, hk, 64, d, 183)
    t = torch.arange(pages, device=DEV, dtype=torch.int32)[None].contiguous()
    qkv = torch.randn((nq, hq + 2 * hk, d), generator=gen(184), device=DEV).bfloat16()
    args = (c, t, i32([n]), i32([0, nq]))
    before = qkv.clone()
    want = nv.kv8_attention(qkv[:, :hq], *args, causal=True)
    for _ in range(5):
        qkv.copy_(before)
        nv.kv8_attention(qkv[:, :hq], *args, causal=True, out=qkv[:, :hq])
        assert torch.equal(qkv[:, :hq], want) and torch.equal(qkv[:, hq:], before[:, hq:])
