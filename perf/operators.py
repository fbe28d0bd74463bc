"""The attention-side operators around the low-precision KV cache, as workloads.

Four operators a video or language model runs between its projections:

* ``rope``    rotary positions over several axes (time, height, width) on queries
              and keys, forward and backward (the inverse rotation);
* ``write``   quantizing keys and values into an 8-bit paged cache as they come,
              one power-of-two scale per page and head;
* ``read``    the dequantized tokens of a cache back as contiguous rows;
* ``attend``  attention of queries over that cache, from one token to chunks.

``run`` computes the plain form (elementary torch operations in 32 bits) or,
with ``own`` set, makes the package's calls.  The cache of both forms:

    codes  uint8 (E4M3) [pages, heads, page_tokens, head_dim], K and V
    scales float32 [pages, heads], powers of two: 2^e with the smallest e that
           has amax <= 448 * 2^e over the finite values written to that page and
           head so far, e in [-40, 40]; a page's earlier codes are brought to a
           scale that has grown

Sequence b of a batch holds its tokens in the pages page_table[b, 0], [b, 1], ...
"""
import math

import torch

own = False

E_MIN, E_MAX = -40, 40  # exponents of the cache's scales


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one new token of one stream: the call is all latency
        dict(name="rope token", op="rope", tokens=1, q_heads=24, k_heads=24, head_dim=128,
             sections="22,21,21", grid_h=30, grid_w=52, first=20, theta=10000.0, dtype="bf16",
             interleaved=True, per_axis=True, inverse=False),
        # a chunk of three latent frames of 30 x 52 tokens, q and k out of one QKV projection
        dict(name="rope chunk", op="rope", tokens=4680, q_heads=24, k_heads=24, head_dim=128,
             sections="22,21,21", grid_h=30, grid_w=52, first=18, theta=10000.0, dtype="bf16",
             interleaved=True, per_axis=True, inverse=False),
        # a training step's gradients of q and k in fp32: grouped heads, far positions, an odd length
        dict(name="rope gradient fp32", op="rope", tokens=2641, q_heads=16, k_heads=4, head_dim=128,
             sections="16,24,24", grid_h=17, grid_w=31, first=70000, theta=1000000.0, dtype="f32",
             interleaved=False, per_axis=False, inverse=True),
        # a serving step: one token of each of 32 streams into partly filled pages
        dict(name="write tokens", op="write", seqs=32, least=1, most=1, before=700, heads=8,
             head_dim=128, page=64, dtype="bf16"),
        # eight latent frames of 1560 tokens after an odd number of cached tokens
        dict(name="write chunk", op="write", seqs=1, least=12480, most=12480, before=4711, heads=24,
             head_dim=128, page=64, dtype="bf16"),
        # the sink and window of a stream, 15 frames of 1560 tokens, as bf16 rows
        dict(name="read window", op="read", seqs=1, least=23400, most=23400, begin=1560, heads=24,
             head_dim=128, page=64, dtype="bf16"),
        # short ragged streams, read back in fp32 to be looked at
        dict(name="read ragged fp32", op="read", seqs=7, least=90, most=900, begin=13, heads=4,
             head_dim=64, page=32, dtype="f32"),
        # one token of one stream over a frame of context
        dict(name="attend token", op="attend", seqs=1, q_least=1, q_most=1, kv_least=1561,
             kv_most=1561, q_heads=24, k_heads=24, head_dim=128, page=64, causal=True, window=-1,
             sink=0, lse=False),
        # a serving step: 32 ragged streams, up to a 21-frame cache each, grouped heads
        dict(name="attend batch", op="attend", seqs=32, q_least=1, q_most=1, kv_least=800,
             kv_most=32760, q_heads=32, k_heads=8, head_dim=128, page=64, causal=True, window=-1,
             sink=0, lse=False),
        # a few drafted tokens of each stream are checked at once; small heads and pages
        dict(name="attend drafts", op="attend", seqs=8, q_least=5, q_most=5, kv_least=4100,
             kv_most=8200, q_heads=24, k_heads=4, head_dim=64, page=32, causal=True, window=-1,
             sink=0, lse=True),
        # prompts of three streams, causal with a sliding window and a sink
        dict(name="attend prompts", op="attend", seqs=3, q_least=1000, q_most=4000, kv_least=4000,
             kv_most=8190, q_heads=32, k_heads=8, head_dim=128, page=128, causal=True, window=2500,
             sink=64, lse=True),
        # a chunk of three frames attends to the whole 21-frame cache
        dict(name="attend chunk", op="attend", seqs=1, q_least=4680, q_most=4680, kv_least=32760,
             kv_most=32760, q_heads=24, k_heads=24, head_dim=128, page=64, causal=False, window=-1,
             sink=0, lse=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attend", "attend"])
    d = rng.choice([64, 128])
    page = rng.choice([32, 64, 128])
    if op == "rope":
        pairs = d // 2
        a = rng.randint(1, pairs // 2)
        b = rng.randint(0, (pairs - a) // 2)
        c = pairs - a - b - rng.choice([0, 0, 4])
        k = rng.choice([1, 4, 8, 24])
        return dict(op=op, tokens=_log(rng, 1, 4680), q_heads=rng.choice([k, 24]), k_heads=k,
                    head_dim=d, sections="%d,%d,%d" % (a, b, c), grid_h=rng.randint(3, 30),
                    grid_w=rng.randint(3, 52), first=_log(rng, 1, 100000),
                    theta=rng.choice([10000.0, 1000000.0]), dtype=rng.choice(["bf16", "f32"]),
                    interleaved=rng.random() < 0.5, per_axis=rng.random() < 0.5,
                    inverse=rng.random() < 0.5)
    if op == "write":
        most = _log(rng, 1, 12480)
        return dict(op=op, seqs=max(1, min(32, 12480 // most, _log(rng, 1, 32))),
                    least=max(1, most // 3), most=most, before=_log(rng, 1, 5000),
                    heads=rng.choice([1, 4, 8, 24]), head_dim=d, page=page,
                    dtype=rng.choice(["bf16", "f32"]))
    if op == "read":
        most = _log(rng, 1, 20000)
        return dict(op=op, seqs=max(1, min(32, 20000 // most, _log(rng, 1, 32))),
                    least=max(1, most // 3), most=most, begin=rng.randint(0, 200),
                    heads=rng.choice([1, 4, 8, 24]), head_dim=d, page=page,
                    dtype=rng.choice(["bf16", "f32"]))
    k = rng.choice([1, 2, 4, 8, 24])
    group = rng.choice([1, 1, 4, 6, 8]) if k < 24 else 1
    q_most = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 17, 4000)])
    kv = max(_log(rng, 200, 32760), q_most)
    room = 4.0e8 if q_most > 1 else 1.6e9  # values of the scores, or of the cache
    size = q_most * kv * k * group if q_most > 1 else kv * k * d
    return dict(op=op, seqs=max(1, min(32, int(room / size), _log(rng, 1, 32))),
                q_least=max(1, q_most // 2), q_most=q_most, kv_least=max(q_most, kv // 3),
                kv_most=kv, q_heads=k * group, k_heads=k, head_dim=d, page=page,
                causal=rng.random() < 0.7, window=rng.choice([-1, -1, max(1, kv // 4)]),
                sink=rng.choice([0, 40]), lse=rng.random() < 0.5)


# ----------------------------------------------------------------- the inputs
def _between(least, most, n):
    """n lengths spread over [least, most], the longest last."""
    return [most - (most - least) * (n - 1 - i) // max(1, n - 1) for i in range(n)]


def _starts(lens, dev="cuda"):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device=dev), c[-1]


def _cache(g, case, lens, heads):
    """A paged cache of random tokens: per page and head a power-of-two scale and
    codes that fill its range the way normally distributed values do."""
    pt, d = case["page"], case["head_dim"]
    need = [-(-n // pt) for n in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda")
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n].to(torch.int32)
        at += n

    def codes():
        c = torch.empty((pages, heads, pt, d), dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 27) // (heads * pt * d))
        for p in range(0, pages, step):
            x = torch.randn((min(step, pages - p), heads, pt, d), generator=g, device="cuda",
                            dtype=torch.float32)
            c[p:p + step] = (x * 80.0).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        return c

    def scales(lo, hi):
        e = torch.randint(lo, hi + 1, (pages, heads), generator=g, device="cuda")
        return torch.ldexp(torch.ones((), device="cuda"), e).float()

    return dict(k_codes=codes(), v_codes=codes(), k_scales=scales(-7, -6), v_scales=scales(-8, -5),
                table=table)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = torch.bfloat16 if case.get("dtype", "bf16") == "bf16" else torch.float32
    op, d = case["op"], case["head_dim"]

    def rows(t, heads, std=1.0):
        return (torch.randn((t, heads, d), generator=g, device="cuda") * std).to(dt)

    s = dict(case=case)
    if op == "rope":
        t, hq, hk = case["tokens"], case["q_heads"], case["k_heads"]
        qkv = rows(t, hq + 2 * hk)  # the projection's output: q, k and v side by side
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        i = torch.arange(t, device="cuda")
        h, w = case["grid_h"], case["grid_w"]
        shift = int(torch.randint(0, 8, (1,), generator=g, device="cuda").item())
        s["positions"] = torch.stack([case["first"] + shift + i // (h * w), i // w % h, i % w],
                                     dim=1).to(torch.int32)
        s["sections"] = [int(v) for v in case["sections"].split(",")]
    elif op == "write":
        new = _between(case["least"], case["most"], case["seqs"])
        before = [case["before"] + 37 * b for b in range(case["seqs"])]
        s.update(_cache(g, case, [a + n for a, n in zip(before, new)], case["heads"]))
        s["cu"], total = _starts(new)
        s["lens"] = torch.tensor(before, dtype=torch.int32, device="cuda")
        s["most"] = case["most"]
        kv = rows(total, 2 * case["heads"])
        s["k"], s["v"] = kv[:, :case["heads"]], kv[:, case["heads"]:]
        # the pages a write touches, as (sequence, place in its table)
        pt = case["page"]
        touched = [(b, p) for b, (a, n) in enumerate(zip(before, new))
                   for p in range(a // pt, (a + n - 1) // pt + 1)]
        s["touched"] = torch.tensor(touched, device="cuda")
    elif op == "read":
        n = _between(case["least"], case["most"], case["seqs"])
        begin = [case["begin"] + 5 * b for b in range(case["seqs"])]
        s.update(_cache(g, case, [a + m for a, m in zip(begin, n)], case["heads"]))
        s["cu"], s["total"] = _starts(n)
        s["begin"] = torch.tensor(begin, dtype=torch.int32, device="cuda")
        s["most"] = case["most"]
        s["row_seq"] = torch.repeat_interleave(torch.arange(len(n), device="cuda"),
                                               torch.tensor(n, device="cuda"))
    else:
        nq = _between(case["q_least"], case["q_most"], case["seqs"])
        kv = _between(case["kv_least"], case["kv_most"], case["seqs"])
        s.update(_cache(g, case, kv, case["k_heads"]))
        s["cu"], total = _starts(nq)
        s["lens"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
        s["most"] = case["q_most"]
        s["q"] = rows(total, case["q_heads"], 1.5)
        s["row_seq"] = torch.repeat_interleave(torch.arange(len(nq), device="cuda"),
                                               torch.tensor(nq, device="cuda"))
    return s


# -------------------------------------------------------------- the plain forms
def _plain_rope(s):
    c = s["case"]
    sec = s["sections"]
    n = sum(sec)
    freqs, axes = [], []
    for a, m in enumerate(sec):
        for j in range(m):
            power = j / m if c["per_axis"] else (sum(sec[:a]) + j) / n
            freqs.append(c["theta"] ** -power)
            axes.append(a)
    freqs = torch.tensor(freqs, dtype=torch.float64, device="cuda")
    axes = torch.tensor(axes, device="cuda")
    angle = s["positions"][:, axes].double() * freqs  # far positions: 64 bits
    if c["inverse"]:
        angle = -angle
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    outs = []
    for x in (s["q"], s["k"]):
        f = x.float()
        if c["interleaved"]:
            a, b = f[..., 0:2 * n:2], f[..., 1:2 * n:2]
            turned = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
        else:
            a, b = f[..., :n], f[..., n:2 * n]
            turned = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
        outs.append(torch.cat([turned, f[..., 2 * n:]], dim=-1).to(x.dtype))
    return outs


def _plain_write(s):
    c = s["case"]
    pt = c["page"]
    b, p = s["touched"][:, 0], s["touched"][:, 1]
    pos = p[:, None] * pt + torch.arange(pt, device="cuda")  # [touched, pt]
    start, lens = s["cu"][:-1].long()[b][:, None], s["lens"].long()[b][:, None]
    count = (s["cu"][1:] - s["cu"][:-1]).long()[b][:, None]
    new = (pos >= lens) & (pos < lens + count)
    old = pos < lens
    row = (start + pos - lens).clamp(0, s["k"].shape[0] - 1)
    page = s["table"].long()[b, p]
    out = []
    for x, codes, scales in ((s["k"], s["k_codes"], s["k_scales"]),
                             (s["v"], s["v_codes"], s["v_scales"])):
        x = x[row].float().transpose(1, 2)  # [touched, heads, pt, d]
        here = new[:, None, :, None]
        size = torch.where(here & torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax((2, 3))
        m, e = torch.frexp(size)
        e = torch.where(size > 0, e - 9 + (m > 0.875).int(), torch.full_like(e, E_MIN))
        scale = torch.ldexp(torch.ones_like(size), e.clamp(E_MIN, E_MAX))
        before = scales[page]
        scale = torch.where(old.any(1)[:, None], torch.maximum(scale, before), scale)
        wide = scale[..., None, None]
        was = codes[page].view(torch.float8_e4m3fn).float()
        kept = was * (before / scale)[..., None, None]
        y = torch.where(here, (x / wide).clamp(-448, 448), torch.where(old[:, None, :, None], kept, was))
        codes[page] = y.to(torch.float8_e4m3fn).view(torch.uint8)
        scales[page] = scale
        out += [codes.view(torch.float8_e4m3fn), scales]
    return out


def _plain_read(s):
    c = s["case"]
    pt = c["page"]
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    b = s["row_seq"]
    pos = torch.arange(s["total"], device="cuda") - s["cu"].long()[b] + s["begin"].long()[b]
    page, slot = s["table"].long()[b, pos // pt], pos % pt
    out = []
    for codes, scales in ((s["k_codes"], s["k_scales"]), (s["v_codes"], s["v_scales"])):
        x = codes.view(torch.float8_e4m3fn)[page, :, slot].float()
        out.append((x * scales[page][..., None]).to(dt))
    return out


def _plain_attend(s):
    c = s["case"]
    pt, d, hk, n = c["page"], c["head_dim"], c["k_heads"], c["seqs"]
    group = c["q_heads"] // hk
    table = s["table"].long().clamp(min=0)
    width = table.shape[1] * pt

    def tokens(codes, scales):  # [n, heads, tokens, d]
        x = codes[table].view(torch.float8_e4m3fn).float() * scales[table][..., None, None]
        return x.transpose(1, 2).reshape(n, hk, width, d)

    cu, lens = s["cu"].long(), s["lens"].long()
    count = cu[1:] - cu[:-1]
    i = torch.arange(s["most"], device="cuda")
    row = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)  # [n, queries]
    q = s["q"][row].float().reshape(n, s["most"], hk, group, d).permute(0, 2, 3, 1, 4)
    q = q.reshape(n, hk, group * s["most"], d)
    k = tokens(s["k_codes"], s["k_scales"])
    scores = (q @ k.transpose(-1, -2)).reshape(n, hk, group, s["most"], width) * d ** -0.5
    del k
    at = (lens[:, None] - count[:, None] + i)[..., None]  # a query's place in its sequence
    j = torch.arange(width, device="cuda")
    seen = (j < lens[:, None, None]).expand(n, s["most"], width)
    if c["causal"]:
        seen = seen & (j <= at)
    if c["window"] >= 0:
        seen = seen & ((at - j <= c["window"]) | (j < c["sink"]))
    scores = scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    weights = scores.sub_(top).exp_()
    total = weights.sum(-1)
    v = tokens(s["v_codes"], s["v_scales"])
    o = weights.reshape(n, hk, group * s["most"], width) @ v
    o = o.reshape(n, hk, group, s["most"], d)
    o = torch.where(total[..., None] > 0, o / total[..., None], torch.zeros_like(o))
    place = torch.arange(s["q"].shape[0], device="cuda") - cu[s["row_seq"]]
    out = o.permute(0, 3, 1, 2, 4)[s["row_seq"], place].reshape(-1, c["q_heads"], d).to(s["q"].dtype)
    if not c["lse"]:
        return [out]
    lse = (top[..., 0] + total.log()).permute(0, 3, 1, 2)[s["row_seq"], place]
    return [out, lse.reshape(-1, c["q_heads"])]


# --------------------------------------------------------------- one pass of each
def run(state):
    s, c = state, state["case"]
    if own:
        import nvfp4_block_scaled_20_b200 as nv
        if c["op"] == "rope":
            return nv.rope([s["q"], s["k"]], s["positions"], s["sections"], theta=c["theta"],
                           interleaved=c["interleaved"], per_axis=c["per_axis"],
                           inverse=c["inverse"])
        cache = s.get("cache")
        if cache is None:  # kept by a program as long as its cache lives
            cache = s["cache"] = nv.KV8Cache(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"])
            s["ws"] = nv.workspace(0) if c["op"] != "attend" else nv.kv8_attention_workspace(
                cache, s["table"], s["cu"], c["q_heads"], max_q=s["most"])
        if c["op"] == "write":
            nv.kv8_write(cache, s["k"], s["v"], s["table"], s["lens"], s["cu"], max_new=s["most"],
                         ws=s["ws"])
            return [cache.k_codes.view(torch.float8_e4m3fn), cache.k_scales,
                    cache.v_codes.view(torch.float8_e4m3fn), cache.v_scales]
        if c["op"] == "read":
            return nv.kv8_read(cache, s["table"], s["begin"], s["cu"], s["total"],
                               max_tokens=s["most"],
                               out_dtype=torch.bfloat16 if c["dtype"] == "bf16" else torch.float32,
                               ws=s["ws"])
        lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda") if c["lse"] else None
        out = nv.kv8_attention(s["q"], cache, s["table"], s["lens"], s["cu"], max_q=s["most"],
                               causal=c["causal"], window=c["window"], sink=c["sink"], lse=lse,
                               ws=s["ws"])
        return [out] if lse is None else [out, lse]
    return {"rope": _plain_rope, "write": _plain_write, "read": _plain_read,
            "attend": _plain_attend}[c["op"]](s)


# ---------------------------------------------------------- what a pass cannot do without
def _seen(case, nq, kv):
    """Key positions that the queries of one sequence see, summed, and how many
    distinct ones."""
    total, least, sunk = 0, kv, 0
    for i in range(nq):
        at = kv - nq + i
        hi = min(kv, at + 1) if case["causal"] else kv
        lo = max(0, at - case["window"]) if case["window"] >= 0 else 0
        sink = min(case["sink"], lo, hi) if case["window"] >= 0 else 0
        total += max(0, hi - lo) + sink
        least, sunk = min(least, lo), max(sunk, sink)
    return total, (kv - least) + min(sunk, least)


def work(case):
    op, d = case["op"], case["head_dim"]
    size = 2 if case.get("dtype", "bf16") == "bf16" else 4
    if op == "rope":
        values = case["tokens"] * (case["q_heads"] + case["k_heads"]) * d
        return dict(bytes=2 * values * size + case["tokens"] * 12, flops=3 * values)
    if op == "write":
        tokens = sum(_between(case["least"], case["most"], case["seqs"]))
        values = 2 * tokens * case["heads"] * d
        return dict(bytes=values * (size + 1) + 8 * case["heads"] * -(-tokens // case["page"]),
                    flops=3 * values)
    if op == "read":
        tokens = sum(_between(case["least"], case["most"], case["seqs"]))
        values = 2 * tokens * case["heads"] * d
        return dict(bytes=values * (size + 1) + 8 * case["heads"] * -(-tokens // case["page"]),
                    flops=values)
    nbytes = flops = 0
    for nq, kv in zip(_between(case["q_least"], case["q_most"], case["seqs"]),
                      _between(case["kv_least"], case["kv_most"], case["seqs"])):
        pairs, keys = _seen(case, nq, kv)
        nbytes += 4 * nq * case["q_heads"] * d + 2 * keys * case["k_heads"] * d
        nbytes += 8 * case["k_heads"] * -(-keys // case["page"])
        nbytes += 4 * nq * case["q_heads"] if case["lse"] else 0
        flops += 4 * pairs * case["q_heads"] * d
    return dict(bytes=nbytes, flops=flops)


# ------------------------------------------------------------------- in 64 bits
def _e4m3(y):
    """The nearest E4M3 value (ties to even, saturating) of float64 values."""
    a = y.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(y) * torch.clamp(torch.round(a / step) * step, max=448.0)


def _token(s, which, b, pos):
    """Dequantized rows [len(pos), heads, d] of sequence b, in float64."""
    pt = s["case"]["page"]
    page = s["table"][b].long()[pos // pt]
    codes, scales = s[which + "_codes"], s[which + "_scales"]
    x = codes.view(torch.float8_e4m3fn)[page, :, pos % pt].double()
    return x * scales[page].double()[:, :, None]


def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], case["head_dim"]
    if op == "rope":
        n, outs = sum(s["sections"]), []
        axis = [a for a, m in enumerate(s["sections"]) for _ in range(m)]
        local = [j for m in s["sections"] for j in range(m)]
        for x in (s["q"], s["k"]):
            y = x.double().clone()
            for i in range(n):
                part = s["sections"][axis[i]] if case["per_axis"] else n
                rate = math.exp(-math.log(case["theta"]) * (local[i] if case["per_axis"] else i) / part)
                turn = s["positions"][:, axis[i]].double() * rate * (-1 if case["inverse"] else 1)
                z = torch.polar(torch.ones_like(turn), turn)[:, None]
                at = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + n)
                z = z * torch.complex(x[..., at[0]].double(), x[..., at[1]].double())
                y[..., at[0]], y[..., at[1]] = z.real, z.imag
            outs.append(y)
        return outs
    if op == "write":
        pt, cu, lens = case["page"], s["cu"].tolist(), s["lens"].tolist()
        out = []
        for which in ("k", "v"):
            codes = s[which + "_codes"].view(torch.float8_e4m3fn).double()
            scales = s[which + "_scales"].double()
            for b in range(case["seqs"]):
                x, at = s[which][cu[b]:cu[b + 1]].double(), lens[b]
                while x.shape[0]:
                    page, first = int(s["table"][b, at // pt]), at % pt
                    m = min(pt - first, x.shape[0])
                    part = x[:m].transpose(0, 1)  # [heads, m, d]
                    e = torch.ceil(torch.log2(part.abs().amax((1, 2)) / 448.0))
                    scale = torch.exp2(e.clamp(E_MIN, E_MAX))
                    if first:
                        scale = torch.maximum(scale, scales[page])
                        codes[page, :, :first] = _e4m3(codes[page, :, :first]
                                                       * (scales[page] / scale)[:, None, None])
                    codes[page, :, first:first + m] = _e4m3(part / scale[:, None, None])
                    scales[page] = scale
                    x, at = x[m:], at + m
            out += [codes, scales]
        return out
    if op == "read":
        cu, begin = s["cu"].tolist(), s["begin"].tolist()
        return [torch.cat([_token(s, w, b, begin[b] + torch.arange(cu[b + 1] - cu[b], device="cuda"))
                           for b in range(case["seqs"])]) for w in ("k", "v")]
    cu, lens, group = s["cu"].tolist(), s["lens"].tolist(), case["q_heads"] // case["k_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b in range(case["seqs"]):
        j = torch.arange(lens[b], device="cuda")
        k, v = _token(s, "k", b, j), _token(s, "v", b, j)
        nq = cu[b + 1] - cu[b]
        at = torch.arange(lens[b] - nq, lens[b], device="cuda")[:, None]
        hidden = torch.zeros((nq, lens[b]), dtype=torch.bool, device="cuda")
        if case["causal"]:
            hidden |= j > at
        if case["window"] >= 0:
            hidden |= (j < at - case["window"]) & (j >= case["sink"])
        for h in range(case["q_heads"]):
            x = s["q"][cu[b]:cu[b + 1], h].double() @ k[:, h // group].T / math.sqrt(d)
            x = x.masked_fill(hidden, -math.inf)
            lse[cu[b]:cu[b + 1], h] = torch.logsumexp(x, dim=-1)
            out[cu[b]:cu[b + 1], h] = torch.softmax(x, dim=-1) @ v[:, h // group]
    empty = torch.isinf(lse)
    out[empty] = 0.0
    return [out, lse] if case["lse"] else [out]
