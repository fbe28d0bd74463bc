"""Plain float64 forms of the attention-side operators (rotary positions, the
8-bit paged cache, attention over it), with error bounds, for the tests."""
import math

import torch

E_MIN, E_MAX = -40, 40


# ------------------------------------------------------------------- rope
def rope(x, positions, sections, theta, interleaved, per_axis, inverse):
    """float64 [tokens, heads, dim] of any input type."""
    y = x.double().cpu().clone()
    pos = positions.cpu().double()
    n = sum(sections)
    at = 0
    for axis, m in enumerate(sections):
        for j in range(m):
            power = j / m if per_axis else at / n
            turn = pos[:, axis] * theta ** -power * (-1 if inverse else 1)
            a, b = (2 * at, 2 * at + 1) if interleaved else (at, at + n)
            c, s = turn.cos()[:, None], turn.sin()[:, None]
            x0, x1 = x[..., a].double().cpu(), x[..., b].double().cpu()
            y[..., a] = x0 * c - x1 * s
            y[..., b] = x0 * s + x1 * c
            at += 1
    return y


def rope_bound(x, sections, interleaved, ref, dtype):
    """|error| of the fp32 rotation: the angle's fraction of a turn rounded to
    fp32 (half a step of 0.5: 2^-26 turns = 9.4e-8 rad), 2 ulp each of the sine
    and cosine (2^-23), two products and a sum (3 half steps of 2^-24): below
    4e-7 (|x0| + |x1|); then half a step of the output's type."""
    n = sum(sections)
    a = x.double().cpu().abs()
    size = torch.zeros_like(a)
    for i in range(n):
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        size[..., p] = size[..., q] = a[..., p] + a[..., q]
    half = torch.finfo(dtype).eps / 2
    return 4e-7 * size + half * ref.abs()


# ------------------------------------------------------------------ cache
def e4m3(y):
    """The nearest E4M3 value (ties to even, saturating), NaN kept; float64."""
    a = y.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.copysign(torch.clamp(torch.round(a / step) * step, max=448.0), y)


def values(codes):
    return codes.view(torch.float8_e4m3fn).double()


def write(codes, scales, x, table, lens, starts):
    """In place on CPU float64 `codes` (values before the scale) [pages, heads,
    pt, d] and `scales`; x [rows, heads, d]."""
    pt = codes.shape[2]
    x = x.double().cpu()
    for s in range(len(lens)):
        rows, at = x[starts[s]:starts[s + 1]], lens[s]
        while rows.shape[0]:
            page, first = table[s][at // pt], at % pt
            m = min(pt - first, rows.shape[0])
            part = rows[:m].transpose(0, 1)
            finite = torch.where(torch.isfinite(part), part.abs(), torch.zeros_like(part))
            amax = finite.amax((1, 2))
            e = torch.ceil(torch.log2(amax / 448.0)).clamp(E_MIN, E_MAX)
            e = torch.where(amax == 0, torch.full_like(e, E_MIN), e)
            scale = torch.exp2(e)
            if first:
                scale = torch.maximum(scale, scales[page])
                ratio = (scales[page] / scale)[:, None, None]
                codes[page, :, :first] = e4m3(codes[page, :, :first] * ratio)
            codes[page, :, first:first + m] = e4m3(part / scale[:, None, None])
            scales[page] = scale
            rows, at = rows[m:], at + m


def tokens(codes, scales, table_row, n):
    """Dequantized float64 [n, heads, d] of the first n tokens of a sequence."""
    pt = codes.shape[2]
    pos = torch.arange(n, device=codes.device)
    page = table_row.long()[pos // pt]
    return values(codes)[page, :, pos % pt] * scales[page].double()[:, :, None]


# -------------------------------------------------------------- attention
def seen(nq, n, causal, window, sink, device):
    j = torch.arange(n, device=device)[None]
    at = torch.arange(n - nq, n, device=device)[:, None]
    ok = torch.ones((nq, n), dtype=torch.bool, device=device)
    if causal:
        ok &= j <= at
    if window >= 0:
        ok &= (j >= torch.clamp(at, min=0) - window) | (j < sink)
    return ok


def attention(q, k, v, v_codes_abs, v_scale, scale, ok):
    """One sequence in float64: q [nq, hq, d], k, v [n, hk, d] dequantized, ok
    [nq, n].  Returns out, lse, and bounds on the error of each.

    Weights: a score is a sum of d exact products in fp32, each step off by at
    most one unit of the partial sums (2^-23 of sum |q k|); times the scale, and
    minus the maximum, in units of log2, two roundings of 2^-24 of the numbers
    met (|t|, 40 for a V scale's exponent, the maximum): delta per weight in
    all; 2^-21 for exp2 and the fp32 sums' first steps, n 2^-24 for long sums.
    Each weight is rounded to fp16: 2^-11 of itself, or, below fp16's normal
    range, 2^-25 where the largest is at least 1."""
    nq, hq, d = q.shape
    n, hk = k.shape[0], k.shape[1]
    group = hq // hk
    out = torch.zeros((nq, hq, d), dtype=torch.float64, device=q.device)
    lse = torch.full((nq, hq), -math.inf, dtype=torch.float64, device=q.device)
    e_out, e_lse = torch.zeros_like(out), torch.zeros_like(lse)
    if n == 0:
        return out, lse, e_out, e_lse
    for h in range(hq):
        kk, vv = k[:, h // group], v[:, h // group]
        s = (q[:, h] @ kk.T) * scale
        size = (q[:, h].abs() @ kk.abs().T) * scale
        s = s.masked_fill(~ok, -math.inf)
        some = ok.any(-1)
        top = s.amax(-1, keepdim=True)
        w = torch.exp(s - torch.where(some[:, None], top, torch.zeros_like(top)))
        w = w.masked_fill(~ok, 0.0)
        total = w.sum(-1, keepdim=True).clamp(min=1e-300)
        p = w / total
        out[:, h] = p @ vv
        lse[:, h] = torch.where(some, (top + total.log())[:, 0], lse[:, h])
        delta = torch.where(ok, d * 2.0 ** -23 * size + 2.0 ** -23 * (2 * s.abs() + 40), 0 * size)
        delta = delta.amax(-1) + 2.0 ** -21 + n * 2.0 ** -24
        spread = p @ vv.abs()
        tiny = 2.0 ** -25 * (ok.double() @ v_codes_abs[:, h // group]) * v_scale[:, h // group].max()
        e_out[:, h] = (2 * delta[:, None] + 2.0 ** -11) * spread + tiny
        e_lse[:, h] = delta + 2.0 ** -23 * lse[:, h].abs().nan_to_num(posinf=0.0)
    e_out += (out.abs() + e_out) * 2.0 ** -8  # bf16
    return out, lse, e_out, e_lse
