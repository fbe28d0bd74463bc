"""Rotary positions, the 8-bit paged KV cache and attention over it.

Torch-facing helpers of nvfp4_rope, nvfp4_kv8_write, nvfp4_kv8_read and
nvfp4_kv8_attention (include/nvfp4.h): they check shapes and types, allocate
outputs and marshal pointers and streams.  Work goes to the current stream of
the tensors' device, or to ``stream``.
"""
from __future__ import annotations

import math
from dataclasses import dataclass

from . import _dtype_code, _torch, capi, workspace


@dataclass
class KV8Cache:
    """A paged KV cache in E4M3: codes uint8 [pages, heads, page_tokens,
    head_dim], one fp32 power-of-two scale per page and head [pages, heads]."""
    k_codes: object
    v_codes: object
    k_scales: object
    v_scales: object

    def __post_init__(self):
        torch = _torch()
        k = self.k_codes
        if k.dim() != 4 or self.v_codes.shape != k.shape:
            raise ValueError("codes are [pages, heads, page_tokens, head_dim], K and V alike")
        for t in (k, self.v_codes):
            if t.dtype != torch.uint8 or not t.is_contiguous():
                raise ValueError("codes are contiguous uint8 tensors")
        for t in (self.k_scales, self.v_scales):
            if t.dtype != torch.float32 or not t.is_contiguous() or t.shape != k.shape[:2]:
                raise ValueError("scales are contiguous fp32 [pages, heads] tensors")
        if any(t.device != k.device for t in (self.v_codes, self.k_scales, self.v_scales)):
            raise ValueError("a cache lives on one device")
        self.desc = capi.nvfp4_kv8_cache(k.data_ptr(), self.v_codes.data_ptr(),
                                         self.k_scales.data_ptr(), self.v_scales.data_ptr(),
                                         k.shape[0], k.shape[1], k.shape[2], k.shape[3])

    @property
    def page_tokens(self):
        return self.k_codes.shape[2]


def kv8_cache(pages, heads, page_tokens=64, head_dim=128, device=None):
    """An empty cache: zero codes, smallest scales."""
    torch = _torch()
    device = device or "cuda"

    def codes():
        return torch.zeros((pages, heads, page_tokens, head_dim), dtype=torch.uint8, device=device)

    def scales():
        return torch.full((pages, heads), 2.0 ** -40, dtype=torch.float32, device=device)

    return KV8Cache(codes(), codes(), scales(), scales())


def _launch(device, stream, call):
    """call(stream handle) with `device` current."""
    torch = _torch()
    s = torch.cuda.current_stream(device) if stream is None else stream
    if device.index in (None, torch.cuda.current_device()):
        return call(s.cuda_stream)
    with torch.cuda.device(device):
        return call(s.cuda_stream)


def _packed(x, heads, dim, what):
    if x.dim() != 3 or x.shape[1] != heads or x.shape[2] != dim:
        raise ValueError("%s is [rows, %d, %d], not %s" % (what, heads, dim, tuple(x.shape)))
    if x.stride(2) != 1:
        raise ValueError("%s: the elements of a head are not contiguous" % what)
    return x


def _batch(cache, page_table, lens, starts, rows, max_rows):
    torch = _torch()
    i32, dev = torch.int32, cache.k_codes.device
    if page_table.dtype != i32 or lens.dtype != i32 or starts.dtype != i32:
        raise TypeError("page_table, lens and starts are int32 tensors")
    if page_table.device != dev or lens.device != dev or starts.device != dev:
        raise ValueError("page_table, lens and starts are on the cache's device")
    n = lens.shape[0]
    if page_table.dim() != 2 or page_table.shape[0] != n or starts.shape != (n + 1,):
        raise ValueError("page_table is [n, pages], lens [n], starts [n + 1]")
    if page_table.stride(1) != 1 and page_table.shape[1] > 1 or not (
            lens.is_contiguous() and starts.is_contiguous()):
        raise ValueError("page_table's rows, lens and starts are contiguous")
    return capi.nvfp4_kv8_batch(page_table.data_ptr(), max(page_table.stride(0), page_table.shape[1]),
                                page_table.shape[1], lens.data_ptr(), starts.data_ptr(), n, rows,
                                rows if max_rows is None else max_rows)


def rope(xs, positions, sections, theta=10000.0, interleaved=True, per_axis=True, inverse=False,
         outs=None, stream=None):
    """One nvfp4_rope call: every tensor of xs ([tokens, heads, head_dim], of one
    type, strided) turned by positions (int32 [tokens, axes]).  With ``inverse``
    the gradients of xs from those of the outputs.  outs may be xs (in place)."""
    torch = _torch()
    n = len(xs)
    axes = len(sections)
    if n < 1 or not 1 <= axes <= 4:
        raise ValueError("rope takes at least one tensor and 1 to 4 sections")
    tokens, _, dim = xs[0].shape
    if positions.dtype != torch.int32 or positions.dim() != 2 or positions.shape[0] != tokens or (
            positions.shape[1] < axes):
        raise ValueError("positions is int32 [tokens, axes]")
    if positions.stride(1) != 1 and positions.shape[1] > 1:
        raise ValueError("positions' rows are contiguous")
    if outs is None:
        outs = [torch.empty(x.shape, dtype=x.dtype, device=x.device) for x in xs]
    descs = (capi.nvfp4_rope_tensor * n)()
    for i, (x, o) in enumerate(zip(xs, outs)):
        if x.dim() != 3 or x.shape[0] != tokens or x.shape[2] != dim or o.shape != x.shape:
            raise ValueError("rope's tensors are [tokens, heads, head_dim] of one token count")
        if x.dtype != xs[0].dtype or o.dtype != x.dtype or x.device != positions.device:
            raise ValueError("rope's tensors are of one type and device")
        xt, xh, xe = x.stride()
        ot, oh, oe = o.stride()
        if xe != 1 or oe != 1:
            raise ValueError("rope: the elements of a head are not contiguous")
        descs[i] = capi.nvfp4_rope_tensor(x.data_ptr(), o.data_ptr(), x.shape[1], xt, xh, ot, oh)
    rp = capi.nvfp4_rope_params(axes, tuple(sections), theta, bool(interleaved), bool(per_axis),
                                bool(inverse))
    st = _launch(positions.device, stream, lambda s: capi.nvfp4_rope(
        descs, n, _dtype_code(xs[0]), tokens, dim, positions.data_ptr(),
        max(positions.stride(0), positions.shape[1]), rp, s))
    capi.check("nvfp4_rope", st)
    return outs


def kv8_write(cache, k, v, page_table, lens, starts, max_new=None, ws=None, stream=None):
    """One nvfp4_kv8_write call: rows starts[s]..starts[s+1] of k and v ([rows,
    heads, head_dim]) become sequence s's tokens from lens[s] on.  max_new: at
    least the most rows of a sequence (default: all rows)."""
    _, heads, _, dim = cache.k_codes.shape
    _packed(k, heads, dim, "k")
    _packed(v, heads, dim, "v")
    if v.shape[0] != k.shape[0] or v.dtype != k.dtype:
        raise ValueError("k and v have the same rows and type")
    if k.device != cache.k_codes.device or v.device != k.device:
        raise ValueError("k and v are on the cache's device")
    ws = workspace(0, k.device) if ws is None else ws
    b = _batch(cache, page_table, lens, starts, k.shape[0], max_new)
    st = _launch(k.device, stream, lambda s: capi.nvfp4_kv8_write(
        cache.desc, b, _dtype_code(k), k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(),
        v.stride(0), v.stride(1), ws.data_ptr(), ws.numel(), s))
    capi.check("nvfp4_kv8_write", st)


def kv8_read(cache, page_table, begins, starts, rows, max_tokens=None, out_dtype=None, outs=None,
             ws=None, stream=None):
    """One nvfp4_kv8_read call: sequence s's tokens from begins[s] on become rows
    starts[s]..starts[s+1] of the returned (k, v), [rows, heads, head_dim]."""
    torch = _torch()
    _, heads, _, dim = cache.k_codes.shape
    dev = cache.k_codes.device
    if outs is None:
        out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
        outs = tuple(torch.empty((rows, heads, dim), dtype=out_dtype, device=dev) for _ in "kv")
    k, v = outs
    _packed(k, heads, dim, "k")
    _packed(v, heads, dim, "v")
    if k.shape[0] != rows or v.shape[0] != rows or v.dtype != k.dtype:
        raise ValueError("the outputs have `rows` rows and one type")
    if k.device != dev or v.device != dev:
        raise ValueError("the outputs are on the cache's device")
    ws = workspace(0, dev) if ws is None else ws
    b = _batch(cache, page_table, begins, starts, rows, max_tokens)
    st = _launch(dev, stream, lambda s: capi.nvfp4_kv8_read(
        cache.desc, b, _dtype_code(k), k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(),
        v.stride(0), v.stride(1), ws.data_ptr(), ws.numel(), s))
    capi.check("nvfp4_kv8_read", st)
    return outs


def kv8_attention_workspace(cache, page_table, starts, q_heads, max_q):
    """Workspace for kv8_attention of these sizes, error word zeroed (the rest
    needs no initialization).  Serves one call in flight at a time."""
    torch = _torch()
    _, heads, page_tokens, dim = cache.k_codes.shape
    ws = torch.empty(capi.nvfp4_kv8_attention_workspace_bytes(
        heads, dim, page_tokens, q_heads, starts.shape[0] - 1, max_q, page_table.shape[1]),
        dtype=torch.uint8, device=cache.k_codes.device)
    ws[:capi.nvfp4_workspace_bytes(0)].zero_()
    return ws


def kv8_attention(q, cache, page_table, lens, starts, max_q=None, scale=None, causal=False,
                  window=-1, sink=0, out=None, lse=None, ws=None, stream=None):
    """One nvfp4_kv8_attention call: q bf16 [rows, q_heads, head_dim], sequence
    s's queries in rows starts[s]..starts[s+1], over its lens[s] cached tokens.
    max_q: at least the most queries of a sequence (default: all rows).  lse: an
    fp32 [rows, q_heads] tensor that receives the log-sum-exps."""
    torch = _torch()
    _, heads, page_tokens, dim = cache.k_codes.shape
    rows, q_heads = q.shape[0], q.shape[1]
    _packed(q, q_heads, dim, "q")
    if out is None:
        out = torch.empty((rows, q_heads, dim), dtype=q.dtype, device=q.device)
    _packed(out, q_heads, dim, "out")
    if q.dtype != torch.bfloat16 or out.dtype != q.dtype:
        raise TypeError("q and out are bfloat16")
    if out.shape[0] != rows:
        raise ValueError("out has q's rows")
    dev = cache.k_codes.device
    if q.device != dev or out.device != dev or (lse is not None and lse.device != dev):
        raise ValueError("q, out and lse are on the cache's device")
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != (rows, q_heads)
                            or not lse.is_contiguous()):
        raise ValueError("lse is contiguous fp32 [rows, q_heads]")
    b = _batch(cache, page_table, lens, starts, rows, max_q)
    if ws is None:
        ws = kv8_attention_workspace(cache, page_table, starts, q_heads, b.max_rows)
    query = capi.nvfp4_kv8_query(q.data_ptr(), out.data_ptr(),
                                 None if lse is None else lse.data_ptr(), q_heads, q.stride(0),
                                 q.stride(1), out.stride(0), out.stride(1),
                                 1.0 / math.sqrt(dim) if scale is None else scale, bool(causal),
                                 window, sink)
    st = _launch(dev, stream, lambda s: capi.nvfp4_kv8_attention(
        cache.desc, b, query, ws.data_ptr(), ws.numel(), s))
    capi.check("nvfp4_kv8_attention", st)
    return out
