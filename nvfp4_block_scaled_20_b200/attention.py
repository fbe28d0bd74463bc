"""Rotary positions, the 8-bit paged KV cache and attention over it.

Torch-facing helpers of nvfp4_rope, nvfp4_kv8_write, nvfp4_kv8_read and
nvfp4_kv8_attention (include/nvfp4.h): they check shapes and types, allocate
outputs and marshal pointers and streams.  Work goes to the current stream of
the tensors' device, or to ``stream``.  What a call allocates itself belongs to
the stream it works on (an output may be dropped while the caller's current stream
still reads it); tensors that it is given are ordered by the caller, as for any
other work on two streams.

What is wrong in device values (lengths, rows, pages that do not fit) shows in the
workspace's error word, nvfp4_get_device_error / device_error(ws), and nowhere
else: such sequences are skipped.  A call without ``ws`` takes a workspace that it
drops, and its error word with it.  Rows of no sequence, and of skipped ones, are
left as they are; in outputs that the call allocates they hold anything.

These calls are made once per layer and token, so the host side is kept short:
the C structs are packed with ``struct`` (the formats below) instead of being
built field by field.
"""
from __future__ import annotations

import math
import struct
from dataclasses import dataclass

from . import NVFP4_BF16, NVFP4_F32, capi, workspace

torch = None  # from the first call on: the package can be imported without it

_ROPE_TENSOR = "PPqqqqq"                        # nvfp4_rope_tensor
_ROPE_PARAMS = struct.Struct("@5id3i4x")        # nvfp4_rope_params
_BATCH = struct.Struct("@Pqi4xPPi4xqi4x")       # nvfp4_kv8_batch
_QUERY = struct.Struct("@PPPi4xqqqqfiii")       # nvfp4_kv8_query
_ROPE_TENSORS = [struct.Struct("@" + _ROPE_TENSOR * n) for n in range(9)]


def _need_torch():
    global torch
    import torch


@dataclass(frozen=True)
class KV8Cache:
    """A paged KV cache in E4M3: codes uint8 [pages, heads, page_tokens,
    head_dim], one fp32 power-of-two scale per page and head [pages, heads].
    Its tensors stay the ones that it was made of and keep their memory (no set_,
    resize_ or .data on them).  A copy (copy.deepcopy, pickle) has its own."""
    k_codes: object
    v_codes: object
    k_scales: object
    v_scales: object

    def __post_init__(self):
        torch is None and _need_torch()
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
        vars(self).update(
            heads=k.shape[1], page_tokens=k.shape[2], head_dim=k.shape[3], device=k.device,
            index=k.get_device(), desc=bytes(capi.nvfp4_kv8_cache(
                k.data_ptr(), self.v_codes.data_ptr(), self.k_scales.data_ptr(),
                self.v_scales.data_ptr(), *k.shape)))

    def __reduce__(self):
        # a copied or unpickled cache is made of its own tensors, and not given the
        # addresses of this one's
        return type(self), (self.k_codes, self.v_codes, self.k_scales, self.v_scales)


def kv8_cache(pages, heads, page_tokens=64, head_dim=128, device=None):
    """An empty cache: zero codes, smallest scales."""
    torch is None and _need_torch()
    device = device or "cuda"

    def codes():
        return torch.zeros((pages, heads, page_tokens, head_dim), dtype=torch.uint8, device=device)

    def scales():
        return torch.full((pages, heads), 2.0 ** -40, dtype=torch.float32, device=device)

    return KV8Cache(codes(), codes(), scales(), scales())


def _type(kind):
    if kind is torch.bfloat16:
        return NVFP4_BF16
    if kind is torch.float32:
        return NVFP4_F32
    raise TypeError("unsupported dtype %s" % kind)


def _on(stream, index, given, call, *args):
    """call(*args) with `stream` current: the workspace and the outputs that it
    allocates then belong to that stream -- their first use is ordered after
    whatever had the memory before, and so is what gets it next.  Outputs that
    were not `given` are noted as in use by the caller's stream too, which has yet
    to read them when they are dropped."""
    torch is None and _need_torch()
    if stream.device.index != index:
        raise ValueError("the stream is of another device than the tensors")
    caller = torch.cuda.current_stream(index)
    with torch.cuda.stream(stream):
        outs = call(*args)
    if not given:
        for t in outs if isinstance(outs, (list, tuple)) else (outs,):
            t.record_stream(caller)
    return outs


def _call(fn, index, *args):
    """fn, a call of capi, with device `index`'s current stream as the last
    argument and with that device current."""
    if index < 0:
        raise ValueError("%s works on CUDA tensors" % fn.__name__)
    handle = torch._C._cuda_getCurrentRawStream(index)
    if torch._C._cuda_getDevice() == index:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            st = fn(*args, handle)
    if st:
        raise capi.NVFP4Error(fn.__name__, st)


def _packed(x, rows, cache, what):
    """Heads and strides of a [rows, heads, head_dim] tensor of the cache's device."""
    shape = x.shape
    if len(shape) != 3 or shape[0] != rows or shape[2] != cache.head_dim:
        raise ValueError("%s is [%d, heads, %d], not %s" % (what, rows, cache.head_dim,
                                                            tuple(shape)))
    if x.get_device() != cache.index:
        raise ValueError("%s is not on the cache's device" % what)
    t, h, e = x.stride()
    if e != 1:
        raise ValueError("%s: the elements of a head are not contiguous" % what)
    return shape[1], t, h


def _rows_of_cache(k, v, rows, cache):
    """Strides of k and v, which have the cache's heads and one type."""
    nk, kt, kh = _packed(k, rows, cache, "k")
    nv, vt, vh = _packed(v, rows, cache, "v")
    if nk != cache.heads or nv != nk or v.dtype is not k.dtype:
        raise ValueError("k and v have the cache's heads and one type")
    return kt, kh, vt, vh


def _workspace(ws, cache):
    if ws.get_device() != cache.index or not ws.is_contiguous():
        raise ValueError("the workspace is contiguous and on the cache's device")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _batch(cache, page_table, lens, starts, rows, max_rows):
    i32 = torch.int32
    if not (page_table.dtype is i32 and lens.dtype is i32 and starts.dtype is i32):
        raise TypeError("page_table, lens and starts are int32 tensors")
    at = cache.index
    if page_table.get_device() != at or lens.get_device() != at or starts.get_device() != at:
        raise ValueError("page_table, lens and starts are on the cache's device")
    shape = page_table.shape
    if len(shape) != 2 or lens.shape != shape[:1] or starts.dim() != 1 or (
            starts.numel() != shape[0] + 1):
        raise ValueError("page_table is [n, pages], lens [n], starts [n + 1]")
    n, width = shape
    stride, one = page_table.stride()
    if stride < width and n > 1:
        raise ValueError("page_table's rows overlap")
    if (one != 1 and width > 1) or not lens.is_contiguous() or not starts.is_contiguous():
        raise ValueError("page_table's rows, lens and starts are contiguous")
    return _BATCH.pack(page_table.data_ptr(), stride if n > 1 else width, width,
                       lens.data_ptr(), starts.data_ptr(), n, rows, max_rows)


def rope(xs, positions, sections, theta=10000.0, interleaved=True, per_axis=True, inverse=False,
         outs=None, stream=None):
    """One nvfp4_rope call: every tensor of xs ([tokens, heads, head_dim], of one
    type, strided) turned by positions (int32 [tokens, axes]).  With ``inverse``
    the gradients of xs from those of the outputs.  outs may be xs (in place)."""
    if stream is not None:
        return _on(stream, positions.get_device(), outs is not None, rope, xs, positions, sections,
                   theta, interleaved, per_axis, inverse, outs)
    torch is None and _need_torch()
    n, axes = len(xs), len(sections)
    if not 1 <= n <= 8 or not 1 <= axes <= 4:
        raise ValueError("rope takes 1 to 8 tensors and 1 to 4 sections")
    given = outs is not None
    if not given:
        outs = [torch.empty_like(x, memory_format=torch.contiguous_format) for x in xs]
    elif len(outs) != n:
        raise ValueError("rope has one output per tensor")
    first, places = xs[0], positions.shape
    if first.dim() != 3:
        raise ValueError("rope's tensors are [tokens, heads, head_dim]")
    tokens, _, dim = first.shape
    at, kind = positions.get_device(), first.dtype
    if positions.dtype is not torch.int32 or len(places) != 2 or places[0] != tokens or (
            places[1] < axes):
        raise ValueError("positions is int32 [tokens, axes]")
    stride, one = positions.stride()
    if one != 1 and places[1] > 1:
        raise ValueError("positions' rows are contiguous")
    if tokens < 2:
        stride = axes
    elif stride < axes:
        raise ValueError("positions' rows overlap")
    fields = []
    for x, o in zip(xs, outs):
        shape = x.shape
        if len(shape) != 3 or shape[0] != tokens or shape[2] != dim:
            raise ValueError("rope's tensors are [tokens, heads, head_dim] of one token count")
        if x.dtype is not kind or x.get_device() != at:
            raise ValueError("rope's tensors are of one type and device")
        heads = shape[1]
        xt, xh, xe = x.stride()
        ot, oh, oe = heads * dim, dim, 1
        if given:
            if o.shape != shape:
                raise ValueError("rope's tensors are [tokens, heads, head_dim] of one token count")
            if o.dtype is not kind or o.get_device() != at:
                raise ValueError("rope's tensors are of one type and device")
            ot, oh, oe = o.stride()
        if (xe != 1 or oe != 1) and dim > 1:
            raise ValueError("rope: the elements of a head are not contiguous")
        fields += (x.data_ptr(), o.data_ptr(), heads, xt, xh, ot, oh)
    pad = (0, 0, 0, 0)
    rp = _ROPE_PARAMS.pack(axes, *sections, *pad[axes:], theta, bool(interleaved), bool(per_axis),
                           bool(inverse))
    _call(capi.nvfp4_rope, at, _ROPE_TENSORS[n].pack(*fields), n, _type(kind), tokens, dim,
          positions.data_ptr(), stride, rp)
    return outs


def kv8_write(cache, k, v, page_table, lens, starts, max_new=None, ws=None, stream=None):
    """One nvfp4_kv8_write call: rows starts[s]..starts[s+1] of k and v ([rows,
    heads, head_dim]) become sequence s's tokens from lens[s] on.  max_new: at
    least the most rows of a sequence (default: all rows)."""
    if stream is not None:
        return _on(stream, cache.index, True, kv8_write, cache, k, v, page_table, lens, starts,
                   max_new, ws)
    torch is None and _need_torch()
    rows = k.shape[0]
    kt, kh, vt, vh = _rows_of_cache(k, v, rows, cache)
    b = _batch(cache, page_table, lens, starts, rows, rows if max_new is None else max_new)
    ws = workspace(0, cache.device) if ws is None else ws
    _call(capi.nvfp4_kv8_write, cache.index, cache.desc, b, _type(k.dtype), k.data_ptr(), kt, kh,
          v.data_ptr(), vt, vh, *_workspace(ws, cache))


def kv8_read(cache, page_table, begins, starts, rows, max_tokens=None, out_dtype=None, outs=None,
             ws=None, stream=None):
    """One nvfp4_kv8_read call: sequence s's tokens from begins[s] on become rows
    starts[s]..starts[s+1] of the returned (k, v), [rows, heads, head_dim]."""
    if stream is not None:
        return _on(stream, cache.index, outs is not None, kv8_read, cache, page_table, begins, starts,
                   rows, max_tokens, out_dtype, outs, ws)
    torch is None and _need_torch()
    if outs is None:
        kind = out_dtype or torch.bfloat16
        kh = vh = cache.head_dim
        kt = vt = cache.heads * kh
        k = torch.empty_strided((rows, cache.heads, kh), (kt, kh, 1), device=cache.device, dtype=kind)
        outs = k, v = k, torch.empty_like(k)
    else:
        k, v = outs
        kt, kh, vt, vh = _rows_of_cache(k, v, rows, cache)
    b = _batch(cache, page_table, begins, starts, rows, rows if max_tokens is None else max_tokens)
    ws = workspace(0, cache.device) if ws is None else ws
    _call(capi.nvfp4_kv8_read, cache.index, cache.desc, b, _type(k.dtype), k.data_ptr(), kt, kh,
          v.data_ptr(), vt, vh, *_workspace(ws, cache))
    return outs


def kv8_attention_workspace(cache, page_table, starts, q_heads, max_q):
    """Workspace for kv8_attention of these sizes, error word zeroed (the rest
    needs no initialization).  Serves one call in flight at a time."""
    torch is None and _need_torch()
    ws = torch.empty(capi.nvfp4_kv8_attention_workspace_bytes(
        cache.heads, cache.head_dim, cache.page_tokens, q_heads, starts.numel() - 1, max_q,
        page_table.shape[1]), dtype=torch.uint8, device=cache.device)
    ws[:capi.nvfp4_workspace_bytes(0)].zero_()
    return ws


def kv8_attention(q, cache, page_table, lens, starts, max_q=None, scale=None, causal=False,
                  window=-1, sink=0, out=None, lse=None, ws=None, stream=None):
    """One nvfp4_kv8_attention call: q bf16 [rows, q_heads, head_dim], sequence
    s's queries in rows starts[s]..starts[s+1], over its lens[s] cached tokens.
    max_q: at least the most queries of a sequence (default: all rows); it chooses
    the kernel for all of them, so prompts and single tokens are faster in calls of
    their own.  lse: an fp32 [rows, q_heads] tensor that receives the log-sum-exps."""
    if stream is not None:
        return _on(stream, cache.index, out is not None, kv8_attention, q, cache, page_table, lens,
                   starts, max_q, scale, causal, window, sink, out, lse, ws)
    torch is None and _need_torch()
    if q.dtype is not torch.bfloat16:
        raise TypeError("q and out are bfloat16")
    rows = q.shape[0]
    q_heads, qt, qh = _packed(q, rows, cache, "q")
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        ot, oh = q_heads * cache.head_dim, cache.head_dim
    elif out.dtype is not torch.bfloat16:
        raise TypeError("q and out are bfloat16")
    else:
        heads, ot, oh = _packed(out, rows, cache, "out")
        if heads != q_heads:
            raise ValueError("out has q's heads")
    at = 0
    if lse is not None:
        if lse.dtype is not torch.float32 or lse.shape != (rows, q_heads) or (
                not lse.is_contiguous() or lse.get_device() != cache.index):
            raise ValueError("lse is contiguous fp32 [rows, q_heads] on the cache's device")
        at = lse.data_ptr()
    if max_q is None:
        max_q = rows
    b = _batch(cache, page_table, lens, starts, rows, max_q)
    if ws is None:
        ws = kv8_attention_workspace(cache, page_table, starts, q_heads, max_q)
    if scale is None:
        scale = 1.0 / math.sqrt(cache.head_dim)
    query = _QUERY.pack(q.data_ptr(), out.data_ptr(), at, q_heads, qt, qh, ot, oh, scale,
                        bool(causal), window, sink)
    _call(capi.nvfp4_kv8_attention, cache.index, cache.desc, b, query, *_workspace(ws, cache))
    return out
