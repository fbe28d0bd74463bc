"""Refusals of the attention-side calls (rotary positions, the 8-bit cache,
attention over it): every call here ends in host-side validation, before any
CUDA work.  And the plain forms that the GPU tests compare with, against
something other than themselves."""
import math

import pytest
import torch

import attention_ref as ref
from nvfp4_block_scaled_20_b200 import build, capi

A = 1 << 20  # a fake, well-aligned address: never dereferenced
OK, INVALID, SHAPE, ALIGN, WORKSPACE = 0, 1, 2, 3, 4


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return capi.load()


def _rope(x=A, out=A, heads=24, strides=(128 * 24, 128, 128 * 24, 128), dtype=1, tokens=4, dim=128,
          pos=A, pos_stride=3, axes=3, sections=(22, 21, 21), theta=1e4, n=1):
    t = (capi.nvfp4_rope_tensor * max(n, 1))()
    for i in range(n):
        t[i] = capi.nvfp4_rope_tensor(x, out, heads, *strides)
    rp = capi.nvfp4_rope_params(axes, tuple(sections), theta, 1, 1, 0)
    return capi.nvfp4_rope(t, n, dtype, tokens, dim, pos, pos_stride, rp, None)


def test_rope_refusals():
    assert _rope(x=None) == INVALID and _rope(out=None) == INVALID and _rope(pos=None) == INVALID
    assert _rope(dtype=2) == INVALID and _rope(axes=0) == INVALID and _rope(axes=5) == INVALID
    assert _rope(theta=0.0) == INVALID and _rope(theta=math.inf) == INVALID
    assert _rope(theta=math.nan) == INVALID
    assert _rope(dim=127) == SHAPE and _rope(dim=514) == SHAPE and _rope(tokens=-1) == SHAPE
    assert _rope(sections=(33, 21, 21)) == SHAPE and _rope(sections=(-1, 21, 21)) == SHAPE
    assert _rope(pos_stride=2) == SHAPE and _rope(n=9) == SHAPE and _rope(heads=-1) == SHAPE
    assert _rope(strides=(-2, 128, 2, 128)) == SHAPE
    assert _rope(strides=(128 * 24 + 1, 128, 128 * 24, 128)) == ALIGN
    assert _rope(x=A + 2) == ALIGN and _rope(out=A + 2) == ALIGN and _rope(pos=A + 2) == ALIGN
    assert _rope(x=A + 4, dtype=0) == ALIGN
    # nothing to do
    assert _rope(tokens=0, x=None, pos=None) == OK
    assert _rope(heads=0, x=None) == OK and _rope(n=0) == OK


def _cache(**kw):
    d = dict(k_codes=A, v_codes=A, k_scales=A, v_scales=A, pages=10, heads=8, page_tokens=64,
             head_dim=128)
    d.update(kw)
    return capi.nvfp4_kv8_cache(**d)


def _batch(**kw):
    d = dict(page_table=A, table_stride=4, table_pages=4, lens=A, starts=A, n=2, rows=6, max_rows=3)
    d.update(kw)
    return capi.nvfp4_kv8_batch(**d)


BAD_CACHES = [(dict(k_codes=None), INVALID), (dict(v_scales=None), INVALID),
              (dict(head_dim=96), SHAPE), (dict(page_tokens=16), SHAPE),
              (dict(page_tokens=256), SHAPE), (dict(heads=0), SHAPE), (dict(heads=40000), SHAPE),
              (dict(pages=0), SHAPE), (dict(k_codes=A + 8), ALIGN), (dict(k_scales=A + 2), ALIGN)]
BAD_BATCHES = [(dict(page_table=None), INVALID), (dict(lens=None), INVALID),
               (dict(starts=None), INVALID), (dict(n=-1), SHAPE), (dict(n=70000), SHAPE),
               (dict(rows=-1), SHAPE), (dict(max_rows=-1), SHAPE), (dict(table_pages=0), SHAPE),
               (dict(table_stride=3), SHAPE), (dict(max_rows=(1 << 30) + 1), SHAPE),
               (dict(table_pages=1 << 25, table_stride=1 << 25), SHAPE), (dict(lens=A + 1), ALIGN)]


@pytest.mark.parametrize("call", ["write", "read"])
def test_cache_refusals(call):
    fn = capi.nvfp4_kv8_write if call == "write" else capi.nvfp4_kv8_read
    ws = capi.nvfp4_workspace_bytes(0)

    def go(cache=None, batch=None, dtype=1, k=A, strides=(1024, 128, 1024, 128), v=A, w=A, wb=ws):
        return fn(cache or _cache(), batch or _batch(), dtype, k, strides[0], strides[1], v,
                  strides[2], strides[3], w, wb, None)

    for kw, want in BAD_CACHES:
        assert go(cache=_cache(**kw)) == want, kw
    for kw, want in BAD_BATCHES:
        assert go(batch=_batch(**kw)) == want, kw
    assert go(dtype=3) == INVALID and go(k=None) == INVALID and go(v=None) == INVALID
    assert go(k=A + 8) == ALIGN and go(strides=(1028, 128, 1024, 128)) == ALIGN
    assert go(strides=(1024, -128, 1024, 128)) == SHAPE
    assert go(w=None) == WORKSPACE and go(wb=ws - 1) == WORKSPACE
    for kw in (dict(n=0), dict(rows=0), dict(max_rows=0)):
        assert go(batch=_batch(**kw), k=None) == OK


def test_attention_refusals():
    need = capi.nvfp4_kv8_attention_workspace_bytes(8, 128, 64, 24, 2, 3, 4)

    def go(cache=None, batch=None, w=A, wb=need, **kw):
        d = dict(q=A, out=A, lse=None, q_heads=24, q_token_stride=24 * 128, q_head_stride=128,
                 out_token_stride=24 * 128, out_head_stride=128, scale=0.1, causal=1, window=-1,
                 sink=0)
        d.update(kw)
        return capi.nvfp4_kv8_attention(cache or _cache(), batch or _batch(),
                                        capi.nvfp4_kv8_query(**d), w, wb, None)

    for kw, want in BAD_CACHES:
        assert go(cache=_cache(**kw)) == want, kw
    for kw, want in BAD_BATCHES:
        assert go(batch=_batch(**kw)) == want, kw
    for s in (0.0, -1.0, math.inf, math.nan):
        assert go(scale=s) == INVALID
    assert go(causal=2) == INVALID and go(window=-2) == INVALID and go(sink=-1) == INVALID
    assert go(q=None) == INVALID and go(out=None) == INVALID
    assert go(q_heads=20) == SHAPE and go(q_heads=4) == SHAPE and go(q_token_stride=-8) == SHAPE
    assert go(q=A + 8) == ALIGN and go(out=A + 2) == ALIGN and go(lse=A + 2) == ALIGN
    assert go(q_head_stride=132) == ALIGN and go(w=A + 8) == ALIGN
    assert go(w=None) == WORKSPACE and go(wb=need - 1) == WORKSPACE
    assert go(batch=_batch(n=0), q=None) == OK
    # too many tiles of query rows
    assert go(batch=_batch(n=60000, max_rows=1 << 29, rows=1 << 40)) == SHAPE


def test_python_refusals():
    import nvfp4_block_scaled_20_b200 as nv
    with pytest.raises(ValueError):
        nv.KV8Cache(torch.zeros(2, 3, 64, 128), torch.zeros(2, 3, 64, 128), torch.ones(2, 3),
                    torch.ones(2, 3))
    c = nv.kv8_cache(4, 2, 32, 64, device="cpu")
    t = torch.zeros((1, 2), dtype=torch.int32)
    one, two = torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    k = torch.zeros(3, 2, 64)
    with pytest.raises(ValueError):
        nv.kv8_write(c, k[:, :1], k, t, one, two, ws=one)
    with pytest.raises(ValueError):
        nv.kv8_write(c, k, k.bfloat16(), t, one, two, ws=one)
    with pytest.raises(TypeError):
        nv.kv8_write(c, k, k, t.long(), one, two, ws=one)
    with pytest.raises(ValueError):
        nv.kv8_write(c, k, k, t, one, one, ws=one)
    with pytest.raises(TypeError):
        nv.kv8_attention(k, c, t, one, two, ws=one)
    with pytest.raises(ValueError):
        nv.rope([k], torch.zeros(3, 2, dtype=torch.int64), [4, 4])
    with pytest.raises(ValueError):
        nv.rope([k, k[:2]], torch.zeros(3, 2, dtype=torch.int32), [4, 4])


def test_workspace_grows_with_the_split():
    base = capi.nvfp4_workspace_bytes(0)
    f = capi.nvfp4_kv8_attention_workspace_bytes
    assert f(8, 128, 64, 8, 1, 1, 1) >= base
    assert f(8, 128, 64, 8, 1, 1, 512) > f(8, 128, 64, 8, 1, 1, 8) > base


def test_workspace_of_sizes_that_a_call_refuses():
    base = capi.nvfp4_workspace_bytes(0)
    f = capi.nvfp4_kv8_attention_workspace_bytes
    for bad in ((0, 128, 64, 8, 1, 1, 4), (8, 256, 64, 8, 1, 1, 4), (8, 0, 64, 8, 1, 1, 4),
                (8, 96, 64, 8, 1, 1, 4), (8, 128, 0, 8, 1, 1, 4), (8, 128, 64, 12, 1, 1, 4),
                (8, 128, 64, 8, 0, 1, 4), (8, 128, 64, 8, 1, 1, 0), (32767, 64, 64, 32767, 1, 33, 4)):
        assert f(*bad) == base, bad
    # more tiles and heads than a grid dimension holds
    need = 1 << 30
    query = dict(q=A, out=A, lse=None, q_heads=32767, q_token_stride=32767 * 64, q_head_stride=64,
                 out_token_stride=32767 * 64, out_head_stride=64, scale=0.1, causal=1, window=-1,
                 sink=0)
    assert capi.nvfp4_kv8_attention(_cache(heads=32767, head_dim=64), _batch(max_rows=33, rows=66),
                                    capi.nvfp4_kv8_query(**query), A, need, None) == SHAPE


def test_python_refuses_rows_that_overlap_and_workspaces_elsewhere():
    import nvfp4_block_scaled_20_b200 as nv
    c = nv.kv8_cache(4, 2, 32, 64, device="cpu")
    lens, starts = torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    k = torch.zeros(3, 2, 64)
    t = torch.zeros((1, 2), dtype=torch.int32).expand(2, 2)
    with pytest.raises(ValueError, match="overlap"):
        nv.kv8_write(c, k, k, t, lens, starts, ws=starts)
    with pytest.raises(ValueError, match="overlap"):
        nv.kv8_attention(k.bfloat16(), c, t, lens, starts, ws=starts)
    with pytest.raises(ValueError, match="overlap"):
        nv.rope([k], torch.zeros((1, 2), dtype=torch.int32).expand(3, 2), [4, 4])
    with pytest.raises(ValueError, match="one output"):
        nv.rope([k], torch.zeros((3, 2), dtype=torch.int32), [4, 4], outs=[k, k])
    with pytest.raises(ValueError, match="workspace"):
        nv.kv8_write(c, k, k, t.contiguous(), lens, starts,
                     ws=torch.zeros((8, 8), dtype=torch.uint8).t())
    with pytest.raises(AttributeError):
        c.k_codes = c.v_codes


# ------------------------------------------------------- the plain forms
def test_plain_e4m3_is_the_nearest_value():
    grid = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    y = torch.cat([torch.rand(2000, dtype=torch.float64) * 500, torch.rand(2000).double() * 0.05,
                   (grid[1:] + grid[:-1]) / 2, grid])
    d = (y[:, None] - grid).abs()
    near = d == d.amin(1, keepdim=True)
    even = torch.arange(127) % 2 == 0
    best = torch.where(near.sum(1) > 1, (near & even).double().argmax(1), near.double().argmax(1))
    assert torch.equal(ref.e4m3(y), grid[best])
    assert torch.equal(ref.e4m3(-y), -grid[best])


def test_plain_rope_keeps_lengths_and_inverts():
    x = torch.randn(5, 2, 16, dtype=torch.float64)
    pos = torch.randint(-50, 5000, (5, 3), dtype=torch.int32)
    for inter in (True, False):
        y = ref.rope(x, pos, [3, 2, 2], 1e4, inter, True, False)
        assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1))
        assert torch.allclose(ref.rope(y, pos, [3, 2, 2], 1e4, inter, True, True), x)
        assert torch.equal(y[..., 14:], x[..., 14:])


def test_plain_attention_against_softmax():
    q, k, v = (torch.randn(n, 2, 8, dtype=torch.float64) for n in (3, 9, 9))
    ok = ref.seen(3, 9, True, 4, 1, "cpu")
    assert ok[0].tolist() == [True, False, True, True, True, True, True, False, False]
    out, lse, _, _ = ref.attention(q, k, v, v.abs(), torch.ones(1, 2).double(), 0.3, ok)
    for h in range(2):
        s = (q[:, h] @ k[:, h].T * 0.3).masked_fill(~ok, -math.inf)
        assert torch.allclose(out[:, h], torch.softmax(s, -1) @ v[:, h])
        assert torch.allclose(lse[:, h], torch.logsumexp(s, -1))


@pytest.mark.parametrize("how", ["deepcopy", "pickle", "save", "copy", "replace"])
def test_a_copied_cache_names_its_own_memory(how):
    import copy
    import dataclasses
    import io
    import pickle
    import nvfp4_block_scaled_20_b200 as nv
    c = nv.kv8_cache(4, 2, 32, 64, device="cpu")
    c.k_codes.random_(0, 120)
    if how == "deepcopy":
        d = copy.deepcopy([c])[0]
    elif how == "pickle":
        d = pickle.loads(pickle.dumps(c))
    elif how == "save":
        f = io.BytesIO()
        torch.save(dict(cache=c), f)
        f.seek(0)
        d = torch.load(f, weights_only=False)["cache"]
    elif how == "copy":
        d = copy.copy(c)
    else:
        d = dataclasses.replace(c, k_codes=c.k_codes.clone())
    names = ("k_codes", "v_codes", "k_scales", "v_scales")
    at = capi.nvfp4_kv8_cache.from_buffer_copy(d.desc)
    for n in names:
        assert getattr(at, n) == getattr(d, n).data_ptr()
        assert torch.equal(getattr(d, n), getattr(c, n))
    own = [n for n in names if getattr(d, n).data_ptr() != getattr(c, n).data_ptr()]
    assert own == {"copy": [], "replace": ["k_codes"]}.get(how, list(names))
    assert (at.pages, at.heads, at.page_tokens, at.head_dim) == (4, 2, 32, 64)
    assert (d.heads, d.page_tokens, d.head_dim, d.index) == (2, 32, 64, -1)


def test_a_stream_of_another_device_is_refused():
    import nvfp4_block_scaled_20_b200 as nv

    class Stream:
        device, cuda_stream = torch.device("cuda", 3), 0

    c = nv.kv8_cache(4, 2, 32, 64, device="cpu")
    k, one = torch.zeros(3, 2, 64), torch.zeros(1, dtype=torch.int32)
    t, starts = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: nv.kv8_write(c, k, k, t, one, starts, ws=one, stream=Stream()),
                 lambda: nv.kv8_read(c, t, one, starts, 3, stream=Stream()),
                 lambda: nv.kv8_attention(k.bfloat16(), c, t, one, starts, ws=one, stream=Stream()),
                 lambda: nv.rope([k], torch.zeros((3, 1), dtype=torch.int32), [4], stream=Stream())):
        with pytest.raises(ValueError, match="another device"):
            call()


@pytest.mark.parametrize("call", ["write", "read"])
def test_cache_calls_refuse_a_misaligned_workspace(call):
    """The error word is written by an atomic of four bytes."""
    fn = capi.nvfp4_kv8_write if call == "write" else capi.nvfp4_kv8_read
    for shift in (1, 2, 3):
        assert fn(_cache(), _batch(), 1, A, 1024, 128, A, 1024, 128, A + shift,
                  capi.nvfp4_workspace_bytes(0), None) == ALIGN


OVERLAPS = [(0, 128), (1024, 0), (1024, 120), (1000, 128), (896, 128), (128, 128), (136, 128)]
APART = [(1024, 128), (2048, 128), (128, 6 * 128), (256, 16 * 128), (1032, 128)]


def test_outputs_whose_rows_overlap_are_refused():
    """[6 rows, 8 heads, 128]: token and head strides.  The next check refuses the
    calls whose rows lie apart: no call here reaches a launch."""
    ws = capi.nvfp4_workspace_bytes(0)

    def read(strides):
        return capi.nvfp4_kv8_read(_cache(), _batch(), 1, A, *strides[:2], 2 * A, *strides[2:], None,
                                   ws, None)

    def attend(strides):
        d = dict(q=A, out=2 * A, lse=None, q_heads=8, q_token_stride=0, q_head_stride=0,
                 out_token_stride=strides[0], out_head_stride=strides[1], scale=0.1, causal=1,
                 window=-1, sink=0)
        return capi.nvfp4_kv8_attention(_cache(), _batch(), capi.nvfp4_kv8_query(**d), None, ws, None)

    def rope(strides, **kw):
        return _rope(out=2 * A, heads=8, tokens=6, strides=(0, 0, *strides), pos=None, **kw)

    good = (1024, 128)
    for bad in OVERLAPS:
        assert read(good + bad) == SHAPE and read(bad + good) == SHAPE, bad
        assert attend(bad) == SHAPE and rope(bad) == SHAPE, bad
    for ok in APART:  # no workspace, no positions
        assert read(ok + good) == WORKSPACE and read(good + ok) == WORKSPACE, ok
        assert attend(ok) == WORKSPACE and rope(ok) == INVALID, ok
    # one tensor for both (the size of the launch would be refused next)
    many = dict(cache=_cache(heads=32767), batch=_batch(max_rows=1 << 30))
    wide = (32767 * 128, 128)
    for v, want in ((A, INVALID), (2 * A, SHAPE)):
        assert capi.nvfp4_kv8_read(many["cache"], many["batch"], 1, A, *wide, v, *wide, A, ws,
                                   None) == want
    # in place of q, but at other strides
    same = dict(q=A, out=A, lse=None, q_heads=8, out_token_stride=1024, out_head_stride=128, scale=0.1,
                causal=1, window=-1, sink=0)
    for tq, hq, want in ((1024, 128, WORKSPACE), (2048, 128, INVALID), (1024, 256, INVALID)):
        query = capi.nvfp4_kv8_query(q_token_stride=tq, q_head_stride=hq, **same)
        assert capi.nvfp4_kv8_attention(_cache(), _batch(), query, None, ws, None) == want
    # one token, one head: a stride that is not used may be anything
    assert _rope(out=2 * A, heads=8, tokens=1, strides=(0, 0, 0, 128), pos=None) == INVALID
    assert _rope(out=2 * A, heads=1, tokens=6, strides=(0, 0, 128, 0), pos=None) == INVALID


def test_rope_refuses_outputs_in_the_place_of_other_tensors():
    def go(*tensors):  # (x, out, token stride of x)
        t = (capi.nvfp4_rope_tensor * len(tensors))()
        for i, (x, out, xt) in enumerate(tensors):
            t[i] = capi.nvfp4_rope_tensor(x, out, 8, xt, 128, 1024, 128)
        rp = capi.nvfp4_rope_params(3, (22, 21, 21), 1e4, 1, 1, 0)
        # (a position that is not aligned ends the calls that pass)
        return capi.nvfp4_rope(t, len(tensors), 1, 6, 128, A + 2, 3, rp, None)

    assert go((A, A, 1024), (2 * A, 2 * A, 1024)) == ALIGN  # in place
    assert go((A, 2 * A, 1024), (A, 3 * A, 1024)) == ALIGN  # one input twice
    assert go((A, 2 * A, 1024), (2 * A, A, 1024)) == INVALID  # swapped
    assert go((A, 3 * A, 1024), (2 * A, 3 * A, 1024)) == INVALID
    assert go((A, A, 1024), (A, 2 * A, 1024)) == INVALID
    assert go((A, A, 2048)) == INVALID


def test_a_batch_of_no_sequences_is_no_work():
    """As empty tensors have it: arrays without an address."""
    none = _batch(n=0, rows=0, max_rows=0, page_table=None, lens=None, starts=None)
    query = capi.nvfp4_kv8_query(q=None, out=None, lse=None, q_heads=8, scale=0.1, causal=1, window=-1)
    assert capi.nvfp4_kv8_write(_cache(), none, 1, None, 0, 0, None, 0, 0, None, 0, None) == OK
    assert capi.nvfp4_kv8_read(_cache(), none, 1, None, 0, 0, None, 0, 0, None, 0, None) == OK
    assert capi.nvfp4_kv8_attention(_cache(), none, query, None, 0, None) == OK
