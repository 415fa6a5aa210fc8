"""Host-side checks of the rotary, cache and cache-attention entry points (no GPU): table
values, argument validation, workspace sizes and the oracle's own rounding."""
import ctypes
import math

import numpy as np
import pytest

import cache_oracle as co
import hybrid_gated_linear_gb300 as lz

OK, INVALID, UNSUPPORTED, CUDA, TIMEOUT, CHECK, WORKSPACE = range(7)
A = 0x7f0000000000  # fake, 16-byte aligned device addresses: validation never dereferences


@pytest.fixture(scope="module")
def lib():
    lz.build()
    return lz.library()


def _a(i):
    return A + i * 0x100000000


# ---------------------------------------------------------------------------------------
# the rotary table
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("scaling,name", [(0, "plain"), (1, "linear"), (2, "parts")])
@pytest.mark.parametrize("rot", [2, 20, 128])
def test_rope_table_holds_turns(lib, scaling, name, rot):
    t = lz.lizard_rope_table(lz.lizard_rope_spec(rot, scaling, 10000.0, 4.0, 1.0, 4.0, 2048))
    turns = [int(x) & (2 ** 64 - 1) for x in t.tolist()]
    want = co.theta(rot, 10000.0, name, 4.0, 1.0, 4.0, 2048) / (2 * math.pi) * 2.0 ** 64
    assert len(turns) == rot // 2
    for a, b in zip(turns, want):
        assert abs(a - b) <= 2.0 ** -50 * b + 1  # a few roundings of doubles


def test_rope_table_refusals(lib):
    def st(**kw):
        a = dict(rot=64, scaling=0, base=1e4, factor=2.0, low=1.0, high=4.0, original=2048)
        a.update(kw)
        buf = (ctypes.c_uint64 * 256)()
        return lib.lizard_rope_table(ctypes.byref(lz.lizard_rope_spec(*a.values())), buf)
    assert st() == OK
    for bad in (dict(rot=0), dict(rot=7), dict(rot=514), dict(base=1.0), dict(base=float("nan")),
                dict(scaling=3), dict(scaling=-1), dict(scaling=1, factor=0.5), dict(scaling=1, factor=float("inf")),
                dict(scaling=2, low=4.0, high=4.0), dict(scaling=2, low=-1.0), dict(scaling=2, original=0)):
        assert st(**bad) == INVALID, bad
    assert lib.lizard_rope_table(None, None) == INVALID


# ---------------------------------------------------------------------------------------
# rotary calls
# ---------------------------------------------------------------------------------------
def _rope(rot=128, layout=0, factor=1.0, turns=_a(50)):
    r = lz.lizard_rope.__new__(lz.lizard_rope)
    r.turns, r.rot, r.layout, r.attn_factor = turns, rot, layout, factor
    return r


def _strides(s):
    return None if s is None else ctypes.byref(lz.lizard_strides(*s))


def _rope_st(lib, dims=(2, 4, 2, 8, 128, lz.LIZARD_BF16), rope="", xq=_a(1), sxq=None, xk=_a(2), sxk=None,
             pos=_a(3), yq=_a(4), syq=None, yk=_a(5), syk=None, name="lizard_rope_fwd"):
    d = None if dims is None else ctypes.byref(lz.lizard_rope_dims(*dims))
    r = ctypes.byref(_rope()) if rope == "" else rope if rope is None else ctypes.byref(rope)
    return getattr(lib, name)(d, r, xq, _strides(sxq), xk, _strides(sxk), pos, yq, _strides(syq), yk,
                              _strides(syk), None)


@pytest.mark.parametrize("name", ["lizard_rope_fwd", "lizard_rope_bwd"])
def test_rope_refusals(lib, name):
    def st(**kw):
        return _rope_st(lib, name=name, **kw)
    bf = lz.LIZARD_BF16
    assert st(dims=None) == INVALID
    assert st(rope=None) == INVALID
    for dims in ((0, 4, 2, 8, 128, bf), (2, 0, 2, 8, 128, bf), (2, 4, -1, 8, 128, bf), (2, 4, 2, -1, 128, bf),
                 (2, 4, 2, 8, 128, 7)):
        assert st(dims=dims) == INVALID, dims
    for d in (4, 12, 520):
        assert st(dims=(2, 4, 2, 8, d, bf)) == UNSUPPORTED
    for rope in (_rope(rot=0), _rope(rot=3), _rope(rot=130), _rope(layout=2), _rope(factor=0.0),
                 _rope(factor=float("nan")), _rope(turns=0), _rope(turns=_a(50) + 8)):
        assert st(rope=rope) == INVALID
    for kw in (dict(xq=None), dict(yq=None), dict(xk=None), dict(yk=None), dict(xq=_a(1) + 2), dict(yk=_a(5) + 8),
               dict(pos=_a(3) + 8)):
        assert st(**kw) == INVALID, kw
    # strides: not multiples of 16 bytes, negative, outputs that fold onto themselves
    for kw in (dict(sxq=(4096, 1024, 100)), dict(sxq=(4096, -1024, 128)), dict(syq=(0, 1024, 128)),
               dict(syq=(4096, 1024, 64)), dict(syq=(4096, 512, 128))):
        assert st(**kw) == INVALID, kw
    # overlaps: outputs with each other, partly with inputs, with the table and the positions
    for kw in (dict(yk=_a(4)), dict(yq=_a(1) + 256), dict(yq=_a(2)), dict(yq=_a(50)), dict(yq=_a(3)),
               dict(yq=_a(1), syq=(4096, 128, 512))):
        assert st(**kw) == INVALID, kw
    # no tokens: nothing to do, no pointers needed
    assert st(dims=(2, 4, 2, 0, 128, bf), xq=None, xk=None, yq=None, yk=None) == OK


def test_rope_slices_of_one_projection_may_not_share_a_head(lib):
    """In place on a packed [N,T,(H+2 Hk) d] projection, q and k slices interleave in memory.  One
    head into each other they are refused.  (That slices side by side are accepted is tested where
    the memory exists, on the GPU: a call that passes validation would be launched.)"""
    w = (4 + 2 * 2) * 128
    s = (8 * w, 128, w)
    k = _a(1) + 3 * 128 * 2  # the queries' last head
    assert _rope_st(lib, xq=_a(1), sxq=s, yq=_a(1), syq=s, xk=k, sxk=s, yk=k, syk=s) == INVALID


# ---------------------------------------------------------------------------------------
# the cache
# ---------------------------------------------------------------------------------------
def _cache(**kw):
    a = dict(k_codes=_a(10), v_codes=_a(11), k_scale=_a(12), v_scale=_a(13), table=_a(14), N=2, max_pages=4,
             pages=9, Hk=2, page_tokens=64, d=128, format=0)
    a.update(kw)
    c = lz.lizard_cache.__new__(lz.lizard_cache)
    for k, v in a.items():
        setattr(c, k, v)
    return c


BAD_CACHES = [dict(N=0), dict(N=65536), dict(max_pages=0), dict(pages=0), dict(Hk=0), dict(format=2), dict(k_codes=0),
              dict(v_codes=_a(11) + 4), dict(k_scale=0), dict(v_scale=_a(13) + 4), dict(table=0),
              dict(pages=2 ** 31 - 1, Hk=32767)]


def _io_st(lib, write, cache=None, T=8, dtype=1, k=_a(1), sk=None, v=_a(2), sv=None, rope=None, pos=_a(3),
           count=_a(4), ws=_a(5), wsn=256, **kw):
    c = ctypes.byref(cache or _cache(**kw))
    io = ctypes.byref(lz.lizard_cache_io(T, dtype))
    if write:
        return lib.lizard_cache_write(c, io, k, _strides(sk), v, _strides(sv),
                                      None if rope is None else ctypes.byref(rope), pos, count, ws, wsn, None)
    return lib.lizard_cache_read(c, io, pos, count, k, _strides(sk), v, _strides(sv), ws, wsn, None)


@pytest.mark.parametrize("write", [True, False])
def test_cache_io_refusals(lib, write):
    def st(**kw):
        return _io_st(lib, write, **kw)
    for bad in BAD_CACHES:
        assert st(**bad) == INVALID, bad
    for bad in (dict(d=96), dict(page_tokens=24), dict(page_tokens=256), dict(page_tokens=8)):
        assert st(**bad) == UNSUPPORTED, bad
    for bad in (dict(T=-1), dict(dtype=9), dict(k=None), dict(v=_a(2) + 2), dict(pos=None), dict(count=_a(4) + 4),
                dict(sk=(2048, 1024, 100)), dict(ws=_a(1)), dict(ws=_a(10)), dict(k=_a(10)), dict(v=_a(12)),
                dict(ws=_a(3))):
        assert st(**bad) == INVALID, bad
    for bad in (dict(ws=None), dict(wsn=255), dict(ws=_a(5) + 4)):
        assert st(**bad) == WORKSPACE, bad
    if write:
        assert st(rope=_rope(rot=130)) == INVALID
        assert st(rope=_rope(turns=_a(10))) == INVALID
    else:
        assert st(sk=(2048, 0, 128)) == INVALID
        assert st(v=_a(1)) == INVALID
        assert st(k=_a(14)) == INVALID
    assert st(k_codes=_a(11)) == INVALID
    assert st(k_scale=_a(14)) == INVALID
    assert st(T=0, k=None, v=None) == OK


def _attn_st(lib, dims=(4, 1, 0, 0, 1, 0.0, 1.0), cache=None, q=_a(1), sq=None, rope=None, pos=_a(3), count=_a(4),
             first=None, mk=None, mv=None, add=None, sadd=None, y=_a(6), sy=None, ws=_a(7), wsn=None, **kw):
    c = ctypes.byref(cache or _cache(**kw))
    d = None if dims is None else ctypes.byref(lz.lizard_cache_attn_dims(*dims))
    if wsn is None:
        wsn = max(256, lib.lizard_cache_attn_workspace_bytes(c, d))
    return lib.lizard_cache_attn(c, d, q, _strides(sq), None if rope is None else ctypes.byref(rope), pos, count,
                                 first, mk, mv, add, _strides(sadd), y, _strides(sy), ws, wsn, None)


def test_cache_attn_refusals(lib):
    def st(**kw):
        return _attn_st(lib, **kw)
    for bad in BAD_CACHES:
        assert st(**bad) == INVALID, bad
    assert st(dims=None) == INVALID
    for dims in ((0, 1, 0, 0, 1, 0.0, 1.0), (5, 1, 0, 0, 1, 0.0, 1.0), (4, -1, 0, 0, 1, 0.0, 1.0),
                 (4, 1, 17, 0, 1, 0.0, 1.0), (4, 1, -1, 0, 1, 0.0, 1.0), (4, 1, 0, -1, 1, 0.0, 1.0),
                 (4, 1, 0, 0, 3, 0.0, 1.0), (4, 1, 0, 0, 1, float("inf"), 1.0), (4, 1, 0, 0, 1, 0.0, float("nan")),
                 (4, 1, 2, 0, 1, 0.0, 1.0), (4, 2 ** 30, 0, 0, 1, 0.0, 1.0)):
        assert st(dims=dims) == INVALID, dims
    for bad in (dict(q=None), dict(y=None), dict(y=_a(6) + 2), dict(pos=None), dict(first=_a(8) + 8),
                dict(y=_a(1)), dict(y=_a(10)), dict(y=_a(14)), dict(ws=_a(6)), dict(ws=_a(12)), dict(ws=_a(3)),
                dict(add=_a(6) + 128, y=_a(6)), dict(add=_a(7)), dict(sy=(0, 128, 128)),
                dict(add=_a(6), sadd=(1024, 256, 128)), dict(rope=_rope(rot=200))):
        assert st(**bad) == INVALID, bad
    for bad in (dict(ws=None), dict(wsn=16), dict(ws=_a(7) + 8)):
        assert st(**bad) == WORKSPACE, bad
    assert st(dims=(4, 0, 0, 0, 1, 0.0, 1.0), q=None, y=None) == OK


def test_workspace_sizes(lib):
    assert lib.lizard_cache_workspace_bytes() >= 4
    d = lz.lizard_cache_attn_dims(4, 1, 0, 0, 1, 0.0, 1.0)
    assert lib.lizard_cache_attn_workspace_bytes(ctypes.byref(_cache()), ctypes.byref(d)) >= 4
    assert lib.lizard_cache_attn_workspace_bytes(ctypes.byref(_cache(N=0)), ctypes.byref(d)) == 0


# ---------------------------------------------------------------------------------------
# binding
# ---------------------------------------------------------------------------------------
def test_binding_refuses_wrong_tensors():
    import torch
    z = torch.zeros
    k, s, t = z(3, 2, 16, 64, dtype=torch.uint8), z(3, 2), z(1, 3, dtype=torch.int32)
    lz.lizard_cache(k, k.clone(), s, s.clone(), t, 0)
    for args in ((k, k[:2], s, s, t), (k.float(), k, s, s, t), (k, k, s.double(), s, t), (k, k, s, s[:, :1], t),
                 (k, k, s, s, t.long()), (k.transpose(1, 2), k.transpose(1, 2), s, s, t)):
        with pytest.raises(ValueError):
            lz.lizard_cache(*args, 0)
    with pytest.raises(ValueError):
        lz.lizard_rope(z(4, dtype=torch.int64), 10, 0)
    rope = lz.lizard_rope(z(4, dtype=torch.int64), 8, 0)
    dims = lz.lizard_rope_dims(1, 1, 0, 4, 8, lz.LIZARD_F32)
    with pytest.raises(ValueError):  # host memory
        lz.lizard_rope_fwd(dims, rope, z(1, 1, 4, 8), None, None, z(1, 1, 4, 8), None, stream=0)


# ---------------------------------------------------------------------------------------
# the oracle itself
# ---------------------------------------------------------------------------------------
def test_oracle_codes():
    b = np.arange(256)
    ok = (b & 127) != 127
    v = co.e4m3_decode(b)
    assert v[0x7e] == 448 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[0xb8] == -1.0
    np.testing.assert_array_equal(co.encode(v, "e4m3")[ok], b[ok])
    # halfway values go to the even code, beyond the largest saturates
    mid = (v[:126] + v[1:127]) / 2
    np.testing.assert_array_equal(co.encode(mid, "e4m3"), [i if i % 2 == 0 else i + 1 for i in range(126)])
    assert co.encode(np.array([1e9, -1e9]), "e4m3").tolist() == [0x7e, 0xfe]
    assert co.encode(np.array([2.5, -3.5, 300.0, -300.0]), "i8").view(np.int8).tolist() == [2, -4, 127, -127]


def test_oracle_rotation_is_orthogonal_and_its_adjoint_undoes_it():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 5, 24))
    for layout in ("half", "interleaved"):
        th = co.theta(20)
        pos = np.array([0, 1, 77, 10 ** 9, 2 ** 40])
        y = co.rotate(x, pos, th, layout)
        np.testing.assert_allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-12)
        np.testing.assert_allclose(co.rotate(y, pos, th, layout, sign=-1.0), x, atol=1e-12)
        # relative: <R(p) a, R(q) b> depends on p - q
        a, b = x[0, :1], x[1, :1]
        d1 = (co.rotate(a, [9], th, layout) * co.rotate(b, [4], th, layout)).sum()
        d2 = (co.rotate(a, [105], th, layout) * co.rotate(b, [100], th, layout)).sum()
        np.testing.assert_allclose(d1, d2, atol=1e-12)


def test_binding_refuses_host_memory_everywhere():
    """Handles, workspaces, rows and integers on the host raise before the library is called."""
    import torch
    z = torch.zeros
    k, s, t = z(3, 2, 16, 64, dtype=torch.uint8), z(3, 2), z(1, 3, dtype=torch.int32)
    cache = lz.lizard_cache(k, k.clone(), s, s.clone(), t, 0)
    io, pos, ws = lz.lizard_cache_io(1, lz.LIZARD_F32), z(1, dtype=torch.int64), z(256, dtype=torch.uint8)
    x = z(1, 2, 1, 64)
    dims = lz.lizard_cache_attn_dims(2, 1, 0, 0, lz.LIZARD_F32, 0.0, 1.0)
    for call in (lambda: lz.lizard_cache_write(cache, io, x, x, None, pos, None, ws, stream=0),
                 lambda: lz.lizard_cache_read(cache, io, pos, None, x, x, ws, stream=0),
                 lambda: lz.lizard_cache_attn(cache, dims, x, None, pos, None, None, None, None, None, x, ws, stream=0)):
        with pytest.raises(ValueError, match="device"):
            call()
    rope = lz.lizard_rope(z(32, dtype=torch.int64), 64, 0)
    with pytest.raises(ValueError, match="device"):
        lz.lizard_rope_fwd(lz.lizard_rope_dims(1, 2, 0, 0, 64, lz.LIZARD_F32), rope, None, None, None, None, None, stream=0)
    for bad in (dict(workspace=ws), dict(workspace=None)):
        with pytest.raises(ValueError):
            lz.lizard_cache_write(cache, io, x, x, rope, pos, None, bad["workspace"], stream=0)


def test_binding_refuses_tables_and_positions_that_are_not_integers():
    import torch

    class OnDevice:  # a device tensor's checks, without a device
        is_cuda = True

        def __init__(self, t):
            self.t = t

        def __getattr__(self, name):
            return getattr(self.t, name)

    for dtype in (torch.float64, torch.complex64, torch.int32):
        with pytest.raises(ValueError):
            lz.lizard_rope(torch.zeros(4, dtype=dtype), 8, 0)
        with pytest.raises(ValueError):
            lz._ints(OnDevice(torch.zeros(2, 3, dtype=dtype)), (2, 3), 8)
    ok = torch.zeros(2, 3, dtype=torch.int64)
    assert lz._ints(OnDevice(ok), (2, 3), 8) == ok.data_ptr()


def test_current_stream_without_torchs_private_names(monkeypatch):
    """The shortcut to the current stream's handle is torch's own affair; without it the public
    call is used."""
    import torch

    class Stream:
        cuda_stream = 0x1230
    monkeypatch.setattr(torch.cuda, "current_stream", Stream)
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        with monkeypatch.context() as m:
            m.delattr(torch._C, name, raising=False)
            assert lz._stream(None).value == 0x1230
    assert lz._stream(Stream()).value == 0x1230 and lz._stream(0x50).value == 0x50


# ---------------------------------------------------------------------------------------
# slices of one buffer that share an element
# ---------------------------------------------------------------------------------------
def test_slices_of_one_buffer_that_share_an_element_are_refused(lib):
    """Token-major and head-major, one new token included; every call here shares a head, a part of
    one, or steps over its neighbour differently (those that share nothing run on the GPU)."""
    H, Hk, d, f32 = 4, 2, 128, lz.LIZARD_F32
    for N, T in ((3, 1), (3, 5), (1, 5)):
        for head_major in (False, True):
            w = (H + 2 * Hk) * d
            s = (T * w, T * d, d) if head_major else (T * w, d, w)
            head = (T if head_major else 1) * d * 4  # bytes from one head to the next
            for k in (_a(1) + (H - 1) * head, _a(1) + H * head - 16, _a(1) + 16):
                assert _rope_st(lib, dims=(N, H, Hk, T, d, f32), xq=_a(1), sxq=s, yq=_a(1), syq=s, xk=k, sxk=s, yk=k,
                                syk=s) == INVALID, (N, T, head_major)
                kw = dict(N=N, Hk=Hk, dims=(H, T, 0, 0, f32, 0.0, 1.0))
                assert _attn_st(lib, q=_a(1), sq=s, y=k, sy=s, **kw) == INVALID
                assert _attn_st(lib, q=_a(2), add=_a(1), sadd=s, y=k, sy=s, **kw) == INVALID
            # the last head reaches into the next sequence's or token's first
            if N > 1 or not head_major:
                assert _attn_st(lib, q=_a(1), sq=s, y=_a(1) + (2 * Hk + 1) * head, sy=s, N=N, Hk=Hk,
                                dims=(H, T, 0, 0, f32, 0.0, 1.0)) == INVALID
            v = _a(1) + (Hk - 1) * head
            assert _io_st(lib, False, N=N, Hk=Hk, T=T, dtype=f32, k=_a(1), sk=s, v=v, sv=s) == INVALID
            # beside each other in the first token (sequence), but the second tensor steps differently
            if N > 1 and T > 1:
                t = (s[0] + d, s[1], s[2])
                assert _io_st(lib, False, N=N, Hk=Hk, T=T, dtype=f32, k=_a(1), sk=s, v=_a(1) + Hk * head, sv=t) == INVALID
