"""Host-side checks of the decay attention and layer norm entry points (no GPU): argument validation,
workspace sizes, and the 64-bit formulas against differences."""
import ctypes

import pytest
import torch

import decay_oracle as do
import hybrid_gated_linear_gb300 as lz

OK, INVALID, UNSUPPORTED, CUDA, TIMEOUT, CHECK, WORKSPACE = range(7)
A = 0x7f0000000000  # fake, 16-byte aligned device addresses: validation never dereferences


@pytest.fixture(scope="module")
def lib():
    lz.build()
    return lz.library()


def _a(i):
    return A + i * 0x100000000


def _s(*x):
    return ctypes.byref(lz.lizard_strides(*x))


def _dims(**kw):
    a = dict(B=2, H=4, Hk=2, L=0, dk=64, dv=128, dtype=lz.LIZARD_BF16, scale=0.0)
    a.update(kw)
    return lz.lizard_decay_dims(*a.values())


FWD = dict(q=_a(1), s_q=None, k=_a(2), s_k=None, v=_a(3), s_v=None, g=_a(4), s_g=None, count=None, h0=None, y=_a(5),
           s_y=None, hf=None, ws=_a(6), bytes=1 << 30)
BWD = dict(q=_a(1), s_q=None, k=_a(2), s_k=None, v=_a(3), s_v=None, g=_a(4), s_g=None, count=None, h0=None, dy=_a(5),
           s_dy=None, dhf=None, dq=_a(6), s_dq=None, dk=_a(7), s_dk=None, dv=_a(8), s_dv=None, dg=_a(9), dh0=None,
           ws=_a(10), bytes=1 << 30)
STEP = dict(q=_a(1), s_q=None, k=_a(2), s_k=None, v=_a(3), s_v=None, g=_a(4), s_g=None, h=_a(6), y=_a(5), s_y=None)


def _call(fn, dims, base, **kw):
    """Refused calls only: an accepted one would be launched where a GPU is present."""
    a = dict(base)
    a.update(kw)
    st = fn(None if dims is None else ctypes.byref(dims), *a.values(), None)
    assert st != OK and st != CUDA, "not refused"
    return st


def _three(lib):
    return [(lib.lizard_decay_attn_fwd, FWD, "y"), (lib.lizard_decay_attn_bwd, BWD, "dq"),
            (lib.lizard_decay_attn_step, STEP, "y")]


@pytest.mark.parametrize("bad", [dict(B=0), dict(B=65536), dict(H=0), dict(Hk=0), dict(H=4, Hk=3), dict(L=-1), dict(dtype=2),
                                 dict(scale=float("nan")), dict(scale=float("inf")), dict(L=1 << 29)])
def test_decay_dims_refused(lib, bad):
    for fn, base, _ in _three(lib):
        assert _call(fn, _dims(**{"L": 5, **bad}), base) == INVALID
    assert lib.lizard_decay_attn_workspace_bytes(ctypes.byref(_dims(**{"L": 5, **bad})), 1) == 0


@pytest.mark.parametrize("L", [2 ** 31 - 1, 2 ** 31 - 64, 2 ** 31 - 128])
def test_decay_axes_whose_last_chunk_ends_past_31_bits_refused(lib, L):
    d = _dims(B=1, H=1, Hk=1, L=L, dk=64, dv=64)
    for fn, base, _ in _three(lib):
        assert _call(fn, d, base, **({"bytes": 1 << 62} if "bytes" in base else {})) == INVALID
    for bwd in (0, 1):
        assert lib.lizard_decay_attn_workspace_bytes(ctypes.byref(d), bwd) == 0


def test_decay_widths_and_missing_arguments_refused(lib):
    for fn, base, _ in _three(lib):
        for bad in (dict(dk=32), dict(dv=96), dict(dk=256), dict(dv=0)):
            assert _call(fn, _dims(L=5, **bad), base) == UNSUPPORTED
        assert _call(fn, None, base) == INVALID
        for name in ("q", "k", "v", "g", "y", "dy", "dq", "dk", "dv", "h"):
            if name in base:
                assert _call(fn, _dims(L=5), base, **{name: None}) == INVALID, name
        for name in base:
            if name in ("ws", "bytes") or name.startswith("s_"):
                continue
            assert _call(fn, _dims(L=5), base, **{name: _a(20) + (2 if name == "g" else 4)}) == INVALID, name


def test_decay_strides_refused(lib):
    for fn, base, out in _three(lib):
        for s in ("s_q", "s_k", "s_v"):
            assert _call(fn, _dims(L=5), base, **{s: _s(-64, 64, 64)}) == INVALID
            assert _call(fn, _dims(L=5), base, **{s: _s(4096, 64, 4)}) == INVALID  # not 16 bytes
            assert _call(fn, _dims(L=5), base, **{s: _s(1 << 50, 64, 64)}) == INVALID
        assert _call(fn, _dims(L=5), base, s_g=_s(20, 5, -1)) == INVALID
        assert _call(fn, _dims(L=5), base, s_g=_s(1 << 47, 5, 1)) == INVALID
        # outputs: no repeated rows
        assert _call(fn, _dims(L=5), base, **{"s_" + out: _s(0, 640, 128)}) == INVALID
        assert _call(fn, _dims(L=5), base, **{"s_" + out: _s(512, 128, 128)}) == INVALID


def test_decay_overlaps_refused(lib):
    for fn, base, out in _three(lib):
        for x in ("q", "k", "v", "g", "dy"):
            if x in base:
                assert _call(fn, _dims(L=5), base, **{out: base[x]}) == INVALID, x
    for x in ("q", "k", "v", "y", "g"):
        assert _call(lib.lizard_decay_attn_fwd, _dims(L=5), FWD, hf=FWD[x]) == INVALID
        assert _call(lib.lizard_decay_attn_fwd, _dims(L=5), FWD, ws=FWD[x]) == INVALID
        assert _call(lib.lizard_decay_attn_step, _dims(L=5), STEP, h=STEP[x]) == INVALID
    assert _call(lib.lizard_decay_attn_fwd, _dims(L=5), FWD, h0=_a(30), hf=_a(30)) == INVALID
    assert _call(lib.lizard_decay_attn_bwd, _dims(L=5), BWD, dhf=_a(30), dh0=_a(30)) == INVALID
    for x in ("dq", "dk", "dv"):
        assert _call(lib.lizard_decay_attn_bwd, _dims(L=5), BWD, dg=BWD[x]) == INVALID
        assert _call(lib.lizard_decay_attn_bwd, _dims(L=5), BWD, dk=BWD["dq"]) == INVALID


def test_decay_workspace(lib):
    for bwd, fn, base in ((0, lib.lizard_decay_attn_fwd, FWD), (1, lib.lizard_decay_attn_bwd, BWD)):
        for kw in (dict(L=5), dict(L=4096, B=2, H=32, Hk=8), dict(L=1, B=1, H=1, Hk=1, dtype=lz.LIZARD_F32)):
            d = _dims(**kw)
            n = lib.lizard_decay_attn_workspace_bytes(ctypes.byref(d), bwd)
            assert n >= 256
            assert _call(fn, d, base, bytes=n - 1) == WORKSPACE
            assert _call(fn, d, base, ws=None) == WORKSPACE
            assert _call(fn, d, base, ws=_a(20) + 8) == WORKSPACE


# ---------------------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------------------
def _norm_dims(**kw):
    a = dict(N=2, H=3, T=5, d=64, per_head=1, dtype=lz.LIZARD_BF16, eps=1e-5)
    a.update(kw)
    return lz.lizard_norm_dims(*a.values())


NORM = dict(x=_a(1), s_x=None, w=_a(2), b=_a(3), y=_a(4), s_y=None)
NORM_BWD = dict(x=_a(1), s_x=None, w=_a(2), dy=_a(3), s_dy=None, dx=_a(4), s_dx=None, dw=_a(5), db=_a(6), ws=_a(7), bytes=1 << 30)


def test_norm_refusals(lib):
    for fn, base in ((lib.lizard_layer_norm_fwd, NORM), (lib.lizard_layer_norm_bwd, NORM_BWD)):
        for bad in (dict(N=0), dict(H=0), dict(T=-1), dict(per_head=2), dict(dtype=7), dict(eps=float("nan")),
                    dict(T=1 << 30), dict(H=65536)):
            assert _call(fn, _norm_dims(**bad), base) == INVALID, bad
            assert lib.lizard_layer_norm_workspace_bytes(ctypes.byref(_norm_dims(**bad))) == 0
        for d in (0, 4, 12, 16392):
            assert _call(fn, _norm_dims(d=d), base) == UNSUPPORTED
        assert _call(fn, None, base) == INVALID
        assert _call(fn, _norm_dims(), base, x=None) == INVALID
        assert _call(fn, _norm_dims(), base, x=_a(1) + 2) == INVALID
        assert _call(fn, _norm_dims(), base, w=_a(1) + 2) == INVALID
        assert _call(fn, _norm_dims(), base, s_x=_s(960, 320, 60)) == INVALID
        out, s_out = ("y", "s_y") if fn is lib.lizard_layer_norm_fwd else ("dx", "s_dx")
        assert _call(fn, _norm_dims(), base, **{s_out: _s(960, 0, 64)}) == INVALID
        assert _call(fn, _norm_dims(), base, **{out: _a(2)}) == INVALID  # over the weight
        assert _call(fn, _norm_dims(), base, **{out: _a(1) + 128}) == INVALID  # one row on
        assert _call(fn, _norm_dims(), base, **{out: _a(1), s_out: _s(960, 64, 192)}) == INVALID  # in place, another order
    assert _call(lib.lizard_layer_norm_fwd, _norm_dims(), NORM, y=None) == INVALID
    for name in ("dw", "db", "ws"):
        for x in ("x", "dy", "dx", "w"):
            assert _call(lib.lizard_layer_norm_bwd, _norm_dims(), NORM_BWD, **{name: NORM_BWD[x]}) == INVALID
    n = lib.lizard_layer_norm_workspace_bytes(ctypes.byref(_norm_dims()))
    assert n >= 256 and _call(lib.lizard_layer_norm_bwd, _norm_dims(), NORM_BWD, bytes=n - 1) == WORKSPACE
    assert _call(lib.lizard_layer_norm_bwd, _norm_dims(), NORM_BWD, ws=None) == WORKSPACE


def test_calls_without_work_return_ok(lib):
    """Nothing to compute and nothing asked for: accepted before anything is launched."""
    d = _dims(L=0)
    assert lib.lizard_decay_attn_fwd(ctypes.byref(d), *FWD.values(), None) == OK
    assert lib.lizard_decay_attn_bwd(ctypes.byref(d), *BWD.values(), None) == OK
    assert lib.lizard_decay_attn_step(ctypes.byref(d), *STEP.values(), None) == OK
    n = _norm_dims(T=0)
    assert lib.lizard_layer_norm_fwd(ctypes.byref(n), *NORM.values(), None) == OK
    none = {**NORM_BWD, "dx": None, "dw": None, "db": None}
    assert lib.lizard_layer_norm_bwd(ctypes.byref(_norm_dims()), *none.values(), None) == OK


# ---------------------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------------------
def test_binding_refuses_host_and_wrong_tensors(lib):
    d = lz.lizard_decay_dims(1, 2, 2, 3, 64, 64, lz.LIZARD_F32, 0.0)
    q = torch.zeros(1, 2, 3, 64)
    g = torch.zeros(1, 2, 3)
    with pytest.raises(ValueError):
        lz.lizard_decay_attn_step(d, q, q, q, g, torch.zeros(1, 2, 64, 64), q)
    with pytest.raises(ValueError):
        lz.lizard_decay_attn_fwd(d, q, q, q, g, None, None, q, None, None)
    n = lz.lizard_norm_dims(1, 2, 3, 64, 0, lz.LIZARD_F32, 0.0)
    with pytest.raises(ValueError):
        lz.lizard_layer_norm_fwd(n, q, None, None, q)


# ---------------------------------------------------------------------------------------
# the 64-bit formulas against differences
# ---------------------------------------------------------------------------------------
def test_decay_gradients_against_differences():
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    B, H, L, dk, dv = 2, 2, 6, 3, 4
    x = dict(q=r(B, H, L, dk), k=r(B, H, L, dk), v=r(B, H, L, dv), lg=-r(B, H, L).abs(), h0=r(B, H, dk, dv))
    dy, df = r(B, H, L, dv), r(B, H, dk, dv)

    def loss(x):
        y, hs = do.forward(x["q"], x["k"], x["v"], torch.exp(x["lg"]), x["h0"], 0.7)
        return float((y * dy).sum() + (hs[-1] * df).sum())

    g = torch.exp(x["lg"])
    _, hs = do.forward(x["q"], x["k"], x["v"], g, x["h0"], 0.7)
    grads = dict(zip(("q", "k", "v", "lg", "h0"), do.backward(x["q"], x["k"], x["v"], g, hs, dy, df, 0.7)))
    e = 1e-5
    for name, t in x.items():
        for i in range(0, t.numel(), 5):
            at = t.view(-1)[i].item()
            t.view(-1)[i] = at + e
            up = loss(x)
            t.view(-1)[i] = at - e
            down = loss(x)
            t.view(-1)[i] = at
            # central differences: e^2 times a third derivative of some hundreds, and 1e-16 / e of a loss of ~1e2
            assert abs((up - down) / (2 * e) - grads[name].reshape(-1)[i].item()) < 1e-6, (name, i)


def test_norm_gradients_against_differences():
    gen = torch.Generator().manual_seed(4)
    x, w, b, dy = (torch.randn(*s, generator=gen, dtype=torch.float64) for s in ((3, 8), (8,), (8,), (3, 8)))
    dx, dw, db, _ = do.norm_backward(x, w, dy, 1e-2, (0,))
    e = 1e-5
    for t, grad in ((x, dx), (w, dw), (b, db)):
        for i in range(t.numel()):
            at = t.view(-1)[i].item()
            t.view(-1)[i] = at + e
            up = float((do.norm(x, w, b, 1e-2)[0] * dy).sum())
            t.view(-1)[i] = at - e
            down = float((do.norm(x, w, b, 1e-2)[0] * dy).sum())
            t.view(-1)[i] = at
            assert abs((up - down) / (2 * e) - grad.reshape(-1)[i].item()) < 1e-6
