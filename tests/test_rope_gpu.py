"""Rotary positions on the GPU against the 64-bit oracle.

Tolerance: the angle's fp32 rounding (pi 2^-25), cosine and sine (2 ulp), the factor and the
two products and their sum each add at most a few 2^-24 relative to |a| + |b| of the pair:
below 2^-21 f (|a| + |b|); then one rounding to the output type.
"""
import numpy as np
import pytest

import cache_oracle as co
import hybrid_gated_linear_gb300 as lz

pytestmark = pytest.mark.gpu

KIND = {"plain": 0, "linear": 1, "parts": 2}


def make_rope(rot, layout="half", scaling="plain", factor=1.0, attn=1.0):
    import torch
    spec = lz.lizard_rope_spec(rot, KIND[scaling], 500000.0, factor, 1.0, 4.0, 8192)
    th = co.theta(rot, 500000.0, scaling, factor)
    turns = lz.lizard_rope_table(spec).cuda()
    return lz.lizard_rope(turns, rot, 0 if layout == "half" else 1, attn), th


def rows(rng, N, H, T, d, dtype, order):
    """A device tensor [N,H,T,d] and its values; order "blhd" is a view of token-major memory,
    "packed" a slice of a wider row."""
    import torch
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    if order == "bhld":
        t = torch.from_numpy(rng.standard_normal((N, H, T, d)).astype(np.float32)).to(dt).cuda()
    elif order == "blhd":
        t = torch.from_numpy(rng.standard_normal((N, T, H, d)).astype(np.float32)).to(dt).cuda().permute(0, 2, 1, 3)
    else:
        t = torch.from_numpy(rng.standard_normal((N, T, H + 3, d)).astype(np.float32)).to(dt).cuda()
        t = t[:, :, 1:1 + H].permute(0, 2, 1, 3)
    return t, t.float().cpu().numpy().astype(np.float64)


def check(got, x, pos, th, layout, attn, sign, dtype):
    want = co.rotate(x, pos, th, layout, attn, sign)
    rot = 2 * len(th)
    pair = np.abs(x).copy()
    a, b = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    s = pair[..., a] + pair[..., b]
    pair[..., a], pair[..., b] = s, s
    pair[..., rot:] = 0
    out = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    bound = 2.0 ** -21 * attn * pair + out * np.abs(want) * 1.001
    bound[..., rot:] = 0  # channels that are not rotated are copied
    err = np.abs(got.float().cpu().numpy().astype(np.float64) - want)
    assert (err <= bound).all(), float((err - bound).max())


CASES = [  # N, H, Hk, T, d, rot, layout, scaling, dtype, order, far
    (1, 1, 1, 1, 128, 128, "half", "plain", "bf16", "bhld", True),
    (3, 4, 2, 5, 128, 128, "half", "parts", "bf16", "blhd", True),
    (2, 3, 1, 17, 64, 64, "half", "linear", "f32", "bhld", True),
    (2, 2, 2, 33, 128, 64, "interleaved", "plain", "bf16", "packed", False),
    (1, 5, 5, 7, 64, 20, "half", "plain", "bf16", "blhd", False),
    (1, 2, 1, 7, 64, 22, "interleaved", "parts", "f32", "bhld", True),
    (2, 3, 0, 9, 80, 2, "half", "plain", "f32", "bhld", False),
    (1, 2, 2, 3, 8, 8, "interleaved", "plain", "bf16", "bhld", False),
    (1, 9, 3, 700, 256, 256, "half", "plain", "bf16", "blhd", False),
    (4, 8, 8, 129, 24, 24, "interleaved", "plain", "f32", "blhd", False),
]


@pytest.mark.parametrize("case", CASES, ids=[str(c) for c in CASES])
def test_rope_forward_and_backward(case):
    import torch
    N, H, Hk, T, d, rot, layout, scaling, dtype, order, far = case
    rng = np.random.default_rng(hash(case[:6]) % 2 ** 31)
    attn = 1.25 if scaling == "parts" else 1.0
    rope, th = make_rope(rot, layout, scaling, 8.0, attn)
    q, qn = rows(rng, N, H, T, d, dtype, order)
    k, kn = rows(rng, N, Hk, T, d, dtype, order) if Hk else (None, None)
    pos = rng.integers(0, 2 ** 40 if far else 5000, (N, T))
    if far:
        pos[0, 0] = -3
    dims = lz.lizard_rope_dims(N, H, Hk, T, d, lz.LIZARD_F32 if dtype == "f32" else lz.LIZARD_BF16)
    pt = torch.from_numpy(pos).cuda()
    for call, sign in ((lz.lizard_rope_fwd, 1.0), (lz.lizard_rope_bwd, -1.0)):
        yq = torch.empty_like(q)
        yk = torch.empty_like(k) if Hk else None
        call(dims, rope, q, k, pt, yq, yk)
        check(yq, qn, pos[:, None], th, layout, attn, sign, dtype)
        if Hk:
            check(yk, kn, pos[:, None], th, layout, attn, sign, dtype)
    assert lz.lizard_last_launch_count() == 1


def test_rope_in_place_on_a_packed_projection_and_default_positions():
    import torch
    N, H, Hk, T, d = 2, 4, 2, 19, 64
    rng = np.random.default_rng(5)
    rope, th = make_rope(d)
    w = torch.from_numpy(rng.standard_normal((N, T, H + 2 * Hk, d)).astype(np.float32)).cuda()
    was = w.cpu().numpy().astype(np.float64)
    q, k = w[:, :, :H].permute(0, 2, 1, 3), w[:, :, H:H + Hk].permute(0, 2, 1, 3)
    lz.lizard_rope_fwd(lz.lizard_rope_dims(N, H, Hk, T, d, lz.LIZARD_F32), rope, q, k, None, q, k)
    pos = np.arange(T)[None, None]
    check(q, was[:, :, :H].transpose(0, 2, 1, 3), pos, th, "half", 1.0, 1.0, "f32")
    check(k, was[:, :, H:H + Hk].transpose(0, 2, 1, 3), pos, th, "half", 1.0, 1.0, "f32")
    np.testing.assert_array_equal(w[:, :, H + Hk:].cpu().numpy(), was[:, :, H + Hk:])


def test_rope_gradient_against_differences():
    """d/dx of sum(rotate(x) * dy) by central differences in the oracle's fp64 forward equals
    the backward call (the map is linear: differences are exact up to rounding)."""
    import torch
    T, d, rot = 3, 16, 12
    rng = np.random.default_rng(6)
    rope, th = make_rope(rot, "half", "plain", attn=1.5)
    dy = rng.standard_normal((1, 1, T, d)).astype(np.float32)
    pos = np.array([[3, 50, 999]])
    x = rng.standard_normal((1, 1, T, d))
    grad = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = 0.5
        f = [(co.rotate(x + s * e, pos[:, None], th, "half", 1.5) * dy).sum() for s in (1, -1)]
        grad[i] = f[0] - f[1]
    g = torch.from_numpy(dy).cuda()
    dx = torch.empty_like(g)
    lz.lizard_rope_bwd(lz.lizard_rope_dims(1, 1, 0, T, d, lz.LIZARD_F32), rope, g, None,
                       torch.from_numpy(pos).cuda(), dx, None)
    np.testing.assert_allclose(dx.cpu().numpy(), grad, atol=2.0 ** -20 * 1.5 * 2 * np.abs(dy).max(), rtol=0)


def test_rope_around_the_window_branch_of_the_operator():
    """rotate -> lizard_attn_fwd, lizard_attn_bwd -> rotate back: the gradients of the raw
    window queries and keys equal the oracle's chain (the tolerance of the operator's bf16
    parity tests, relative L2 2e-2)."""
    import torch

    import oracle
    import synth
    from gpu_util import NAMES, gpu_bwd, host, rel_l2, to_dev
    B, H, L, d, M, W = 1, 2, 70, 64, 2, 16
    x = synth.make_fwd_inputs(B, H, L, d, d, M, "f32", "plain", seed=9, with_dy=True)
    rope, th = make_rope(d)
    pos = np.arange(L)[None, None]
    dims = lz.lizard_rope_dims(B, H, H, L, d, lz.LIZARD_F32)
    t = to_dev({n: x[n] for n in ("q", "k")}, "f32")
    yq, yk = torch.empty_like(t["q"]), torch.empty_like(t["k"])
    lz.lizard_rope_fwd(dims, rope, t["q"], t["k"], None, yq, yk)
    turned = dict(x, q=host(yq), k=host(yk))
    g = gpu_bwd(turned, W, "f32")
    dq, dk = torch.from_numpy(g["d_q"]).cuda(), torch.from_numpy(g["d_k"]).cuda()
    lz.lizard_rope_bwd(dims, rope, dq, dk, None, dq, dk)
    ref_in = dict(x, q=co.rotate(x["q"], pos, th).astype(np.float32), k=co.rotate(x["k"], pos, th).astype(np.float32))
    ref = oracle.bwd(*(ref_in[n] for n in NAMES), x["dy"], W=W)
    assert rel_l2(host(dq), co.rotate(ref["d_q"], pos, th, sign=-1.0)) < 2e-2
    assert rel_l2(host(dk), co.rotate(ref["d_k"], pos, th, sign=-1.0)) < 2e-2


@pytest.mark.parametrize("order", ["token", "head"])
@pytest.mark.parametrize("N,T", [(5, 1), (1, 1), (3, 4)])
def test_rope_in_place_on_slices_of_a_packed_projection(N, T, order):
    """q and k inside one [N,T,(H+2Hk),d] or [N,(H+2Hk),T,d] projection, one new token included:
    the slices share no element, although their spans overlap."""
    import torch
    H, Hk, d = 4, 2, 64
    rng = np.random.default_rng(N + T)
    rope, th = make_rope(d)
    shape = (N, T, H + 2 * Hk, d) if order == "token" else (N, H + 2 * Hk, T, d)
    w = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda()
    x = w.permute(0, 2, 1, 3) if order == "token" else w
    was = x.cpu().numpy().astype(np.float64)
    q, k = x[:, :H], x[:, H:H + Hk]
    lz.lizard_rope_fwd(lz.lizard_rope_dims(N, H, Hk, T, d, lz.LIZARD_F32), rope, q, k, None, q, k)
    pos = np.arange(T)[None, None]
    check(q, was[:, :H], pos, th, "half", 1.0, 1.0, "f32")
    check(k, was[:, H:H + Hk], pos, th, "half", 1.0, 1.0, "f32")
    np.testing.assert_array_equal(x[:, H + Hk:].cpu().numpy(), was[:, H + Hk:])
