"""Attention over the 8-bit cache at the edges of its inputs' range, against the definition in 64
bits over the cache's own values (cache_oracle.attend_bound)."""
import pytest

import hybrid_gated_linear_gb300 as lz
from cache_gpu_util import Filled, assert_within, attend, bound_of, check_attention, definition, gaussian, on_device
from test_rope_gpu import make_rope

pytestmark = pytest.mark.gpu

PATHS = [  # N, H, Hk, d, T, dtype: one of each kernel variant
    (2, 4, 2, 64, 1, "bf16"), (2, 4, 2, 128, 1, "f32"),          # 16 rows
    (2, 6, 2, 64, 7, "bf16"), (2, 3, 1, 64, 7, "f32"),           # 32 rows
    (1, 4, 1, 64, 13, "bf16"), (1, 4, 1, 128, 13, "f32"),        # 64 rows
    (1, 2, 1, 64, 75, "f32"),                                    # 128 rows
    (40, 16, 8, 64, 1, "bf16"), (40, 8, 8, 128, 2, "f32"),       # a warp per sequence and head
    (2, 4, 2, 64, 70, "bf16"), (1, 2, 1, 128, 140, "bf16"),      # tcgen05
]
IDS = ["-".join(map(str, p)) for p in PATHS]


def typed(x, dtype):
    import torch
    return x.to(torch.float32 if dtype == "f32" else torch.bfloat16)


@pytest.mark.parametrize("keys,queries", [(0.0, 0.0), (0.0, 2.0 ** -9), (0.0, 1.0), (2.0 ** -30, 0.0), (1.0, 0.0),
                                          (2.0 ** -100, 2.0 ** -60)])
@pytest.mark.parametrize("path", PATHS, ids=IDS)
def test_zero_and_tiny_queries_and_keys(path, keys, queries):
    """All logits (nearly) 0: the mean of the visible values, although hidden tokens share blocks
    with visible ones and the logits' factor is below the smallest fp32 number."""
    N, H, Hk, d, T, dtype = path
    held = [T + 37 - n % 30 for n in range(N)]
    k, v = gaussian((N, Hk, max(held), d), 1, keys), gaussian((N, Hk, max(held), d), 2)
    q = typed(gaussian((N, H, T, d), 3, queries), dtype)
    add = typed(gaussian((N, H, T, d), 4), dtype)
    f = Filled(k, v, [0] * N, held, 16, "e4m3")
    check_attention(f, q, [h - T for h in held], W=20, y_add=add)


# What the weights cannot resolve, in units of a row's largest: include/lizard.h.
FLOOR = {"bf16": 2.0 ** -31, "f32": 2.0 ** -37}


@pytest.mark.parametrize("below", [12.3, 18.7, 21.4, 24.6])
@pytest.mark.parametrize("path", PATHS, ids=IDS)
def test_a_token_far_above_the_others(path, below):
    """The first token takes nearly all of the weight and has a value of zero (an attention sink):
    the output is what the others, each 2^-below as heavy, add up to."""
    import math
    N, H, Hk, d, T, dtype = path
    L = 600 if N > 2 else 3000
    k, v = gaussian((N, Hk, L + T, d), 1, 0.0), gaussian((N, Hk, L + T, d), 2) + 1.0
    k[:, :, 0, 0], v[:, :, 0] = 16.0, 0.0
    q = gaussian((N, H, T, d), 3)
    q[..., 0] = below * math.log(2) * d ** 0.5 / 16
    f = Filled(k, v, [0] * N, [L + T] * N, 64, "e4m3")
    check_attention(f, typed(q, dtype), [L] * N, floor=FLOOR[dtype])


@pytest.mark.parametrize("path", PATHS, ids=IDS)
def test_bad_positions_see_no_cached_token(path):
    """A position below zero or too far to be counted: the sequence sees the meta tokens only, is
    merged as any other, and the status says so; a bad count leaves rows of zeros."""
    import torch
    N, H, Hk, d, T, dtype = path
    N = max(N, 3)
    k, v = gaussian((N, Hk, T + 40, d), 1), gaussian((N, Hk, T + 40, d), 2)
    f = Filled(k, v, [0] * N, [T + 40] * N, 16, "i8")
    q, add = typed(gaussian((N, H, T, d), 3), dtype), typed(gaussian((N, H, T, d), 4), dtype)
    meta = [typed(gaussian((H, 3, d), 5 + i), dtype) for i in range(2)]
    check = lz.LizardError(5, "").status
    for bad in (-1, -2 ** 63, 2 ** 63 - 1, 2 ** 62 + 5):
        pos = [40, bad] + [40] * (N - 2)
        y = attend(f, q, pos, meta=meta, y_add=add, alpha=0.5, status=check)
        # the same with nothing visible
        kw = dict(meta=meta, y_add=add, alpha=0.5, first=[0, 2 ** 40] + [0] * (N - 2))
        want = definition(f, q, [40] * N, **kw)
        assert_within(y, want[0], bound_of(q, [40], *want, add))
    count = [T] * N
    for bad in (-1, T + 1, -2 ** 31, 2 ** 31 - 1):
        count[1] = bad
        y = attend(f, q, [40] * N, count=count, meta=meta, y_add=add, alpha=0.5, status=check)
        assert (y[1] == 0).all() and torch.isfinite(y).all()


def test_writes_and_reads_at_positions_too_far_to_be_counted_are_flagged():
    import torch
    k = gaussian((2, 1, 5, 64), 1)
    f = Filled(k, k, [0, 0], [5, 5], 16, "e4m3")
    was = [x.clone() for x in f.h._keep]
    ws = torch.zeros(lz.lizard_cache_workspace_bytes(), dtype=torch.uint8, device="cuda")
    io = lz.lizard_cache_io(5, lz.LIZARD_F32)
    for bad in (2 ** 63 - 1, 2 ** 63 - 3, -2 ** 63, -1):
        lz.lizard_cache_write(f.h, io, k, k, None, on_device([bad] * 2), None, ws)
        assert lz.lizard_check_device_errors(ws) == lz.LizardError(5, "").status
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(was, f.h._keep))
        out = [torch.full_like(k, 3.0) for _ in "kv"]
        lz.lizard_cache_read(f.h, io, on_device([bad, 0]), None, *out, ws)
        assert lz.lizard_check_device_errors(ws) == lz.LizardError(5, "").status
        assert all((o[0] == 0).all() and torch.equal(o[1], h[1]) for o, h in zip(out, f.held))


@pytest.mark.parametrize("order", ["token", "head"])
@pytest.mark.parametrize("N,T", [(5, 1), (3, 6)])
def test_outputs_beside_other_tensors_in_one_buffer(N, T, order):
    """Attention into a slice of the buffer that holds its queries and the other branch's output,
    and a read-back of keys and values into one buffer: no element is shared."""
    import torch
    H, Hk, d = 4, 2, 64
    f = Filled(gaussian((N, Hk, 50, d), 1), gaussian((N, Hk, 50, d), 2), [0] * N, [50] * N, 16, "e4m3")
    shape = (N, T, 3 * H, d) if order == "token" else (N, 3 * H, T, d)
    w = gaussian(shape, 3)
    x = w.permute(0, 2, 1, 3) if order == "token" else w
    q, add, y = x[:, :H], x[:, H:2 * H], x[:, 2 * H:]
    pos = [50 - T] * N
    want = attend(f, q.contiguous(), pos, y_add=add.contiguous())
    was = x[:, :2 * H].clone()
    dims = lz.lizard_cache_attn_dims(H, T, 0, 0, lz.LIZARD_F32, 0.0, 1.0)
    ws = torch.zeros(lz.lizard_cache_attn_workspace_bytes(f.h, dims), dtype=torch.uint8, device="cuda")
    lz.lizard_cache_attn(f.h, dims, q, None, on_device(pos), None, None, None, None, add, y, ws)
    assert lz.lizard_check_device_errors(ws) == 0
    assert torch.equal(y, want) and torch.equal(x[:, :2 * H], was)
    shape = (N, T, 2 * Hk, d) if order == "token" else (N, 2 * Hk, T, d)
    both = gaussian(shape, 4)
    both = both.permute(0, 2, 1, 3) if order == "token" else both
    lz.lizard_cache_read(f.h, lz.lizard_cache_io(T, lz.LIZARD_F32), on_device(pos), None, both[:, :Hk], both[:, Hk:], ws)
    assert lz.lizard_check_device_errors(ws) == 0
    for i in range(2):
        assert torch.equal(both[:, i * Hk:(i + 1) * Hk], f.held[i][:, :, 50 - T:])


@pytest.mark.parametrize("rot,T", [(82, 130), (84, 128), (88, 300), (114, 96), (120, 96), (128, 300)])
def test_rotated_writes_of_large_pages(rot, T):
    """Pages of 128 tokens of 128 channels with any number of rotated channels: the angles' shared
    memory is near or above what a launch gets without asking."""
    import numpy as np
    import torch

    import cache_oracle as co
    N, Hk, P, d = 2, 2, 128, 128
    k, v = gaussian((N, Hk, T, d), rot), gaussian((N, Hk, T, d), rot + 1)
    f = Filled(k, v, [0] * N, [T] * N, P, "e4m3")
    rope, th = make_rope(rot)
    ws = torch.zeros(lz.lizard_cache_workspace_bytes(), dtype=torch.uint8, device="cuda")
    io = lz.lizard_cache_io(T, lz.LIZARD_F32)
    lz.lizard_cache_write(f.h, io, k, v, rope, on_device([0] * N), None, ws)
    out = [torch.empty_like(k), torch.empty_like(v)]
    lz.lizard_cache_read(f.h, io, on_device([0] * N), None, *out, ws)
    assert lz.lizard_check_device_errors(ws) == 0
    want = co.rotate(k.cpu().numpy(), np.arange(T), th)
    scale = f.h._keep[2].cpu().numpy()[f.table.cpu().numpy()[:, np.arange(T) // P]].transpose(0, 2, 1)[..., None]
    half = np.maximum(np.abs(want) * 2.0 ** -4, scale * 2.0 ** -10) * 1.001 + 2.0 ** -20 * np.abs(want).max()
    assert (np.abs(out[0].cpu().numpy() - want) <= half).all()
    assert torch.equal(out[1], f.held[1])


def test_rows_that_a_write_repeats_may_be_very_many():
    """One row seen 2^31 - 1 times through a stride of 0, of which the counts take a few."""
    import torch
    row = gaussian((1, 2, 1, 64), 1)
    f = Filled(gaussian((1, 2, 20, 64), 2), gaussian((1, 2, 20, 64), 3), [0], [20], 16, "e4m3")
    many = row.expand(1, 2, 2 ** 31 - 1, 64)
    ws = torch.zeros(lz.lizard_cache_workspace_bytes(), dtype=torch.uint8, device="cuda")
    lz.lizard_cache_write(f.h, lz.lizard_cache_io(2 ** 31 - 1, lz.LIZARD_F32), many, many, None, on_device([16]),
                          on_device([3], 32), ws)
    assert lz.lizard_check_device_errors(ws) == 0
    g = Filled(row.repeat(1, 1, 3, 1), row.repeat(1, 1, 3, 1), [16], [19], 16, "e4m3", slots=2)
    out = [torch.empty(1, 2, 19, 64, device="cuda") for _ in "kv"]
    lz.lizard_cache_read(f.h, lz.lizard_cache_io(19, lz.LIZARD_F32), on_device([0]), None, *out, ws)
    for o, h, w in zip(out, f.held, g.held):
        assert torch.equal(o[:, :, :16], h[:, :, :16]) and torch.equal(o[:, :, 16:], w)


@pytest.mark.parametrize("path", PATHS, ids=IDS)
def test_logits_in_the_millions(path):
    """Logits so large that their own rounding is a good part of 1 still give finite outputs, the
    value of the token they pick where one stands out."""
    import torch
    N, H, Hk, d, T, dtype = path
    L = 500 + T
    k, v = gaussian((N, Hk, L, d), 1, 300.0), gaussian((N, Hk, L, d), 2)
    f = Filled(k, v, [0] * N, [L] * N, 32, "e4m3")
    q = typed(gaussian((N, H, T, d), 3, 3000.0), dtype)
    y = attend(f, q, [L - T] * N).double()
    K, V = (x.double().repeat_interleave(H // Hk, 1) for x in f.held)
    z = q.double() @ K.transpose(2, 3) * d ** -0.5
    z.masked_fill_(torch.arange(L, device="cuda") > L - T + torch.arange(T, device="cuda")[:, None], -float("inf"))
    top, at = z.topk(2, -1)
    clear = (top[..., 0] - top[..., 1] > 2.0 ** -8 * top[..., 0].abs() + 100)
    want = V.gather(2, at[..., :1].expand(-1, -1, -1, d))
    assert torch.isfinite(y).all() and clear.any()
    assert ((y - want).abs() <= 2.0 ** -8 * want.abs())[clear].all()
    assert (y.abs() <= V.abs().amax(2, keepdim=True) * (1 + 2.0 ** -7)).all()
