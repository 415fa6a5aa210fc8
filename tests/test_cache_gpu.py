"""The 8-bit paged cache and the attention over it, on the GPU against the 64-bit oracle.

Codes and scales: the quantisation is exactly defined, so without rotation every byte, scale
and read-back value is equal.  A rotated key has the rotation's fp32 error, which may move a
value across a rounding border: its distance from the exact value is then that of a rounding,
half a step (2^-4 relative or half the smallest code for e4m3, half a code for bytes).
Attention: cache_oracle.attend_bound, elementwise.
"""
import numpy as np
import pytest

import cache_oracle as co
import hybrid_gated_linear_gb300 as lz
from test_rope_gpu import make_rope

pytestmark = pytest.mark.gpu

DT = {"f32": lz.LIZARD_F32, "bf16": lz.LIZARD_BF16}
FMT = {"e4m3": lz.LIZARD_KV_E4M3, "i8": lz.LIZARD_KV_I8}


def dev_rows(x, dtype, order="bhld"):
    """Values [N,H,T,d] rounded to the type, as a device tensor in the order and as numpy."""
    import torch
    t = torch.from_numpy(np.asarray(x, np.float32)).to(torch.float32 if dtype == "f32" else torch.bfloat16).cuda()
    if order == "blhd":
        t = t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    return t, t.float().cpu().numpy().astype(np.float64)


class Dev:
    """Device copy of an oracle cache."""

    def __init__(self, c):
        import torch
        self.k, self.v = (torch.from_numpy(c.codes[x]).cuda() for x in "kv")
        self.ks, self.vs = (torch.from_numpy(c.scale[x]).cuda() for x in "kv")
        self.table = torch.from_numpy(c.table).cuda()
        self.h = lz.lizard_cache(self.k, self.v, self.ks, self.vs, self.table, FMT[c.fmt])
        self.ws = torch.zeros(lz.lizard_cache_workspace_bytes(), dtype=torch.uint8, device="cuda")

    def write(self, k, v, dtype, pos, count=None, rope=None, ok=True):
        io = lz.lizard_cache_io(k.shape[2], DT[dtype])
        lz.lizard_cache_write(self.h, io, k, v, rope, ints(pos, 8), ints(count, 4), self.ws)
        st = lz.lizard_check_device_errors(self.ws)
        assert (st == 0) == ok, st

    def read(self, T, dtype, pos, count=None, order="bhld", ok=True):
        import torch
        dt = torch.float32 if dtype == "f32" else torch.bfloat16
        N, Hk, d = self.h.N, self.h.Hk, self.h.d
        out = [torch.full((N, Hk, T, d), 7.0, dtype=dt, device="cuda") for _ in "kv"]
        if order == "blhd":
            out = [o.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for o in out]
        lz.lizard_cache_read(self.h, lz.lizard_cache_io(T, DT[dtype]), ints(pos, 8), ints(count, 4), *out, self.ws)
        st = lz.lizard_check_device_errors(self.ws)
        assert (st == 0) == ok, st
        return [o.float().cpu().numpy().astype(np.float64) for o in out]


def ints(x, size):
    import torch
    if x is None:
        return None
    return torch.tensor(np.asarray(x), dtype=torch.int64 if size == 8 else torch.int32).cuda()


def assert_same_cache(dev, c, live):
    """Bytes and scales of every live (sequence, token) equal the oracle's."""
    codes = {"k": dev.k.cpu().numpy(), "v": dev.v.cpu().numpy()}
    scale = {"k": dev.ks.cpu().numpy(), "v": dev.vs.cpu().numpy()}
    for x in "kv":
        for n, toks in enumerate(live):
            for t in toks:
                pid, r = c.table[n, t // c.P % c.S], t % c.P
                np.testing.assert_array_equal(scale[x][pid], c.scale[x][pid])
                # a zero may carry either sign
                a, b = (co.decode(m[pid][:, r], c.fmt) for m in (codes[x], c.codes[x]))
                np.testing.assert_array_equal(a, b)


WRITES = [  # N, Hk, P, d, T, dtype, fmt, order, starts
    (1, 1, 16, 64, 1, "bf16", "e4m3", "bhld", [0]),
    (3, 2, 64, 128, 1, "bf16", "e4m3", "bhld", [0, 63, 64]),
    (3, 2, 64, 128, 1, "f32", "i8", "blhd", [5, 127, 1]),
    (2, 3, 16, 64, 50, "bf16", "i8", "blhd", [3, 16]),
    (2, 2, 128, 128, 300, "f32", "e4m3", "bhld", [0, 127]),
    (2, 1, 32, 128, 33, "bf16", "e4m3", "blhd", [31, 30]),
    (2, 1, 128, 64, 129, "bf16", "i8", "bhld", [1, 255]),
]


@pytest.mark.parametrize("case", WRITES, ids=[str(c) for c in WRITES])
def test_write_and_read_back(case):
    """Several writes one after the other (the later ones larger, so that scales grow inside
    a page), uneven counts with an empty sequence, then every token read back."""
    N, Hk, P, d, T, dtype, fmt, order, starts = case
    rng = np.random.default_rng(T * 1000 + P + d)
    S = (max(starts) + 3 * T) // P + 2
    c = co.Cache(N, Hk, P, d, S, fmt, rng)
    pos = np.array(starts[:N])
    for n in range(N):  # the tokens before the first write
        if pos[n]:
            for x in "kv":
                c.write(x, n, 0, (0.1 * rng.standard_normal((Hk, pos[n], d))).astype(np.float32))
    dev = Dev(c)
    for step, amp in enumerate((0.5, 3.0, 40.0)):
        k, kn = dev_rows(amp * rng.standard_normal((N, Hk, T, d)), dtype, order)
        v, vn = dev_rows(amp * rng.standard_normal((N, Hk, T, d)) * (rng.random((N, Hk, T, 1)) < 0.8), dtype, order)
        count = None if step == 0 else [T if n % 2 == step % 2 else T // 2 for n in range(N)]
        dev.write(k, v, dtype, pos, count)
        cn = [T] * N if count is None else count
        for n in range(N):
            c.write("k", n, int(pos[n]), kn[n, :, :cn[n]])
            c.write("v", n, int(pos[n]), vn[n, :, :cn[n]])
        pos = pos + np.array(cn)
        assert_same_cache(dev, c, [range(p) for p in pos])
    Tr = int(pos.max()) + 2
    for rdt in ("f32", "bf16"):
        got = dev.read(Tr, rdt, np.zeros(N), pos.astype(np.int32), order)
        for g, x in zip(got, "kv"):
            for n in range(N):
                want = c.read(x, n, np.arange(pos[n]))
                np.testing.assert_array_equal(g[n, :, :pos[n]], want)
                assert (g[n, :, pos[n]:] == 0).all()
    # a window of positions somewhere inside
    start = np.maximum(pos - T - 1, 0)
    got = dev.read(T + 1, "f32", start, (pos - start).astype(np.int32))
    for n in range(N):
        np.testing.assert_array_equal(got[1][n, :, :pos[n] - start[n]], c.read("v", n, np.arange(start[n], pos[n])))


@pytest.mark.parametrize("layout,rot", [("half", 128), ("half", 44), ("interleaved", 90), ("half", 32)])
@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
def test_write_rotates_keys(layout, rot, fmt):
    N, Hk, P, d, T = 2, 2, 32, 128, 70
    rng = np.random.default_rng(rot)
    c = co.Cache(N, Hk, P, d, 6, fmt, rng)
    dev = Dev(c)
    rope, th = make_rope(rot, layout, "parts", 8.0, 1.1)
    k, kn = dev_rows(rng.standard_normal((N, Hk, T, d)), "bf16", "blhd")
    v, vn = dev_rows(rng.standard_normal((N, Hk, T, d)), "bf16", "blhd")
    pos = np.array([7 + P * 10 ** 6, 0])
    # the rows before token 7 of the first page: written from a fresh page start
    pre, pn = dev_rows(rng.standard_normal((N, Hk, 7, d)), "bf16")
    dev.write(pre, pre, "bf16", pos - [7, 0], [7, 0])
    dev.write(k, v, "bf16", pos, rope=rope)
    got = dev.read(T, "f32", pos)
    for n in range(N):
        want = co.rotate(kn[n], pos[n] + np.arange(T), th, layout, 1.1)
        s = dev.ks.cpu().numpy()[c.table[n, (pos[n] + np.arange(T)) // P % c.S]].T[:, :, None]  # [Hk,T,1]
        half = np.maximum(np.abs(want) * 2.0 ** -4, s * 2.0 ** -10) if fmt == "e4m3" else s / 2
        err = np.abs(got[0][n] - want)
        assert (err <= half * 1.001 + 2.0 ** -20 * np.abs(want).max()).all()
        c.write("v", n, int(pos[n]) - 7 * (n == 0), np.concatenate([pn[n], vn[n]], 1) if n == 0 else vn[n])
        np.testing.assert_array_equal(got[1][n], c.read("v", n, pos[n] + np.arange(T)))


def test_ring_of_pages_and_rewriting():
    """A table shorter than the context is a ring; tokens may be written again from an earlier
    position (rejected drafts)."""
    N, Hk, P, d = 1, 2, 16, 64
    rng = np.random.default_rng(3)
    c = co.Cache(N, Hk, P, d, 3, "e4m3", rng)
    dev = Dev(c)
    pos = 0
    for T, back in ((10, 0), (14, 4), (16, 0), (1, 0), (30, 7), (48, 48 - 16), (9, 2)):
        pos -= back
        x, xn = dev_rows(rng.standard_normal((N, Hk, T, d)) * rng.choice([0.1, 10.0]), "f32")
        fits = (pos + T - 1) // P - pos // P < 3
        dev.write(x, x, "f32", [pos], ok=fits)
        if not fits:
            continue
        for n in "kv":
            c.write(n, 0, pos, xn[0])
        pos += T
        lo = max(0, ((pos - 1) // P - 2) * P)
        lo = max(lo, pos - 2 * P)
        assert_same_cache(dev, c, [range(lo, pos)])


def test_non_finite_values_are_flagged():
    N, Hk, P, d = 1, 1, 16, 64
    for fmt, big in (("e4m3", 448.0), ("i8", 127.0)):
        c = co.Cache(N, Hk, P, d, 2, fmt, np.random.default_rng(1))
        dev = Dev(c)
        x = np.ones((1, 1, 3, d), np.float32)
        x[0, 0, 1, 3], x[0, 0, 1, 4], x[0, 0, 2, 5] = np.nan, np.inf, -np.inf
        t, _ = dev_rows(x, "f32")
        ones, _ = dev_rows(np.ones((1, 1, 3, d)), "f32")
        dev.write(t, ones, "f32", [0], ok=False)
        k, v = dev.read(3, "f32", [0])
        s = co.scale_of(1.0, fmt)
        want = np.clip(np.nan_to_num(x.astype(np.float64), nan=0.0, posinf=1e9, neginf=-1e9), -big * s, big * s)
        np.testing.assert_array_equal(k, want)
        assert (v == 1).all()


def test_bad_positions_counts_and_pages_are_skipped_and_flagged():
    N, Hk, P, d, T = 5, 1, 16, 64, 4
    rng = np.random.default_rng(2)
    c = co.Cache(N, Hk, P, d, 2, "i8", rng)
    c.table[3] = [c.pages, -1]
    dev = Dev(c)
    before = dev.k.cpu().numpy().copy()
    x, xn = dev_rows(rng.standard_normal((N, Hk, T, d)), "f32")
    pos, cnt = [-1, 0, 0, 3, 8], [4, 5, -2, 4, 4]
    dev.write(x, x, "f32", pos, cnt, ok=False)
    c.write("k", 4, 8, xn[4])
    after = dev.k.cpu().numpy()
    own = c.table[4, 0]
    mask = np.ones(len(after), bool)
    mask[own] = False
    np.testing.assert_array_equal(after[mask], before[mask])
    np.testing.assert_array_equal(after[own][:, 8:12], c.codes["k"][own][:, 8:12])
    k, _ = dev.read(T, "f32", pos, cnt, ok=False)
    assert (k[:4] == 0).all() and (k[4] != 0).any()


# ---------------------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------------------
ATTN = [  # N, H, Hk, P, d, T, dtype, fmt, pos, W, M, rope, first, add, order
    (1, 1, 1, 16, 64, 1, "bf16", "e4m3", [0], 0, 0, False, None, False, "bhld"),
    (2, 4, 2, 64, 128, 1, "bf16", "e4m3", [500, 63], 0, 0, True, None, False, "bhld"),
    (2, 4, 4, 16, 64, 1, "f32", "i8", [33, 200], 0, 3, True, None, True, "blhd"),
    (3, 6, 2, 32, 128, 5, "bf16", "i8", [0, 31, 90], 0, 0, True, None, False, "blhd"),
    (2, 8, 1, 128, 128, 3, "f32", "e4m3", [250, 128], 17, 4, False, None, True, "bhld"),
    (4, 2, 2, 16, 64, 2, "f32", "e4m3", [40, 41, 42, 3], 0, 0, False, [0, 100, 42, 2], False, "bhld"),
    (4, 2, 1, 16, 64, 2, "bf16", "i8", [40, 41, 42, 3], 1, 2, True, [0, 100, 42, -5], True, "bhld"),
    (1, 3, 3, 64, 64, 70, "bf16", "e4m3", [1], 0, 0, True, None, False, "blhd"),
    (1, 4, 2, 64, 128, 130, "bf16", "e4m3", [77], 40, 4, False, None, True, "blhd"),
    (2, 2, 1, 128, 128, 33, "f32", "i8", [300, 7], 0, 1, True, None, False, "bhld"),
    (2, 16, 2, 32, 64, 9, "bf16", "e4m3", [64, 600], 100, 0, True, [0, 3], False, "bhld"),
    (1, 12, 1, 16, 128, 40, "f32", "e4m3", [200], 0, 0, False, None, False, "bhld"),
    (2, 10, 2, 64, 128, 200, "bf16", "i8", [20, 300], 0, 7, True, [0, 360], True, "blhd"),
]


def run_attn(case, count=None, spread=1.0, junk_scale=True, alpha=0.7, seed=None):
    import torch
    N, H, Hk, P, d, T, dtype, fmt, pos, W, M, rope, first, add, order = case
    rng = np.random.default_rng(seed if seed is not None else N * 1000 + T * 10 + W + d)
    span = max(pos) + T if not W else W + T - 1
    S = min((max(pos) + T - 1) // P + 1, (span + P - 2) // P + 1) if W else (max(pos) + T - 1) // P + 1
    c = co.Cache(N, Hk, P, d, S, fmt, rng)
    cnt = [T] * N if count is None else count
    for n in range(N):
        lo = max(0, pos[n] - W + 1) // P * P if W else 0
        L = pos[n] + cnt[n] - lo
        if L > 0:
            amp = spread ** rng.standard_normal((Hk, L, 1))
            c.write("k", n, lo, (rng.standard_normal((Hk, L, d)) * np.exp(0.5 * rng.standard_normal(d))).astype(np.float32))
            c.write("v", n, lo, (amp * rng.standard_normal((Hk, L, d))).astype(np.float32))
    dev = Dev(c)
    r, th = make_rope(d // 2 if P == 32 else d, "interleaved" if P == 32 else "half") if rope else (None, None)
    q, qn = dev_rows(1.5 * rng.standard_normal((N, H, T, d)), dtype, order)
    ya, yan = dev_rows(rng.standard_normal((N, H, T, d)), dtype, order) if add else (None, None)
    mk, mkn = dev_rows(rng.standard_normal((1, H, M, d)), dtype) if M else (None, None)
    mv, mvn = dev_rows(rng.standard_normal((1, H, M, d)), dtype) if M else (None, None)
    dims = lz.lizard_cache_attn_dims(H, T, M, W, DT[dtype], 0.0, alpha)
    ws = torch.zeros(lz.lizard_cache_attn_workspace_bytes(dev.h, dims), dtype=torch.uint8, device="cuda")
    y = torch.full_like(q, 9.0)
    args = (dev.h, dims, q, r, ints(pos, 8), ints(count, 4), ints(first, 8), mk[0] if M else None,
            mv[0] if M else None)
    lz.lizard_cache_attn(*args, ya, y, ws)
    assert lz.lizard_check_device_errors(ws) == 0
    want, A, Z = co.attend(c, qn, pos, count, W, first, mkn[0] if M else None, mvn[0] if M else None, yan, alpha,
                           rope=(th, "interleaved" if P == 32 else "half", 1.0) if rope else None)
    got = y.float().cpu().numpy().astype(np.float64)
    bound = co.attend_bound(want, A, Z, dtype, d, max(pos) + T + M)
    if add:
        bound = bound + 2.0 ** -23 * np.abs(yan)
    err = np.abs(got - want)
    assert np.isfinite(got).all()
    assert (err <= bound).all(), (float(err.max()), float((err / bound).max()))
    # once more: the workspace is as it was, results are bit for bit the same
    y2 = torch.full_like(q, 9.0)
    lz.lizard_cache_attn(*args, ya, y2, ws)
    assert torch.equal(y, y2)
    if add and alpha == 0.7:  # added in place
        lz.lizard_cache_attn(*args, ya, ya, ws)
        assert torch.equal(ya, y)
    return got


@pytest.mark.parametrize("case", ATTN, ids=[str(c) for c in ATTN])
def test_attention(case):
    run_attn(case)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_uneven_counts(dtype):
    case = (4, 4, 2, 16, 64, 6, dtype, "e4m3", [0, 17, 100, 5], 0, 0, True, None, False, "bhld")
    got = run_attn(case, count=[6, 0, 3, 1])
    for n, k in enumerate([6, 0, 3, 1]):
        assert (got[n, :, k:] == 0).all()


@pytest.mark.parametrize("T", [1, 150])
@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
def test_attention_pages_of_very_different_scale(T, fmt):
    """Values whose pages differ by factors up to about 2^30."""
    run_attn((1, 4, 2, 16, 128, T, "bf16", fmt, [150], 0, 2, False, None, False, "bhld"), spread=50.0)


@pytest.mark.parametrize("T,H", [(1, 8), (140, 4)])
def test_attention_long_and_uneven_batch(T, H):
    pos = [1, 700, 0, 2100, 64, 63, 1500]
    run_attn((7, H, 2, 64, 64, T, "bf16", "e4m3", pos, 0, 0, True, None, False, "blhd"))


def test_attention_alpha_zero_and_strong_logits():
    run_attn((1, 2, 1, 16, 64, 1, "bf16", "i8", [50], 0, 0, False, None, True, "bhld"), alpha=0.0)
    # one key far above the others
    run_attn((1, 2, 1, 64, 64, 2, "f32", "e4m3", [400], 0, 1, False, None, False, "bhld"), alpha=-2.0, seed=77)


def test_attention_skips_bad_pages_and_flags_them():
    import torch
    N, H, Hk, P, d = 3, 2, 1, 16, 64
    rng = np.random.default_rng(8)
    for T in (1, 140):
        c = co.Cache(N, Hk, P, d, 12, "e4m3", rng)
        for n in range(N):
            for x in "kv":
                c.write(x, n, 0, rng.standard_normal((Hk, 40 + T, d)))
        dev = Dev(c)
        bad = c.table.copy()
        bad[1, 1] = c.pages + 5
        dev.table.copy_(torch.from_numpy(bad))
        q, qn = dev_rows(rng.standard_normal((N, H, T, d)), "bf16")
        dims = lz.lizard_cache_attn_dims(H, T, 0, 0, lz.LIZARD_BF16, 0.0, 1.0)
        ws = torch.zeros(lz.lizard_cache_attn_workspace_bytes(dev.h, dims), dtype=torch.uint8, device="cuda")
        y = torch.full_like(q, 9.0)
        # sequence 2 lies beyond its table
        pos = [40, 40, 12 * P]
        lz.lizard_cache_attn(dev.h, dims, q, None, ints(pos, 8), None, None, None, None, None, y, ws)
        assert lz.lizard_check_device_errors(ws) == lz.LizardError(5, "").status
        got = y.float().cpu().numpy().astype(np.float64)
        want, A, Z = co.attend(c, qn[:1], pos[:1], None)
        assert (np.abs(got[:1] - want) <= co.attend_bound(want, A, Z, "bf16", d, 180)).all()
        # sequence 1 without tokens 16..31
        ref = np.zeros((H, d))
        toks = np.array([t for t in range(41) if not 16 <= t < 32])
        K, V = c.read("k", 1, toks)[0], c.read("v", 1, toks)[0]
        for h in range(H):
            z = K @ qn[1, h, 0] / np.sqrt(d)
            p = np.exp(z - z.max())
            ref[h] = p / p.sum() @ V
        np.testing.assert_allclose(got[1, :, 0], ref, atol=2e-2)
        assert (got[2] == 0).all()
        dev.table.copy_(torch.from_numpy(c.table))
        lz.lizard_cache_attn(dev.h, dims, q, None, ints([40] * 3, 8), None, None, None, None, None, y, ws)
        assert lz.lizard_check_device_errors(ws) == 0


def test_other_stream_and_graph_capture():
    """write + attention + position advance captured into a CUDA graph on a side stream and
    replayed give what eager calls give."""
    import torch
    N, H, Hk, P, d, S = 2, 4, 2, 16, 64, 8
    rng = np.random.default_rng(4)
    c = co.Cache(N, Hk, P, d, S, "e4m3", rng)
    outs = []
    toks = [torch.from_numpy(rng.standard_normal((3, N, Hk, 1, d)).astype(np.float32)).cuda() for _ in range(8)]
    qs = [torch.from_numpy(rng.standard_normal((N, H, 1, d)).astype(np.float32)).cuda() for _ in range(8)]
    rope, _ = make_rope(d)
    for graph in (False, True):
        dev = Dev(c)
        pos = torch.zeros(N, dtype=torch.int64, device="cuda")
        dims = lz.lizard_cache_attn_dims(H, 1, 0, 0, lz.LIZARD_F32, 0.0, 1.0)
        ws = torch.zeros(lz.lizard_cache_attn_workspace_bytes(dev.h, dims), dtype=torch.uint8, device="cuda")
        k, v, q, y = toks[0][0].clone(), toks[0][1].clone(), qs[0].clone(), torch.empty_like(qs[0])
        io = lz.lizard_cache_io(1, lz.LIZARD_F32)
        side = torch.cuda.Stream()

        def step():
            lz.lizard_cache_write(dev.h, io, k, v, rope, pos, None, dev.ws)
            lz.lizard_cache_attn(dev.h, dims, q, rope, pos, None, None, None, None, None, y, ws)
            pos.add_(1)

        got = []
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            if graph:
                step()  # first launches (module loading) happen outside the capture
                pos.zero_()
        side.synchronize()
        g = None
        if graph:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                step()
        for i in range(8):
            with torch.cuda.stream(side):
                k.copy_(toks[i][0]), v.copy_(toks[i][1]), q.copy_(qs[i])
                g.replay() if graph else step()
                got.append(y.clone())
        side.synchronize()
        assert pos.tolist() == [8] * N
        outs.append(torch.stack(got))
    assert torch.equal(*outs)


def test_no_tokens_is_a_no_op():
    import torch
    c = co.Cache(1, 1, 16, 64, 2, "e4m3", np.random.default_rng(0))
    dev = Dev(c)
    dims = lz.lizard_cache_attn_dims(1, 0, 0, 0, lz.LIZARD_F32, 0.0, 1.0)
    e = torch.empty(1, 1, 0, 64, device="cuda")
    ws = torch.zeros(max(256, lz.lizard_cache_attn_workspace_bytes(dev.h, dims)), dtype=torch.uint8, device="cuda")
    lz.lizard_cache_attn(dev.h, dims, e, None, ints([0], 8), None, None, None, None, None, e.clone(), ws)
    assert lz.lizard_last_launch_count() == 0
    lz.lizard_cache_write(dev.h, lz.lizard_cache_io(0, lz.LIZARD_F32), e, e, None, ints([0], 8), None, dev.ws)
    assert lz.lizard_last_launch_count() == 0


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
def test_pages_beyond_32_bits(fmt):
    """The same tokens in pages at the start of a small pool and at the end of one whose codes
    pass 2^32 bytes: writes, reads and both attention paths give the same bits."""
    import torch
    N, H, Hk, P, d, S = 2, 8, 2, 128, 128, 3
    big = 2 ** 32 // (Hk * P * d) + N * S
    rng = np.random.default_rng(12)
    rows = [dev_rows(rng.standard_normal((N, Hk, 300, d)), "bf16")[0] for _ in "kv"]
    pos = torch.tensor([0, 50], device="cuda")
    outs = []
    for pages in (N * S, big):
        codes = [torch.empty(pages, Hk, P, d, dtype=torch.uint8, device="cuda") for _ in "kv"]
        scales = [torch.empty(pages, Hk, device="cuda") for _ in "kv"]
        table = (pages - N * S + torch.randperm(N * S, generator=torch.Generator().manual_seed(1)).to(torch.int32))
        table = table.view(N, S).cuda()
        cache = lz.lizard_cache(*codes, *scales, table, FMT[fmt])
        ws = torch.zeros(lz.lizard_cache_workspace_bytes(), dtype=torch.uint8, device="cuda")
        lz.lizard_cache_write(cache, lz.lizard_cache_io(300, lz.LIZARD_BF16), *rows, None, pos, None, ws)
        back = [torch.empty(N, Hk, 300, d, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        lz.lizard_cache_read(cache, lz.lizard_cache_io(300, lz.LIZARD_BF16), pos, None, *back, ws)
        assert lz.lizard_check_device_errors(ws) == 0
        got = back
        for T in (1, 40):
            q = dev_rows(np.random.default_rng(T).standard_normal((N, H, T, d)), "bf16")[0]
            first, at = pos, pos + 300 - T
            dims = lz.lizard_cache_attn_dims(H, T, 0, 0, lz.LIZARD_BF16, 0.0, 1.0)
            aws = torch.zeros(lz.lizard_cache_attn_workspace_bytes(cache, dims), dtype=torch.uint8, device="cuda")
            y = torch.empty_like(q)
            lz.lizard_cache_attn(cache, dims, q, None, at, None, first, None, None, None, y, aws)
            assert lz.lizard_check_device_errors(aws) == 0
            got = got + [y]
        outs.append(got)
        del codes, cache
    for a, b in zip(*outs):
        assert torch.isfinite(a.float()).all()
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,G", [(1, 4), (80, 1)])
def test_attention_of_a_long_context(T, G):
    """40000 tokens (many parts to be joined), against fp64 on the same cache values."""
    import torch
    Hk, P, d, L = 2, 64, 128, 40000
    H, S = Hk * G, (L + T) // P + 1
    g = torch.Generator(device="cuda").manual_seed(5)
    codes = [torch.empty(S, Hk, P, d, dtype=torch.uint8, device="cuda") for _ in "kv"]
    scales = [torch.empty(S, Hk, device="cuda") for _ in "kv"]
    cache = lz.lizard_cache(*codes, *scales, torch.randperm(S, generator=g, device="cuda").to(torch.int32)[None], 0)
    ws = torch.zeros(lz.lizard_cache_workspace_bytes(), dtype=torch.uint8, device="cuda")
    rows = [torch.randn(1, Hk, L + T, d, generator=g, device="cuda") for _ in "kv"]
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    io = lz.lizard_cache_io(L + T, lz.LIZARD_F32)
    lz.lizard_cache_write(cache, io, *rows, None, zero, None, ws)
    lz.lizard_cache_read(cache, io, zero, None, *rows, ws)
    for dtype, dt in (("f32", torch.float32), ("bf16", torch.bfloat16)):
        q = (1.5 * torch.randn(1, H, T, d, generator=g, device="cuda")).to(dt)
        dims = lz.lizard_cache_attn_dims(H, T, 0, 0, DT[dtype], 0.0, 1.0)
        aws = torch.zeros(lz.lizard_cache_attn_workspace_bytes(cache, dims), dtype=torch.uint8, device="cuda")
        y = torch.empty_like(q)
        lz.lizard_cache_attn(cache, dims, q, None, zero + L, None, None, None, None, None, y, aws)
        assert lz.lizard_check_device_errors(aws) == 0
        k, v = (x[0].double().repeat_interleave(G, 0) for x in rows)
        z = q[0].double() @ k.transpose(1, 2) / d ** 0.5
        hide = torch.arange(L + T, device="cuda") > L + torch.arange(T, device="cuda")[:, None]
        p = torch.softmax(z.masked_fill(hide, -float("inf")), -1)
        want, A = p @ v, p @ v.abs()
        Z = (q[0].double().abs() @ k.abs().transpose(1, 2)).amax(-1, keepdim=True) / d ** 0.5
        bound = co.attend_bound(want.cpu().numpy(), A.cpu().numpy(), Z.cpu().numpy(), dtype, d, L + T)
        assert ((y[0].double() - want).abs().cpu().numpy() <= bound).all()
