"""The linear attention with a decay per head on the GPU against the recurrence in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

import decay_oracle as do
import hybrid_gated_linear_gb300 as lz

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CODE = {torch.bfloat16: lz.LIZARD_BF16, torch.float32: lz.LIZARD_F32}
INF = float("inf")


def rows(shape, dtype, gen, order="bhld"):
    B, H, L, d = shape
    x = torch.randn(shape if order == "bhld" else (B, L, H, d), generator=gen).to(dtype).cuda()
    return x if order == "bhld" else x.permute(0, 2, 1, 3)


class In:
    """Inputs of one call; log decays between about -3 and -0.01."""

    def __init__(self, B, H, Hk, L, dk, dv, dtype, order="bhld", state=True, seed=0):
        g = torch.Generator().manual_seed(seed + 1000 * L + dk + 7 * dv + H)
        self.dims = lz.lizard_decay_dims(B, H, Hk, L, dk, dv, CODE[DT[dtype]], 0.0)
        t = DT[dtype]
        self.q, self.k = rows((B, H, L, dk), t, g, order), rows((B, Hk, L, dk), t, g, order)
        self.v, self.dy = rows((B, Hk, L, dv), t, g, order), rows((B, H, L, dv), t, g, order)
        rate = torch.linspace(-4, 1, H)[None, :, None]
        self.g = -torch.nn.functional.softplus(rate + torch.randn(B, H, L, generator=g)).cuda()
        self.h0 = torch.randn(B, H, dk, dv, generator=g).cuda() if state else None
        self.df = torch.randn(B, H, dk, dv, generator=g).cuda() if state else None
        self.count = None

    def case(self, bwd=False):
        d = self.dims
        return do.Case(self.q, self.k, self.v, self.g, self.count, self.h0, self.dy if bwd else None, self.df, d.scale)

    def counts(self):
        return None if self.count is None else torch.tensor(self.count, dtype=torch.int32, device="cuda")

    def terms(self):
        d = self.dims
        return do.terms(d.L, d.dk, d.dv, d.H // d.Hk)

    def fwd(self, final=True, ws=None, status=0, stream=None, y=None):
        d = self.dims
        ws = workspace(d, False) if ws is None else ws
        y = torch.full_like(self.dy, 9.0) if y is None else y
        h = torch.full((d.B, d.H, d.dk, d.dv), 9.0, device="cuda") if final else None
        lz.lizard_decay_attn_fwd(d, self.q, self.k, self.v, self.g, self.counts(), self.h0, y, h, ws, stream=stream)
        if status is not None:
            assert lz.lizard_check_device_errors(ws) == status
        return y, h

    def bwd(self, gate=True, d_h0=True, ws=None, status=0):
        d = self.dims
        ws = workspace(d, True) if ws is None else ws
        out = [torch.full_like(x, 9.0) for x in (self.q, self.k, self.v)]
        dg = torch.full((d.B, d.H, d.L), 9.0, device="cuda") if gate else None
        dh = torch.full((d.B, d.H, d.dk, d.dv), 9.0, device="cuda") if d_h0 else None
        lz.lizard_decay_attn_bwd(d, self.q, self.k, self.v, self.g, self.counts(), self.h0, self.dy, self.df, *out, dg, dh, ws)
        if status is not None:
            assert lz.lizard_check_device_errors(ws) == status
        return (*out, dg, dh)

    def gradients(self):
        """d_q, d_k, d_v alone, into contiguous rows (inputs may repeat: the caller sums)."""
        d = self.dims
        out = [torch.full(t.shape, 9.0, dtype=t.dtype, device="cuda") for t in (self.q, self.k, self.v)]
        lz.lizard_decay_attn_bwd(d, self.q, self.k, self.v, self.g, self.counts(), self.h0, self.dy, self.df, *out, None, None,
                                 workspace(d, True))
        return out

    def check_fwd(self, **kw):
        y, h = self.fwd(**kw)
        c = self.case()
        do.close(y, c.y, do.bound(c.y, c.y_abs, y.dtype, self.terms()))
        if h is not None:  # fp32 whatever the inputs' type
            do.close(h, c.h, do.bound(c.h, c.h_abs, torch.float32, self.terms()))
        return y, h

    def check_bwd(self, **kw):
        got = self.bwd(**kw)
        c = self.case(True)
        for x, want, s in zip(got[:3], c.grads, c.sums):
            do.close(x, want, do.bound(want, s, x.dtype, self.terms()))
        if got[4] is not None:
            do.close(got[4], c.grads[4], do.bound(c.grads[4], c.sums[4], torch.float32, self.terms()))
        if got[3] is not None:
            # sums of products over every pair of tokens around a token: the fp32 rule of this library
            assert torch.isfinite(got[3]).all()
            assert do.rel_l2(got[3], c.grads[3]) <= 1e-5, do.rel_l2(got[3], c.grads[3])
        return got


def workspace(dims, bwd):
    return torch.zeros(lz.lizard_decay_attn_workspace_bytes(dims, bwd), dtype=torch.uint8, device="cuda")


SIZES = [(1, 1, 1, 1, 64, 64), (2, 2, 1, 2, 64, 128), (1, 4, 2, 63, 128, 64), (2, 3, 3, 64, 128, 128),
         (1, 6, 2, 65, 64, 64), (1, 2, 2, 127, 64, 128), (2, 2, 1, 128, 128, 128), (1, 3, 1, 129, 128, 64),
         (3, 2, 2, 255, 64, 64), (1, 2, 2, 257, 128, 128), (1, 4, 1, 300, 128, 128), (1, 1, 1, 519, 64, 128)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward(size, dtype):
    In(*size, dtype).check_fwd()
    In(*size, dtype, order="blhd", state=False, seed=5).check_fwd(final=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_backward(size, dtype):
    In(*size, dtype).check_bwd()
    In(*size, dtype, order="blhd", state=False, seed=5).check_bwd(d_h0=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_backward_without_what_is_not_wanted(dtype):
    x = In(2, 4, 2, 150, 64, 64, dtype)
    a = x.check_bwd()
    for kw in (dict(gate=False), dict(d_h0=False), dict(gate=False, d_h0=False)):
        # (bf16 calls round operands that no fp32 result is made of: other bits, within the bound)
        for p, q in zip(a, x.check_bwd(**kw)):
            assert q is None or dtype == "bf16" or torch.equal(p, q)
    x.df = None
    x.check_bwd()
    x.h0, x.df = None, torch.randn(2, 4, 64, 64, device="cuda")
    x.check_bwd()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("count", [[0, 300, 131, 64], [1, 128, 129, 0], [300, 299, 2, 127]])
def test_uneven_lengths(dtype, count):
    x = In(4, 4, 2, 300, 64, 128, dtype)
    x.count = count
    clean = x.fwd(), x.bwd()
    for b, c in enumerate(count):  # what lies behind a sequence is not read as tokens
        for t in (x.q, x.k, x.v, x.dy):
            t[b, :, c:] = float("nan")
        x.g[b, :, c:] = float("nan")
    for got in (x.check_fwd(), x.check_bwd()):
        for p, q in zip(got, clean[len(got) > 2]):
            assert torch.equal(p, q)
    y, h = x.fwd()
    for b, c in enumerate(count):
        assert (y[b, :, c:] == 0).all()
        for t in x.bwd()[:4]:
            assert (t[b, :, c:] == 0).all()
    assert torch.equal(h[count.index(0)], x.h0[count.index(0)]) if 0 in count else True


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_documents(dtype):
    """Resets at a row's first and last token, at neighbours, at chunks' ends and starts, and none."""
    x = In(2, 4, 2, 400, 128, 64, dtype)
    for h, at in enumerate([(0, 399), (17, 18, 19, 200), (63, 64, 127, 128, 129, 255, 256), ()]):
        for t in at:
            x.g[0, h, t] = -INF
    x.check_fwd()
    got = x.check_bwd()
    assert (got[3][x.g == -INF] == 0).all()
    # a row of one-token documents sees only itself
    x.g[1] = -INF
    y, h = x.check_fwd()
    k, v = (t[1].repeat_interleave(2, 0).double() for t in (x.k, x.v))
    alone = (x.q[1].double() * k).sum(-1, keepdim=True) * v / 128 ** 0.5
    s = (x.q[1].double().abs() * k.abs()).sum(-1, keepdim=True) * v.abs() / 128 ** 0.5
    do.close(y[1], alone.cpu(), do.bound(alone, s, y.dtype, x.terms()).cpu())
    assert (x.check_bwd()[3][1] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("decay", [0.0, -1e-7, -0.05, -3.0, -60.0, -1e5, 0.02])
def test_constant_decays_of_any_size(dtype, decay):
    """One number per head, repeated by strides of 0; none, weak, strong, and a growing state."""
    x = In(1, 2, 2, 333, 64, 64, dtype)
    x.g = (torch.tensor([decay, decay / 2], device="cuda"))[None, :, None].expand(1, 2, 333)
    x.check_fwd()
    got, c = x.bwd(), x.case(True)
    for p, want, s in zip(got[:3], c.grads, c.sums):
        do.close(p, want, do.bound(want, s, p.dtype, x.terms()))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_mixed_decays(dtype):
    """Strong and weak decays side by side, finite ones far below what fp32 can resolve."""
    x = In(1, 3, 3, 300, 128, 128, dtype)
    x.g[0, 0, ::3] = -40.0
    x.g[0, 1, 100:140] = -3e38
    x.g[0, 2] = 0.0
    x.g[0, 2, 150] = -200.0
    x.check_fwd()
    x.check_bwd()


def test_strided_and_broadcast_inputs():
    """Slices of one packed projection, queries shared by all heads, decays of their own layout."""
    B, H, L, d = 2, 4, 140, 64
    gen = torch.Generator().manual_seed(9)
    for dtype in ("bf16", "f32"):
        packed = torch.randn(B, L, 3 * H, d, generator=gen).to(DT[dtype]).cuda().permute(0, 2, 1, 3)
        x = In(B, H, H, L, d, d, dtype)
        x.q, x.k, x.v = packed[:, :H], packed[:, H:2 * H], packed[:, 2 * H:]
        x.g = x.g.permute(0, 2, 1).contiguous().permute(0, 2, 1)
        x.check_fwd()
        x.check_bwd()
        x.q = x.q[:, :1].expand(B, H, L, d)
        c = x.case(True)
        y, _ = x.fwd()
        do.close(y, c.y, do.bound(c.y, c.y_abs, y.dtype, x.terms()))
        dq = torch.empty(B, H, L, d, dtype=DT[dtype], device="cuda")  # per head: the caller sums
        dk, dv, ws = torch.empty_like(dq), torch.empty_like(dq), workspace(x.dims, True)
        lz.lizard_decay_attn_bwd(x.dims, x.q, x.k, x.v, x.g, None, x.h0, x.dy, x.df, dq, dk, dv, None, None, ws)
        for p, want, s in zip((dq, dk, dv), c.grads, c.sums):
            do.close(p, want, do.bound(want, s, p.dtype, x.terms()))
        # one row for every token
        x.v = x.v[:, :, :1].expand(B, H, L, d)
        x.check_fwd()


def test_outputs_in_place_of_a_packed_gradient():
    B, H, L, d = 1, 2, 130, 64
    x = In(B, H, H, L, d, d, "bf16")
    want = x.bwd(gate=False, d_h0=False)[:3]
    packed = torch.full((B, L, 3 * H, d), 9.0, dtype=torch.bfloat16, device="cuda").permute(0, 2, 1, 3)
    out = packed[:, :H], packed[:, H:2 * H], packed[:, 2 * H:]
    lz.lizard_decay_attn_bwd(x.dims, x.q, x.k, x.v, x.g, None, x.h0, x.dy, x.df, *out, None, None, workspace(x.dims, True))
    for p, q in zip(out, want):
        assert torch.equal(p, q)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_pieces_join(dtype):
    """A prompt in pieces through the states, then single tokens, is the prompt in one piece."""
    x = In(2, 4, 2, 390, 128, 64, dtype)
    want = x.case()
    limit = do.bound(want.y, want.y_abs, DT[dtype], 2 * x.terms())
    h = x.h0.clone()
    for a, b in ((0, 129), (129, 130), (130, 386)):
        d = lz.lizard_decay_dims(2, 4, 2, b - a, 128, 64, x.dims.dtype, 0.0)
        y, nxt = torch.empty(2, 4, b - a, 64, dtype=DT[dtype], device="cuda"), torch.empty_like(h)
        lz.lizard_decay_attn_fwd(d, x.q[:, :, a:b], x.k[:, :, a:b], x.v[:, :, a:b], x.g[:, :, a:b], None, h, y, nxt, workspace(d, False))
        do.close(y, want.y[:, :, a:b], limit[:, :, a:b])
        h = nxt
    for a, b in ((386, 387), (387, 390)):
        d = lz.lizard_decay_dims(2, 4, 2, b - a, 128, 64, x.dims.dtype, 0.0)
        y = torch.empty(2, 4, b - a, 64, dtype=DT[dtype], device="cuda")
        lz.lizard_decay_attn_step(d, x.q[:, :, a:b], x.k[:, :, a:b], x.v[:, :, a:b], x.g[:, :, a:b], h, y)
        do.close(y, want.y[:, :, a:b], limit[:, :, a:b])
    do.close(h, want.h, do.bound(want.h, want.h_abs, torch.float32, 2 * x.terms()))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(1, 1, 1, 1, 64, 64), (1, 32, 8, 1, 128, 128), (3, 5, 5, 1, 128, 64), (2, 6, 2, 4, 64, 128),
                                  (40, 16, 4, 1, 128, 128), (9, 40, 40, 2, 64, 64), (11, 32, 32, 1, 64, 128)], ids=str)
def test_step(size, dtype):
    """Single tokens, fp32 throughout: the states' columns split over CTAs for few heads, not for many."""
    x = In(*size, dtype)
    x.g[0, 0, 0] = -INF
    c = x.case()
    h, y = x.h0.clone(), torch.full_like(x.dy, 9.0)
    lz.lizard_decay_attn_step(x.dims, x.q, x.k, x.v, x.g, h, y)
    limit = torch.finfo(DT[dtype]).eps / 2 * c.y.abs() * 1.001 + x.terms() * 2.0 ** -24 * c.y_abs * 1.01
    do.close(y, c.y, limit)
    do.close(h, c.h, do.bound(c.h, c.h_abs, torch.float32, 16 * size[3]))


def test_bad_counts_are_flagged():
    for dtype in ("bf16", "f32"):
        for bad in (-1, 131, 2 ** 31 - 1):
            x = In(2, 2, 1, 130, 64, 64, dtype)
            x.count = [100, bad]
            y, h = x.fwd(status=5)
            assert (y[1] == 0).all() and torch.equal(h[1], x.h0[1])
            got = x.bwd(status=5)
            assert all((t[1] == 0).all() for t in got[:4]) and torch.equal(got[4][1], x.df[1])
            x.count = [100, 0]
            for p, q in zip((y, h, *got), (*x.check_fwd(), *x.check_bwd())):
                assert torch.equal(p, q)


def test_no_tokens():
    for dtype in ("bf16", "f32"):
        x = In(2, 3, 3, 0, 64, 128, dtype)
        _, h = x.fwd()
        assert torch.equal(h, x.h0)
        assert torch.equal(x.bwd()[4], x.df)
        x.h0 = x.df = None
        _, h = x.fwd()
        assert (h == 0).all() and (x.bwd()[4] == 0).all()


def test_same_bits_on_any_stream_and_in_a_graph():
    for dtype in ("bf16", "f32"):
        x = In(2, 4, 2, 700, 128, 128, dtype)
        want, grads = x.fwd(), x.bwd()
        for _ in range(3):
            assert all(torch.equal(p, q) for p, q in zip(want + grads, x.fwd() + x.bwd()))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        y, h = x.fwd(status=None, stream=side)
        side.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(h, want[1])
        # captured: the forward, the backward and a step after it, replayed over new inputs
        d = x.dims
        y, h = torch.empty_like(x.dy), torch.empty_like(x.h0)
        out = [torch.empty_like(t) for t in (x.q, x.k, x.v)]
        dg, dh = torch.empty_like(x.g), torch.empty_like(h)
        wf, wb = workspace(d, False), workspace(d, True)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            lz.lizard_decay_attn_fwd(d, x.q, x.k, x.v, x.g, None, x.h0, y, h, wf)
            lz.lizard_decay_attn_bwd(d, x.q, x.k, x.v, x.g, None, x.h0, x.dy, x.df, *out, dg, dh, wb)
        for seed in (0, 1):
            z = In(2, 4, 2, 700, 128, 128, dtype, seed=seed)
            for name in ("q", "k", "v", "g", "h0", "dy", "df"):
                getattr(x, name).copy_(getattr(z, name))
            graph.replay()
            for p, q in zip((y, h, *out, dg, dh), z.fwd() + z.bwd()):
                assert torch.equal(p, q)


def test_workspaces_of_other_calls():
    """One workspace, large enough, for calls of other shapes in between."""
    x, z = In(2, 4, 2, 700, 128, 128, "bf16"), In(1, 2, 1, 90, 64, 64, "bf16")
    wf, wb = workspace(x.dims, False), workspace(x.dims, True)
    first = x.fwd(ws=wf) + x.bwd(ws=wb)
    other = z.fwd(ws=wf) + z.bwd(ws=wb)
    for p, q in zip(first + other, x.fwd(ws=wf) + x.bwd(ws=wb) + z.fwd() + z.bwd()):
        assert torch.equal(p, q)


def on_gpu(x, bwd):
    """The recurrence in 64 bits on the device, for lengths that are too long for the CPU: the same
    formulas, whole heads at a time."""
    d = x.dims
    G = d.H // d.Hk
    q, k, v, dy = x.q.double(), x.k.double().repeat_interleave(G, 1), x.v.double().repeat_interleave(G, 1), x.dy.double()
    g = torch.exp(x.g.double())[..., None, None]
    h = torch.zeros(d.B, d.H, d.dk, d.dv, dtype=torch.float64, device="cuda") if x.h0 is None else x.h0.double()
    hs, y = [h], torch.empty_like(dy)
    for t in range(d.L):
        h = g[:, :, t] * h + k[:, :, t, :, None] * v[:, :, t, None]
        y[:, :, t] = (q[:, :, t, None] @ h)[:, :, 0] * d.dk ** -0.5
        hs.append(h)
    if not bwd:
        return y, h
    dh = torch.zeros_like(h) if x.df is None else x.df.double()
    q = q * d.dk ** -0.5
    dq, dk, dv, dg = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(x.g, dtype=torch.float64)
    for t in range(d.L - 1, -1, -1):
        dh = dh + q[:, :, t, :, None] * dy[:, :, t, None]
        dq[:, :, t] = (hs[t + 1] @ dy[:, :, t, :, None])[..., 0] * d.dk ** -0.5
        dk[:, :, t] = (dh @ v[:, :, t, :, None])[..., 0]
        dv[:, :, t] = (k[:, :, t, None] @ dh)[:, :, 0]
        dg[:, :, t] = (g[:, :, t] * hs[t] * dh).sum((2, 3))
        dh = g[:, :, t] * dh
    dk, dv = (t.unflatten(1, (d.Hk, G)).sum(2) for t in (dk, dv))
    return dq, dk, dv, dg, dh


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(1, 3, 3, 5000, 64, 128), (2, 4, 1, 2500, 128, 64), (1, 2, 2, 8192, 128, 128),
                                  (7, 24, 24, 530, 64, 64)], ids=str)
def test_long_sequences(size, dtype):
    """Many chunks, few heads (the axis is split) and more heads than SMs: relative 2-norms, with one
    rounding to bf16 of the result, one of its summands and none in what is fp32 (half a step each:
    2^-8 at most); fp32 by this library's rule."""
    x = In(*size, dtype)
    x.g[:, 0] *= 0.01  # a state that lasts
    tol = 2 * 2.0 ** -8 if dtype == "bf16" else 1e-5
    y, h = x.fwd()
    want = on_gpu(x, False)
    assert do.rel_l2(y, want[0].cpu()) <= tol and do.rel_l2(h, want[1].cpu()) <= 1e-5
    got = x.bwd()
    want = on_gpu(x, True)
    for p, w, limit in zip(got, want, (tol, tol, tol, 1e-5, 1e-5)):
        assert torch.isfinite(p).all()
        assert do.rel_l2(p, w.cpu()) <= limit, (do.rel_l2(p, w.cpu()), limit)


def test_rows_far_apart():
    """Offsets beyond 32 bits, in elements: 300 rows 2^24 elements apart."""
    x = In(1, 1, 1, 300, 64, 64, "bf16", state=False)
    far = torch.zeros(300 << 24, dtype=torch.bfloat16, device="cuda").view(300, -1)
    where = [far[:, 64 * i:64 * i + 64] for i in range(4)]
    for w, t in zip(where, (x.q, x.k, x.v)):
        w.copy_(t[0, 0])
    want, d = x.fwd(final=False)[0], x.dims
    q, k, v, y = (w[None, None] for w in where)
    lz.lizard_decay_attn_fwd(d, q, k, v, x.g, None, None, y, None, workspace(d, False))
    assert torch.equal(y, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_overlapping_and_repeated_rows(dtype):
    """Inputs whose rows overlap in memory or repeat along any axis: heads 16 channels apart, one sequence
    for all, every token's row 16 channels behind the last."""
    B, H, L, d = 2, 3, 140, 64
    gen = torch.Generator().manual_seed(21)
    flat = torch.randn(B * 100000, generator=gen).to(DT[dtype]).cuda()
    x = In(B, H, H, L, d, d, dtype)
    for strides in ((30000, 16, 64), (30000, 10000, 16), (0, 10000, 64), (0, 0, 64)):
        x.q, x.k, x.v = (flat[16 * i:].as_strided((B, H, L, d), (*strides, 1)) for i in range(3))
        x.check_fwd()
        got, c = x.gradients(), x.case(True)
        for p, want, s in zip(got, c.grads, c.sums):
            do.close(p, want, do.bound(want, s, p.dtype, x.terms()))


def test_two_calls_at_once():
    """Two streams, each with a workspace of its own, over and over: nothing is shared."""
    x, z = In(2, 4, 2, 900, 128, 128, "bf16"), In(3, 6, 6, 300, 64, 128, "f32")
    want = [(x.fwd(), x.bwd()), (z.fwd(), z.bwd())]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, (c, s) in enumerate(zip((x, z), streams)):
            with torch.cuda.stream(s):
                got[i].append((c.fwd(status=None), c.bwd(status=None)))
    torch.cuda.synchronize()
    for i in range(2):
        for pair in got[i]:
            for a, b in zip(want[i], pair):
                assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 7, 15, 16, 17, 24, 25])
def test_a_few_tokens(dtype, L):
    """Short forwards take the single tokens' kernel: counts, documents, states, and the step's own result."""
    x = In(4, 6, 2, L, 128, 64, dtype, order="blhd", seed=11)
    x.g[1, 2, L // 2] = -INF
    x.g[2, 0, 0] = -INF
    whole = x.check_fwd()
    if L <= (16 if dtype == "bf16" else 24):  # token for token the same sums
        h, y = x.h0.clone(), torch.full_like(whole[0], 9.0)
        lz.lizard_decay_attn_step(x.dims, x.q, x.k, x.v, x.g, h, y)
        assert torch.equal(y, whole[0]) and torch.equal(h, whole[1])
    x.check_fwd(final=False)
    x.count = [L, 0, (L + 1) // 2, L - 1]
    clean = x.fwd()
    for b, c in enumerate(x.count):
        for t in (x.q, x.k, x.v):
            t[b, :, c:] = float("nan")
        x.g[b, :, c:] = float("nan")
    assert all(torch.equal(p, q) for p, q in zip(clean, x.check_fwd()))
    assert all((clean[0][b, :, c:] == 0).all() for b, c in enumerate(x.count)) and torch.equal(clean[1][1], x.h0[1])
    for bad in (-1, L + 1):
        x.count[0] = bad
        y, h = x.fwd(status=5)
        assert (y[0] == 0).all() and torch.equal(h[0], x.h0[0])
        assert torch.equal(y[1:], clean[0][1:]) and torch.equal(h[1:], clean[1][1:])
    In(2, 4, 4, L, 64, 128, dtype, state=False, seed=12).check_fwd()
