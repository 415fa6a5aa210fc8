"""Layer norm and its gradients on the GPU against 64 bits, and the linear attention with it behind."""
import pytest

torch = pytest.importorskip("torch")

import decay_oracle as do
import hybrid_gated_linear_gb300 as lz

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CODE = {"bf16": lz.LIZARD_BF16, "f32": lz.LIZARD_F32}


def strands(d):
    """Summands that one thread adds up, and the steps of the sums over threads."""
    return 16 + 10 + 2


class In:
    def __init__(self, N, H, T, d, dtype, per_head=False, order="nhtd", weights=True, seed=0, mean=0.5, eps=1e-5):
        g = torch.Generator().manual_seed(seed + d + T)
        self.dims = lz.lizard_norm_dims(N, H, T, d, int(per_head), CODE[dtype], eps)
        self.eps, self.t = eps, DT[dtype]
        shape = (N, H, T, d) if order == "nhtd" else (N, T, H, d)
        x = (torch.randn(shape, generator=g) * torch.exp(torch.randn(*shape[:3], 1, generator=g)) + mean).to(self.t).cuda()
        dy = torch.randn(shape, generator=g).to(self.t).cuda()
        self.x, self.dy = (x, dy) if order == "nhtd" else (x.permute(0, 2, 1, 3), dy.permute(0, 2, 1, 3))
        w = (H, d) if per_head else (d,)
        self.w = (1 + 0.3 * torch.randn(w, generator=g)).to(self.t).cuda() if weights else None
        self.b = torch.randn(w, generator=g).to(self.t).cuda() if weights else None
        self.per_head = per_head

    def wide(self, w):
        return None if w is None else w[:, None] if self.per_head else w

    def fwd(self, y=None):
        y = torch.full_like(self.x, 9.0) if y is None else y
        lz.lizard_layer_norm_fwd(self.dims, self.x, self.w, self.b, y)
        return y

    def bwd(self, dx=None, ws=None):
        d = self.dims
        dx = torch.full_like(self.x, 9.0) if dx is None else dx
        shape = (d.H, d.d) if self.per_head else (d.d,)
        dw, db = (torch.full(shape, 9.0, device="cuda") for _ in range(2))
        ws = torch.zeros(lz.lizard_layer_norm_workspace_bytes(d), dtype=torch.uint8, device="cuda") if ws is None else ws
        lz.lizard_layer_norm_bwd(d, self.x, self.w, self.dy, dx, dw, db, ws)
        return dx, dw, db

    def check(self):
        d, u = self.dims, 2.0 ** -24
        x = self.x.cpu().double()
        y, n, r = do.norm(self.x, self.wide(self.w), self.wide(self.b), self.eps)
        # the mean is off by u * strands of the mean |x|; what follows is that times r, and r's own error
        # (half that of the variance, and two units of its square root and product)
        s = strands(d.d) * u
        slip = s * x.abs().mean(-1, keepdim=True) * r + 2 * u * n.abs() + 2 * u * x.abs() * r
        dn = slip + n.abs() * (s + 4 * u + 2 * (slip * n.abs()).mean(-1, keepdim=True) + (slip ** 2).mean(-1, keepdim=True))
        w = torch.ones(()).double() if self.w is None else self.wide(self.w).cpu().double()
        b = torch.zeros(()).double() if self.b is None else self.wide(self.b).cpu().double()
        half = torch.finfo(self.t).eps / 2
        lim = dn * w.abs() + 2 * u * ((n * w).abs() + b.abs())
        do.close(self.fwd(), y, half * y.abs() + (1 + half) * lim + 1e-30)
        over = (0, 2) if self.per_head else (0, 1, 2)
        dx, dw, db, (a, n, r) = do.norm_backward(self.x, self.wide(self.w), self.dy, self.eps, over)
        got = self.bwd()
        # d_x: every term with its own error; the two means' by the same count of summands
        da = u * a.abs()
        m0 = (da + s * a.abs()).mean(-1, keepdim=True)
        m1 = (a.abs() * dn + da * n.abs() + (s + u) * (a * n).abs()).mean(-1, keepdim=True)
        inner = da + m0 + n.abs() * m1 + dn * (a * n).mean(-1, keepdim=True).abs() + \
            4 * u * (a.abs() + a.mean(-1, keepdim=True).abs() + (n * (a * n).mean(-1, keepdim=True)).abs())
        rr = (dn / n.abs().clamp(min=1e-3)).amax(-1, keepdim=True)  # r's relative error is part of n's
        lim = r * inner + rr * dx.abs()
        do.close(got[0], dx, half * dx.abs() + (1 + half) * lim + 1e-30)
        # sums over rows: each summand's error, and one rounding for every addition it can be part of
        dy = self.dy.cpu().double()
        rows = x.shape[0] * x.shape[2] * (1 if self.per_head else x.shape[1])
        add = (min(rows, rows // 8 + 64) + 80) * u
        do.close(got[1], dw, (dy.abs() * dn).sum(over) + (add + u) * (dy * n).abs().sum(over) + 1e-30)
        do.close(got[2], db, add * dy.abs().sum(over) + 1e-30)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [8, 16, 24, 64, 72, 128, 136, 256, 264, 504, 512, 520, 1000, 1024, 1032, 2048, 2056, 4096, 5000,
                               8192, 8200, 14336, 16384])
def test_widths(d, dtype):
    In(1, 1, 37, d, dtype).check()
    In(2, 1, 3, d, dtype, weights=False, seed=1).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 64), (2, 5, 33, 64), (3, 4, 70, 128), (1, 33, 129, 128), (2, 3, 9, 1024), (1, 700, 2, 64),
                                   (2, 2, 5, 4096)], ids=str)
def test_heads(shape, dtype):
    for per_head in (True, False):
        for order in ("nhtd", "nthd"):
            In(*shape, dtype, per_head, order).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_large_mean_costs_no_digits(dtype):
    """Rows whose mean is a thousand times their spread, and constant rows: the variance is not the
    difference of two large sums."""
    In(1, 1, 19, 512, dtype, mean=1000.0).check()
    x = In(1, 1, 5, 128, dtype)
    x.x.fill_(3.25)
    assert torch.equal(x.fwd(), x.b.expand_as(x.x))
    dx, dw, db = x.bwd()
    assert (dw == 0).all() and torch.isfinite(dx).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_rows(dtype):
    In(4, 3, 1500, 128, dtype, True, "nthd").check()
    In(1, 1, 3001, 1024, dtype).check()


def test_in_place():
    for dtype in ("f32", "bf16"):
        for order in ("nhtd", "nthd"):
            x = In(2, 3, 50, 128, dtype, True, order)
            y, g = x.fwd(), x.bwd()
            kept, dy = x.x.clone(), x.dy.clone()
            lz.lizard_layer_norm_fwd(x.dims, x.x, x.w, x.b, x.x)
            assert torch.equal(x.x, y)
            x.x.copy_(kept)
            for target in (x.x, x.dy):
                x.x.copy_(kept)
                x.dy.copy_(dy)
                assert torch.equal(x.bwd(dx=target)[0], g[0])


def test_parts_of_the_gradient():
    x = In(2, 3, 50, 128, "bf16", True)
    d = x.dims
    dx, dw, db = x.bwd()
    ws = torch.zeros(lz.lizard_layer_norm_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    for want in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1)):
        out = [torch.full_like(t, 9.0) if w else None for w, t in zip(want, (dx, dw, db))]
        lz.lizard_layer_norm_bwd(d, x.x, x.w, x.dy, *out, ws)
        for p, q in zip(out, (dx, dw, db)):
            assert p is None or torch.equal(p, q)
    lz.lizard_layer_norm_bwd(d, x.x, x.w, x.dy, None, None, None, ws)
    e = lz.lizard_norm_dims(2, 3, 0, 128, 1, lz.LIZARD_BF16, 0.0)
    z = x.x[:, :, :0]
    lz.lizard_layer_norm_fwd(e, z, x.w, x.b, torch.empty_like(z))
    lz.lizard_layer_norm_bwd(e, z, x.w, z, torch.empty_like(z), dw, db, ws)
    assert (dw == 0).all() and (db == 0).all()


def test_rows_far_apart():
    far = torch.zeros(200 << 24, dtype=torch.bfloat16, device="cuda").view(200, -1)
    x = In(1, 1, 200, 128, "bf16")
    far[:, :128].copy_(x.x[0, 0])
    lz.lizard_layer_norm_fwd(x.dims, far[None, None, :, :128], x.w, x.b, far[None, None, :, 128:256])
    assert torch.equal(far[:, 128:256], x.fwd()[0, 0])


def test_a_layer_trains_and_serves():
    """Linear attention, the norm of its heads, and both backwards, captured into a graph; then the
    states go on to single tokens.  Each stage against 64 bits over what the stage before gave."""
    B, H, Hk, L, dk, dv = 2, 4, 2, 261, 64, 128
    gen = torch.Generator().manual_seed(11)
    r = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16).cuda()  # noqa: E731
    q, k, v, dn = r(B, L, H, dk).permute(0, 2, 1, 3), r(B, Hk, L, dk), r(B, Hk, L, dv), r(B, L, H, dv).permute(0, 2, 1, 3)
    g = -torch.rand(B, H, L, generator=gen).cuda()
    w, b = r(H, dv), r(H, dv)
    dims = lz.lizard_decay_dims(B, H, Hk, L, dk, dv, lz.LIZARD_BF16, 0.0)
    nd = lz.lizard_norm_dims(B, H, L, dv, 1, lz.LIZARD_BF16, 0.0)
    y, h = torch.empty_like(dn), torch.empty(B, H, dk, dv, device="cuda")
    n, dy, dw, db = torch.empty_like(dn), torch.empty_like(dn), torch.empty(H, dv, device="cuda"), torch.empty(H, dv, device="cuda")
    out = [torch.empty_like(t) for t in (q, k, v)]
    dg = torch.empty_like(g)
    zeros = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    wf, wb = (zeros(lz.lizard_decay_attn_workspace_bytes(dims, x)) for x in (False, True))
    wn = zeros(lz.lizard_layer_norm_workspace_bytes(nd))

    def step():
        lz.lizard_decay_attn_fwd(dims, q, k, v, g, None, None, y, h, wf)
        lz.lizard_layer_norm_fwd(nd, y, w, b, n)
        lz.lizard_layer_norm_bwd(nd, y, w, dn, dy, dw, db, wn)
        lz.lizard_decay_attn_bwd(dims, q, k, v, g, None, None, dy, None, *out, dg, None, wb)

    step()
    eager = [t.clone() for t in (y, h, n, dy, dw, db, *out, dg)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (y, h, n, dy, dw, db, *out, dg):
        t.fill_(7.0)
    graph.replay()
    for p, x in zip(eager, (y, h, n, dy, dw, db, *out, dg)):
        assert torch.equal(p, x)
    case = do.Case(q, k, v, g, dy=dy)
    t = do.terms(L, dk, dv, 2)
    do.close(y, case.y, do.bound(case.y, case.y_abs, y.dtype, t))
    x = In(B, H, L, dv, "bf16", True)
    x.x, x.dy, x.w, x.b = y, dn, w, b
    x.check()
    for got, want, s in zip(out, case.grads, case.sums):
        do.close(got, want, do.bound(want, s, got.dtype, t))
    assert do.rel_l2(dg, case.grads[3]) <= 1e-5
    # serving: the next token from the state, its heads normed
    sd, one = lz.lizard_decay_dims(B, H, Hk, 1, dk, dv, lz.LIZARD_BF16, 0.0), lz.lizard_norm_dims(B, H, 1, dv, 1, lz.LIZARD_BF16, 0.0)
    q1, k1, v1, g1, y1 = r(B, H, 1, dk), r(B, Hk, 1, dk), r(B, Hk, 1, dv), -torch.rand(B, H, 1, generator=gen).cuda(), torch.empty(B, H, 1, dv, dtype=torch.bfloat16, device="cuda")
    case = do.Case(q1, k1, v1, g1, h0=h)
    lz.lizard_decay_attn_step(sd, q1, k1, v1, g1, h, y1)
    do.close(y1, case.y, do.bound(case.y, case.y_abs, y1.dtype, t))
    do.close(h, case.h, do.bound(case.h, case.h_abs, torch.float32, 16))
    x.dims, x.x = one, y1.clone()
    lz.lizard_layer_norm_fwd(one, y1, w, b, y1)
    want, _, _ = do.norm(x.x, w[:, None], b[:, None], 1e-5)
    assert do.rel_l2(y1, want) <= 2.0 ** -8
