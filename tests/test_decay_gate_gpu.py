"""The gradient of the log decays element by element: what passes over a token is small beside what
other tokens exchange, in every way that a sequence can have it."""
import pytest

torch = pytest.importorskip("torch")

import decay_oracle as do
import hybrid_gated_linear_gb300 as lz
from test_decay_gpu import In

pytestmark = pytest.mark.gpu
INF = float("inf")


def limit(want, abs_sum, dims, L=None):
    """d log g_t is a sum of products (q_i k_j) D (dy_i v_j) over the tokens j < t <= i, all of which pass
    over t.  A product has one rounding for every addition of its two factors: scores (dk, dv) or states
    and their gradients (`terms` each); the sums behind them are at most 32 in a row, then trees of 32, 16
    and 8.  So twice `terms` and 64, half a step of the result, relative to the same sum over absolute values
    -- and nothing for tokens that lie on one side of t."""
    rel = (2 * do.terms(L or dims.L, dims.dk, dims.dv) + 64) * 2.0 ** -24
    return torch.finfo(torch.float32).eps / 2 * want.abs() + rel * abs_sum + 1e-30


def check(x):
    c = x.case(True)
    dg = x.bwd()[3]
    do.close(dg, c.grads[3], limit(c.grads[3], c.sums[3], x.dims))
    return dg


def scaled(x, where, by):
    """The rows of some tokens enlarged (a power of two: no rounding)."""
    for t in (x.q, x.k, x.v, x.dy):
        t[:, :, where] *= by


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(1, 1, 1, 1, 64, 64), (2, 2, 1, 2, 64, 128), (1, 2, 2, 33, 128, 64), (1, 2, 1, 64, 64, 64),
                                  (2, 4, 2, 97, 64, 128), (1, 2, 2, 129, 128, 128), (2, 3, 3, 300, 128, 64),
                                  (1, 2, 1, 640, 64, 128)], ids=str)
def test_elements(size, dtype):
    check(In(*size, dtype))
    check(In(*size, dtype, order="blhd", state=False, seed=5))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("order", ["bhld", "blhd"])
def test_large_tokens_far_before(dtype, order):
    """The first 256 tokens 128 times the others, at a decay that leaves 1e-100 of them at the end."""
    x = In(1, 3, 3, 640, 64, 128, dtype, order=order)
    x.g[:, 0], x.g[:, 1], x.g[:, 2] = -1.0, -0.25, -4.0
    scaled(x, slice(0, 256), 128.0)
    check(x)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_tokens_far_behind(dtype):
    x = In(1, 3, 1, 640, 128, 64, dtype)
    x.g[:, 0], x.g[:, 1], x.g[:, 2] = -1.0, -0.25, -4.0
    scaled(x, slice(384, 640), 128.0)
    check(x)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("at", [0, 5, 40, 70, 127, 128, 200])
def test_one_large_token(dtype, at):
    """One token 1024 times the others, its neighbours under strong and weak decays."""
    x = In(2, 2, 2, 260, 64, 64, dtype)
    x.g[0, 0] = -2.0
    scaled(x, slice(at, at + 1), 1024.0)
    check(x)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_and_small_documents_side_by_side(dtype):
    """Documents of very different size in one chunk, before and behind each other."""
    x = In(1, 2, 2, 384, 64, 64, dtype)
    for t in (32, 48, 64, 100, 128, 200, 320):
        x.g[:, :, t] = -INF
    for a, b in ((32, 48), (64, 100), (200, 320)):
        scaled(x, slice(a, b), 256.0)
    dg = check(x)
    assert (dg[x.g == -INF] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_states_at_the_ends(dtype):
    """An initial state and a final state's gradient far larger than the tokens'."""
    x = In(2, 2, 1, 400, 128, 128, dtype)
    x.h0 *= 4096.0
    x.df *= 4096.0
    x.g[0] = -0.5
    check(x)
    x.g[1, :, 150] = -INF
    x.count = [400, 230]
    check(x)


def exact_on_gpu(x):
    """d log g and the same sum over absolute values, in 64 bits on the device."""
    d = x.dims
    G, s, sums = d.H // d.Hk, d.dk ** -0.5, []
    for f in (lambda t: t, torch.abs):
        q, dy = f(x.q.double()) * s, f(x.dy.double())
        k, v = (f(t.double()).repeat_interleave(G, 1) for t in (x.k, x.v))
        g = torch.exp(x.g.double())[..., None, None]
        h, dh = f(x.h0.double()), f(x.df.double())
        hs = []
        for t in range(d.L):
            hs.append(h)
            h = g[:, :, t] * h + k[:, :, t, :, None] * v[:, :, t, None]
        out = torch.empty(d.B, d.H, d.L, dtype=torch.float64, device="cuda")
        for t in range(d.L - 1, -1, -1):
            dh = dh + q[:, :, t, :, None] * dy[:, :, t, None]
            out[:, :, t] = (g[:, :, t] * hs[t] * dh).sum((2, 3))
            dh = g[:, :, t] * dh
        sums.append(out.cpu())
    return sums


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(1, 3, 3, 3000, 64, 128), (2, 4, 1, 2500, 128, 64), (5, 30, 30, 530, 64, 64)], ids=str)
def test_many_chunks(size, dtype):
    """Segments of a long axis, and more heads than SMs; a head whose state lasts beside others whose
    sums are a thousandth of its own, and one loud stretch in the first chunks."""
    x = In(*size, dtype)
    x.g[:, 0] *= 0.01
    x.g[:, 1] = -1.0
    scaled(x, slice(100, 200), 64.0)
    dg, (want, abs_sum) = x.bwd()[3], exact_on_gpu(x)
    do.close(dg, want, limit(want, abs_sum, x.dims))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_that_overlap(dtype):
    """Rows that the tensor maps do not describe."""
    B, H, L, d = 1, 2, 200, 64
    flat = torch.randn(20000, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    x = In(B, H, H, L, d, d, dtype)
    x.k = flat.as_strided((B, H, L, d), (20000, 6400, 16, 1))
    c = x.case(True)
    out = [torch.empty(B, H, L, d, dtype=x.q.dtype, device="cuda") for _ in range(3)]
    dg = torch.empty(B, H, L, device="cuda")
    ws = torch.zeros(lz.lizard_decay_attn_workspace_bytes(x.dims, True), dtype=torch.uint8, device="cuda")
    lz.lizard_decay_attn_bwd(x.dims, x.q, x.k, x.v, x.g, None, x.h0, x.dy, x.df, *out, dg, None, ws)
    do.close(dg, c.grads[3], limit(c.grads[3], c.sums[3], x.dims))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("decay", [0.0, -1e-7, -0.05, -3.0, -60.0, -1e5, 0.02])
def test_constant_decays(dtype, decay):
    """One number per head, none, weak, strong, and a growing state; repeated by strides of 0."""
    x = In(1, 2, 2, 333, 64, 64, dtype)
    x.g = (torch.tensor([decay, decay / 2], device="cuda"))[None, :, None].expand(1, 2, 333)
    check(x)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("order", ["bhld", "blhd"])
def test_uneven_lengths_over_segments(dtype, order):
    """Few heads and a long axis, so that it is cut, with sequences that end in its first part, at a chunk's
    edge, or have no token, documents, and a workspace that holds anything behind its header."""
    x = In(5, 2, 1, 1200, 128, 64, dtype, order=order)
    x.count = [1200, 0, 256, 131, 1025]
    x.g[0, 1, 640] = x.g[4, 0, 1024] = x.g[2, :, 255] = -INF
    scaled(x, slice(120, 136), 64.0)
    for b, c in enumerate(x.count):
        for t in (x.q, x.k, x.v, x.dy):
            t[b, :, c:] = float("nan")
        x.g[b, :, c:] = float("nan")
    want = check(x)
    ws = torch.zeros(lz.lizard_decay_attn_workspace_bytes(x.dims, True), dtype=torch.uint8, device="cuda")
    ws[256:] = 255
    assert torch.equal(x.bwd(ws=ws)[3], want)
    for b, c in enumerate(x.count):
        assert (want[b, :, c:] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_without_the_other_gradients_of_the_ends(dtype):
    """The same bits whether the initial state's gradient is asked for or not; no states at the ends."""
    x = In(2, 4, 2, 500, 64, 128, dtype)
    assert torch.equal(x.bwd()[3], x.bwd(d_h0=False)[3])
    x.h0 = None
    check(x)
    x.df = None
    check(x)
