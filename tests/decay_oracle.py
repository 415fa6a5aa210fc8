"""The linear attention with a decay per head and layer norm in 64 bits, token by token, and bounds
on what rounding may change.  Plain torch on the CPU; shares nothing with the kernels."""
import torch


def live_rows(x, count):
    """x [B,H,L,d] in 64 bits, zeros behind each sequence's last token."""
    x = x.detach().cpu().double().clone()
    for b, c in enumerate(count):
        x[b, :, c:] = 0
    return x


def factors(log_decay, count):
    """g [B,H,L]; 1 behind each sequence's last token."""
    g = torch.exp(log_decay.detach().cpu().double())
    for b, c in enumerate(count):
        g[b, :, c:] = 1
    return g


def heads(x, H):
    return x.repeat_interleave(H // x.shape[1], 1)


def forward(q, k, v, g, h0, scale):
    """y [B,H,L,dv] and the states after every token [L+1,B,H,dk,dv] (the first: h0)."""
    B, H, L, dk = q.shape
    h = torch.zeros(B, H, dk, v.shape[3], dtype=torch.float64) if h0 is None else h0.double()
    hs, y = [h], torch.zeros(B, H, L, v.shape[3], dtype=torch.float64)
    for t in range(L):
        h = g[:, :, t, None, None] * h + k[:, :, t, :, None] * v[:, :, t, None, :]
        y[:, :, t] = scale * torch.einsum("bhk,bhkv->bhv", q[:, :, t], h)
        hs.append(h)
    return y, hs


def backward(q, k, v, g, hs, dy, d_final, scale):
    """dq, dk, dv (per query head), d log g, d h0."""
    L = q.shape[2]
    dh = torch.zeros_like(hs[0]) if d_final is None else d_final.double()
    dq, dk, dv, dg = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(g)
    for t in range(L - 1, -1, -1):
        dh = dh + scale * q[:, :, t, :, None] * dy[:, :, t, None, :]
        dq[:, :, t] = scale * torch.einsum("bhkv,bhv->bhk", hs[t + 1], dy[:, :, t])
        dk[:, :, t] = torch.einsum("bhkv,bhv->bhk", dh, v[:, :, t])
        dv[:, :, t] = torch.einsum("bhkv,bhk->bhv", dh, k[:, :, t])
        dg[:, :, t] = g[:, :, t] * (hs[t] * dh).sum((2, 3))
        dh = g[:, :, t, None, None] * dh
    return dq, dk, dv, dg, dh


class Case:
    """One call's inputs (on any device) with the exact results and, from the same formulas over
    absolute values, the sums that bound the rounding."""

    def __init__(self, q, k, v, log_decay, count=None, h0=None, dy=None, d_final=None, scale=0.0):
        B, self.H, L, dk = q.shape
        self.Hk = k.shape[1]
        n = [L] * B if count is None else list(count)
        self.scale = scale if scale > 0 else dk ** -0.5
        g = factors(log_decay, n)
        rows = [live_rows(q, n), heads(live_rows(k, n), self.H), heads(live_rows(v, n), self.H)]
        h0 = None if h0 is None else h0.detach().cpu().double()
        self.y, hs = forward(*rows, g, h0, self.scale)
        a = [x.abs() for x in rows]
        self.y_abs, hs_abs = forward(*a, g, None if h0 is None else h0.abs(), self.scale)
        self.h, self.h_abs = hs[-1], hs_abs[-1]
        if dy is not None:
            dy = live_rows(dy, n)
            df = None if d_final is None else d_final.detach().cpu().double()
            grads = backward(*rows, g, hs, dy, df, self.scale)
            sums = backward(*a, g, hs_abs, dy.abs(), None if df is None else df.abs(), self.scale)
            self.grads, self.sums = self._shared(grads, n), self._shared(sums, n)

    def _shared(self, grads, n):
        dq, dk, dv, dg, dh = grads
        G = self.H // self.Hk
        dk, dv = (x.unflatten(1, (self.Hk, G)).sum(2) for x in (dk, dv))
        for b, c in enumerate(n):  # log_decay is not read there
            dg[b, :, c:] = 0
        return dq, dk, dv, dg, dh


def bound(want, abs_sum, dtype, terms):
    """Half a step of the result's type, `terms` fp32 roundings of every summand, and for bf16 calls one
    rounding of each summand to bf16 (a score, or the state that a chunk starts from)."""
    half = torch.finfo(dtype).eps / 2
    rel = terms * 2.0 ** -24 + (2.0 ** -8 if dtype == torch.bfloat16 else 0.0)
    return half * want.abs() * (1 + rel) + rel * (1 + half) * abs_sum + 1e-30


def terms(L, dk, dv, G=1):
    """fp32 roundings that a summand can meet: in a score (the wider of the head's widths), in the sum
    over a chunk's tokens and over the state's rows (128 each), per chunk of 64 two for its decay and
    one for the update, eight for the exponentials and scales (each of two units in the last place),
    one for each head of a group."""
    return max(dk, dv) + 128 + max(dk, dv) + 4 * (L // 64 + 1) + 16 + G


def close(got, want, limit):
    got = got.detach().cpu().double()
    assert torch.isfinite(got).all()
    err = (got - want).abs()
    assert (err <= limit).all(), (float(err.max()), float((err / limit).max()))


def rel_l2(got, want):
    n = float(torch.linalg.vector_norm(want))
    return float(torch.linalg.vector_norm(got.detach().cpu().double() - want)) / (n if n else 1.0)


def norm(x, w, b, eps):
    """y, n and 1/sigma of rows x [..., d] (w, b broadcast against x), in 64 bits."""
    x = x.detach().cpu().double()
    m = x - x.mean(-1, keepdim=True)
    r = (m.square().mean(-1, keepdim=True) + eps).rsqrt()
    n = m * r
    y = n if w is None else n * w.detach().cpu().double()
    return y if b is None else y + b.detach().cpu().double(), n, r


def norm_backward(x, w, dy, eps, over):
    _, n, r = norm(x, None, None, eps)
    dy = dy.detach().cpu().double()
    a = dy if w is None else dy * w.detach().cpu().double()
    dx = r * (a - a.mean(-1, keepdim=True) - n * (a * n).mean(-1, keepdim=True))
    return dx, (dy * n).sum(over), dy.sum(over), (a, n, r)
