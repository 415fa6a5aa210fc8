"""What the GPU tests of the cache attention share: a filled cache, one call, and the definition
in 64 bits over the values that the cache itself gives back (so that the quantisation is not part
of the difference)."""
import cache_oracle as co
import hybrid_gated_linear_gb300 as lz

FMT = {"e4m3": lz.LIZARD_KV_E4M3, "i8": lz.LIZARD_KV_I8}


class Filled:
    """A cache that holds tokens lo[n] .. end[n] - 1 of every sequence; k, v [N,Hk,T,d] fp32 are
    the rows from lo[n] on, `held` what the cache gives back for them."""

    def __init__(self, k, v, lo, end, P, fmt, slots=None, seed=0):
        import torch
        N, Hk, T, d = k.shape
        self.lo, self.end = list(lo), list(end)
        S = slots or max((e + P - 1) // P for e in end)
        pages = N * S + 2
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.table = torch.randperm(pages, generator=g, device="cuda")[:N * S].to(torch.int32).view(N, S)
        codes = [torch.randint(0, 256, (pages, Hk, P, d), generator=g, device="cuda", dtype=torch.uint8) for _ in "kv"]
        scales = [torch.full((pages, Hk), float("nan"), device="cuda") for _ in "kv"]
        self.h = lz.lizard_cache(*codes, *scales, self.table, FMT[fmt])
        ws = torch.zeros(lz.lizard_cache_workspace_bytes(), dtype=torch.uint8, device="cuda")
        pos = torch.tensor(self.lo, device="cuda")
        count = torch.tensor([e - a for a, e in zip(lo, end)], dtype=torch.int32, device="cuda")
        io = lz.lizard_cache_io(T, lz.LIZARD_F32)
        lz.lizard_cache_write(self.h, io, k, v, None, pos, count, ws)
        self.held = [torch.empty_like(k), torch.empty_like(v)]
        lz.lizard_cache_read(self.h, io, pos, count, *self.held, ws)
        assert lz.lizard_check_device_errors(ws) == 0


def workspace(cache, dims):
    import torch
    return torch.zeros(lz.lizard_cache_attn_workspace_bytes(cache.h, dims), dtype=torch.uint8, device="cuda")


def on_device(x, bits=64):
    import torch
    return None if x is None else torch.tensor(x, dtype=torch.int64 if bits == 64 else torch.int32, device="cuda")


def definition(f, q, pos, count=None, W=0, first=None, meta=None, y_add=None, alpha=1.0, th=None):
    """y in 64 bits, the sums of cache_oracle.attend_bound (A = sum p |v|, Z = max scale |q| |k|),
    and S = sum over the visible tokens of |v| / sum of the weights in units of the largest."""
    import torch
    N, H, T, d = q.shape
    y, A, S = (torch.zeros(N, H, T, d, dtype=torch.float64, device="cuda") for _ in range(3))
    Z = torch.zeros(N, H, T, 1, dtype=torch.float64, device="cuda")
    G, scale = H // f.held[0].shape[1], d ** -0.5
    qd = q.double()
    at = torch.tensor(pos, device="cuda")[:, None] + torch.arange(T, device="cuda")
    qr = qd if th is None else torch.from_numpy(co.rotate(qd.cpu().numpy(), at.cpu().numpy()[:, None], th)).cuda()
    for n in range(N):
        c = T if count is None else count[n]
        if c and f.end[n] > f.lo[n]:
            tok = torch.arange(f.lo[n], f.end[n], device="cuda")
            K, V = (x[n, :, :len(tok)].double().repeat_interleave(G, 0) for x in f.held)
        else:
            tok, K, V = torch.zeros(0, device="cuda"), *(torch.zeros(H, 0, d, device="cuda").double(),) * 2
        p = at[n, :c, None]
        hide = (tok > p) | (tok < (0 if first is None else first[n])) | ((tok <= p - W) if W else False)
        z = (qr[n, :, :c] @ K.transpose(1, 2) * scale).masked_fill(hide, -float("inf"))
        zz = (qr[n, :, :c].abs() @ K.abs().transpose(1, 2) * scale).masked_fill(hide, 0.0)
        va = V.abs()
        if meta is not None:
            mk, mv = (m.double() for m in meta)
            z = torch.cat([qd[n, :, :c] @ mk.transpose(1, 2) * scale, z], 2)
            zz = torch.cat([qd[n, :, :c].abs() @ mk.abs().transpose(1, 2) * scale, zz], 2)
            V, va = torch.cat([mv, V], 1), torch.cat([mv.abs(), va], 1)
        if not z.shape[2]:
            continue
        m = z.amax(2, keepdim=True)
        w = torch.exp(z - torch.where(m == -float("inf"), 0.0, m))
        l = w.sum(2, keepdim=True).clamp(min=1e-300)
        y[n, :, :c], A[n, :, :c], Z[n, :, :c] = alpha * (w / l) @ V, abs(alpha) * (w / l) @ va, zz.amax(2, keepdim=True)
        S[n, :, :c] = abs(alpha) * (w > 0).double() @ va / l
    if y_add is not None:
        y += y_add.double()
        for n in range(N if count is not None else 0):
            y[n, :, count[n]:] = 0
    return y, A, Z, S


def attend(f, q, pos, count=None, W=0, first=None, meta=None, y_add=None, alpha=1.0, rope=None, ws=None, status=0):
    import torch
    N, H, T, d = q.shape
    dims = lz.lizard_cache_attn_dims(H, T, 0 if meta is None else meta[0].shape[1], W,
                                     lz.LIZARD_F32 if q.dtype == torch.float32 else lz.LIZARD_BF16, 0.0, alpha)
    ws = workspace(f, dims) if ws is None else ws
    y = torch.full_like(q, 9.0)
    mk, mv = meta or (None, None)
    lz.lizard_cache_attn(f.h, dims, q, rope, on_device(pos), on_device(count, 32), on_device(first), mk, mv, y_add, y, ws)
    assert lz.lizard_check_device_errors(ws) == status
    return y


def bound_of(q, pos, want, A, Z, S, y_add=None, floor=0.0):
    """cache_oracle.attend_bound plus `floor` (the smallest step of a weight, in units of the row's
    largest) times S."""
    import torch
    dtype = "f32" if q.dtype == torch.float32 else "bf16"
    bound = co.attend_bound(*(x.cpu().numpy() for x in (want, A, Z)), dtype, q.shape[3], max(pos) + q.shape[2] + 16)
    bound = bound + floor * S.cpu().numpy()
    return bound if y_add is None else bound + 2.0 ** -23 * y_add.double().abs().cpu().numpy()


def assert_within(y, want, bound):
    import torch
    err = (y.double() - want).abs().cpu().numpy()
    assert torch.isfinite(y).all()
    assert (err <= bound).all(), (float(err.max()), float((err / bound).max()))


def check_attention(f, q, pos, floor=0.0, rope=None, **kw):
    """One call against the definition; rope is a handle and its angles per token."""
    handle, th = rope or (None, None)
    y = attend(f, q, pos, rope=handle, **kw)
    want = definition(f, q, pos, th=th, **kw)
    assert_within(y, want[0], bound_of(q, pos, *want, kw.get("y_add"), floor))
    return y


def gaussian(shape, seed, amp=1.0):
    import torch
    return amp * torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")
