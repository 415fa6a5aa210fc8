"""Linear attention with one decay per head, and the layer norm behind it: their cases, plain
forms and 64-bit values.

The state of a head decays by one number per token, h_t = g_t h_{t-1} + k_t v_t^T, and
y_t = scale q_t^T h_t (forward over a prompt, backward, and the recurrent form that serves single
tokens); a layer norm over each head's channels, or over whole rows, follows it in such layers.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
INF = float("inf")
EPS = 1e-5


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def listed():
    return [
        # two prompts of 4096 tokens at the training workload's heads, as the projections leave
        # them (token-major); the final state goes on to the single-token form
        dict(name="prompt", kind="fwd", dtype="bf16", B=2, H=32, Hk=32, L=4096, dk=128, dv=128, order="blhd",
             decay="token", docs=0, ragged=False, h0=False, final=True),
        # one very long context with grouped key and value heads: few heads, a long axis
        dict(name="long prompt", kind="fwd", dtype="bf16", B=1, H=32, Hk=8, L=65536, dk=128, dv=128, order="bhld",
             decay="fixed", docs=0, ragged=False, h0=False, final=True),
        # fp32, uneven lengths, several documents packed in a row, a prompt that continues a state
        dict(name="ragged documents", kind="fwd", dtype="f32", B=5, H=12, Hk=4, L=1999, dk=64, dv=128, order="bhld",
             decay="token", docs=300, ragged=True, h0=True, final=True),
        # a few tokens of several sequences (a short turn of a conversation): latency
        dict(name="short turn", kind="fwd", dtype="bf16", B=8, H=16, Hk=16, L=37, dk=64, dv=64, order="blhd",
             decay="token", docs=0, ragged=True, h0=True, final=True),
        # the training step's backward
        dict(name="training backward", kind="bwd", dtype="bf16", B=2, H=32, Hk=32, L=4096, dk=128, dv=128,
             order="blhd", decay="token", docs=0, ragged=False, h0=False, final=False),
        # fp32 gradients of packed documents of uneven length, shared key heads, gradients that
        # come in and go out through the states
        dict(name="ragged backward", kind="bwd", dtype="f32", B=3, H=6, Hk=3, L=777, dk=64, dv=64, order="bhld",
             decay="token", docs=200, ragged=True, h0=True, final=True),
        # one user, one token: latency
        dict(name="one token", kind="step", dtype="bf16", B=1, H=32, Hk=32, L=1, dk=128, dv=128, order="bhld",
             decay="token", docs=0, ragged=False, h0=True, final=True),
        # a serving batch, one token each: the states have to be read and written
        dict(name="token batch", kind="step", dtype="bf16", B=64, H=32, Hk=8, L=1, dk=128, dv=128, order="bhld",
             decay="token", docs=0, ragged=False, h0=True, final=True),
        # the norm of each head's output with weights of its own, in the attention's layout
        dict(name="norm of heads", kind="norm", dtype="bf16", N=2, H=32, T=4096, d=128, order="blhd", heads=True),
        # the norm of a batch's last tokens over the model's width: latency
        dict(name="norm of a few rows", kind="norm", dtype="f32", N=1, H=1, T=63, d=4096, order="bhld", heads=False),
        # gradients of the heads' norm and of its weights
        dict(name="norm of heads backward", kind="norm_bwd", dtype="bf16", N=2, H=32, T=4096, d=128, order="blhd",
             heads=True),
        # gradients of a norm over wide rows: one weight, summed over every token
        dict(name="norm of rows backward", kind="norm_bwd", dtype="bf16", N=1, H=1, T=8191, d=4096, order="bhld",
             heads=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["fwd", "fwd", "fwd", "bwd", "bwd", "step", "norm", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    order = rng.choice(["bhld", "blhd"])
    if kind in ("norm", "norm_bwd"):
        if rng.random() < 0.5:
            c = dict(N=_log(rng, 1, 16), H=rng.randint(1, 40), d=rng.choice([64, 128]), heads=rng.random() < 0.7)
        else:
            c = dict(N=1, H=1, d=8 * _log(rng, 1, 1792), heads=False)
        c["T"] = _log(rng, 1, max(2, (1 << 25) // (c["N"] * c["H"] * c["d"])))
        return dict(kind=kind, dtype=dtype, order=order, **c)
    hk = rng.randint(1, 16)
    c = dict(kind=kind, dtype=dtype, H=hk * rng.choice([1, 1, 2, 4]), Hk=hk, dk=rng.choice([64, 128]),
             dv=rng.choice([64, 128]), order=order, decay=rng.choice(["token", "token", "fixed"]))
    c["docs"] = 0 if c["decay"] == "fixed" or rng.random() < 0.6 else _log(rng, 8, 1000)
    if kind == "step":
        c.update(B=_log(rng, 1, max(1, min(96, 2048 // c["H"]))), L=1 if rng.random() < 0.7 else rng.randint(2, 8),
                 docs=0, ragged=False, h0=True, final=True)
        return c
    c.update(B=_log(rng, 1, 8), ragged=rng.random() < 0.5, h0=rng.random() < 0.5, final=rng.random() < 0.5)
    c["L"] = _log(rng, 1, max(2, min(16384, (1 << (18 if dtype == "bf16" else 16)) // (c["B"] * c["H"]))))
    return c


def _count(c):
    """Tokens of each sequence: all, or uneven ones, the second of several sequences empty."""
    if not c["ragged"]:
        return [c["L"]] * c["B"]
    return [0 if n == 1 and c["B"] > 2 else c["L"] - (n * 7 + 3) * c["L"] // 23 % max(1, c["L"]) for n in range(c["B"])]


def work(c):
    es = 2 if c["dtype"] == "bf16" else 4
    if c["kind"] in ("norm", "norm_bwd"):
        n, w = c["N"] * c["H"] * c["T"] * c["d"], (c["H"] if c["heads"] else 1) * c["d"]
        if c["kind"] == "norm":
            return {"bytes": 2 * n * es + 2 * w * es, "flops": 8 * n}
        return {"bytes": 3 * n * es + w * (es + 8), "flops": 16 * n}
    H, Hk, dk, dv = c["H"], c["Hk"], c["dk"], c["dv"]
    n, all_n, states = sum(_count(c)), c["B"] * c["L"], 4 * c["B"] * H * dk * dv
    fixed = 4 * H if c["decay"] == "fixed" else 4 * H * n
    # the recurrence's own products: the update k v^T with its decay and the query's product
    flops = n * H * 4 * dk * dv
    if c["kind"] in ("fwd", "step"):
        b = es * (n * (H * dk + Hk * (dk + dv)) + all_n * H * dv) + fixed + states * (c["h0"] + c["final"])
        return {"bytes": b, "flops": flops}
    b = es * (n * (H * (dk + dv) + Hk * (dk + dv)) + all_n * (H * dk + Hk * (dk + dv))) + fixed + 4 * H * all_n
    # h0 is read and its gradient written, the final state's gradient is read
    return {"bytes": b + states * (2 * c["h0"] + c["final"]), "flops": 3 * flops}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _rows(g, dev, N, H, T, d, dtype, order, amp=1.0):
    """Rows of N sequences, H heads, T tokens: head-major, or a view of token-major memory."""
    shape = (N, H, T, d) if order == "bhld" else (N, T, H, d)
    x = (torch.randn(shape, generator=g, device=dev) * amp).to(DT[dtype])
    return x if order == "bhld" else x.permute(0, 2, 1, 3)


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed * 7919 + 17)
    s = dict(case=c)
    if c["kind"] in ("norm", "norm_bwd"):
        x = _rows(g, dev, c["N"], c["H"], c["T"], c["d"], c["dtype"], c["order"])
        # rows of different size and mean, as a residual stream or an attention's heads have them
        size = torch.exp(torch.randn(c["N"], c["H"], c["T"], 1, generator=g, device=dev))
        s["x"] = x.mul_(size.to(x.dtype)).add_((0.5 * size).to(x.dtype))
        w = (c["H"], c["d"]) if c["heads"] else (c["d"],)
        s["weight"] = (1 + 0.2 * torch.randn(w, generator=g, device=dev)).to(DT[c["dtype"]])
        s["bias"] = (0.2 * torch.randn(w, generator=g, device=dev)).to(DT[c["dtype"]])
        if c["kind"] == "norm_bwd":
            s["dy"] = _rows(g, dev, c["N"], c["H"], c["T"], c["d"], c["dtype"], c["order"])
        return s
    B, H, Hk, L, dk, dv = c["B"], c["H"], c["Hk"], c["L"], c["dk"], c["dv"]
    s["q"] = _rows(g, dev, B, H, L, dk, c["dtype"], c["order"])
    s["k"] = _rows(g, dev, B, Hk, L, dk, c["dtype"], c["order"])
    s["v"] = _rows(g, dev, B, Hk, L, dv, c["dtype"], c["order"])
    head = torch.arange(H, device=dev) / H
    if c["decay"] == "fixed":
        # one constant per head, from 1 - 2^-3 to 1 - 2^-11, moved a little by the seed
        rate = torch.exp2(-3 - 8 * head - 0.5 * torch.rand(H, generator=g, device=dev))
        s["log_decay"] = torch.log1p(-rate)[None, :, None].expand(B, H, L)
    else:
        # what a projection of each token gives, around a rate of the head's own (0.5 to 0.001)
        z = math.log(0.5) + head[None, :, None] * math.log(0.002) + torch.randn(B, H, L, generator=g, device=dev)
        s["log_decay"] = -torch.nn.functional.softplus(z)
        if c["docs"]:  # a document begins: nothing of what was before is seen
            new = torch.rand(B, 1, L, generator=g, device=dev) < 1.0 / c["docs"]
            s["log_decay"] = s["log_decay"].masked_fill(new, -INF)
    s["count"] = torch.tensor(_count(c), device=dev, dtype=torch.int32) if c["ragged"] else None
    s["h0"] = 2 * torch.randn(B, H, dk, dv, generator=g, device=dev) if c["h0"] else None
    if c["kind"] == "bwd":
        s["dy"] = _rows(g, dev, B, H, L, dv, c["dtype"], c["order"])
        s["d_final"] = torch.randn(B, H, dk, dv, generator=g, device=dev) if c["final"] else None
    return s


# ---------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------
class _Chunks:
    """The decays of a call between the tokens of chunks of C, from sums in 64 bits: `inside`
    [B,H,n,C,C] from token j to token i >= j, `head` [B,H,n,C] from before a chunk to each of its
    tokens, `tail` from each token to its chunk's end, `across` [B,H,n+1,n+1]: from the end of
    chunk c' - 1 (0: the initial state) to the start of chunk c >= c' (n: the end)."""

    def __init__(self, s):
        c = s["case"]
        self.L, self.C = c["L"], min(128, c["L"])
        self.n = -(-c["L"] // self.C)
        live = torch.ones(c["B"], c["L"], dtype=torch.bool, device=s["q"].device)
        if s["count"] is not None:
            live = torch.arange(c["L"], device=s["q"].device) < s["count"][:, None]
        self.live = live[:, None]
        lg = torch.where(self.live, s["log_decay"], 0.0).double()
        self.reset = lg == -INF
        lg = torch.nn.functional.pad(torch.where(self.reset, 0.0, lg), (0, self.n * self.C - self.L))
        new = torch.nn.functional.pad(self.reset, (0, self.n * self.C - self.L))
        b, doc = lg.cumsum(2).unflatten(2, (self.n, self.C)), new.long().cumsum(2).unflatten(2, (self.n, self.C))
        end_b, end_doc = (torch.nn.functional.pad(x[..., -1], (1, 0)) for x in (b, doc))  # [B,H,n+1]
        tri = torch.ones(self.C, self.C, dtype=torch.bool, device=b.device).tril()

        def decay(later, earlier, doc_l, doc_e, also=True):
            return torch.where((doc_l == doc_e) & also, torch.exp(later - earlier), 0.0).float()

        self.inside = decay(b[..., :, None], b[..., None, :], doc[..., :, None], doc[..., None, :], tri)
        self.head = decay(b, end_b[..., :-1, None], doc, end_doc[..., :-1, None])
        self.tail = decay(end_b[..., 1:, None], b, end_doc[..., 1:, None], doc)
        order = torch.ones(self.n + 1, self.n + 1, dtype=torch.bool, device=b.device).tril()
        self.across = decay(end_b[..., :, None], end_b[..., None, :], end_doc[..., :, None], end_doc[..., None, :], order)

    def cut(self, x, heads):
        """Rows [B,*,L,d] as [B,heads,n,C,d] in fp32, zeros behind each sequence's last token."""
        x = torch.where(self.live[..., None], x.float(), 0.0)
        x = torch.nn.functional.pad(x, (0, 0, 0, self.n * self.C - self.L)).unflatten(2, (self.n, self.C))
        return x if x.shape[1] == heads else x.repeat_interleave(heads // x.shape[1], 1)

    def join(self, x):
        """[B,H,n,C,...] back to [B,H,L,...], zeros behind each sequence's last token."""
        x = x.flatten(2, 3)[:, :, :self.L]
        return torch.where(self.live[..., None] if x.dim() == 4 else self.live, x, 0.0)


def _starts(ch, k, v, h0):
    """The states at the chunks' starts and at the end, [B,H,n+1,dk,dv]."""
    own_part = torch.matmul((k * ch.tail[..., None]).transpose(-1, -2), v)
    first = torch.zeros_like(own_part[:, :, :1]) if h0 is None else h0[:, :, None]
    parts = torch.cat([first, own_part], 2)
    return torch.matmul(ch.across, parts.flatten(3)).view(parts.shape)


def _forward(s):
    c, scale = s["case"], s["case"]["dk"] ** -0.5
    ch = _Chunks(s)
    q, k, v = (ch.cut(s[x], c["H"]) for x in ("q", "k", "v"))
    h = _starts(ch, k, v, s["h0"])
    p = torch.matmul(q, k.transpose(-1, -2)) * ch.inside
    y = torch.matmul(p, v) + torch.matmul(q, h[:, :, :-1]) * ch.head[..., None]
    return (ch.join(y) * scale).to(s["q"].dtype), h[:, :, -1].contiguous()


def _backward(s):
    c, scale = s["case"], s["case"]["dk"] ** -0.5
    ch = _Chunks(s)
    q, k, v, dy = (ch.cut(s[x], c["H"]) for x in ("q", "k", "v", "dy"))
    h = _starts(ch, k, v, s["h0"])[:, :, :-1]
    # the gradients of the states at the chunks' ends (and of the initial one), from later chunks
    part = torch.matmul((q * (ch.head * scale)[..., None]).transpose(-1, -2), dy)
    last = torch.zeros_like(part[:, :, :1]) if s.get("d_final") is None else s["d_final"][:, :, None]
    parts = torch.cat([part, last], 2)
    dh = torch.matmul(ch.across.transpose(-1, -2), parts.flatten(3)).view(parts.shape)
    d_h0, dh = dh[:, :, 0].contiguous(), dh[:, :, 1:]
    p = torch.matmul(q, k.transpose(-1, -2)) * (ch.inside * scale)
    dp = torch.matmul(dy, v.transpose(-1, -2))
    w = (p * dp).tril(-1)
    ds = dp * (ch.inside * scale)
    qh, kd = torch.matmul(q, h) * (ch.head * scale)[..., None], torch.matmul(k, dh) * ch.tail[..., None]
    dq = torch.matmul(ds, k) + torch.matmul(dy, h.transpose(-1, -2)) * (ch.head * scale)[..., None]
    dk = torch.matmul(ds.transpose(-1, -2), q) + torch.matmul(v, dh.transpose(-1, -2)) * ch.tail[..., None]
    dv = torch.matmul(p.transpose(-1, -2), dy) + kd
    # a decay's gradient: everything that passes over its token, within the chunk, out of the
    # state before, into the state after, and from state to state
    rows, cols = (qh * dy).sum(-1).double(), (kd * v).sum(-1).double()
    inner = w.sum(-1).double() - w.sum(-2).double()
    through = (h * dh).flatten(3).sum(-1).double() * ch.across[:, :, 1:, :-1].diagonal(dim1=-2, dim2=-1)
    dg = (inner + rows).flip(-1).cumsum(-1).flip(-1) + cols.cumsum(-1) - cols + through[..., None]
    dg = ch.join(dg).masked_fill(ch.reset, 0.0).float()
    G = c["H"] // c["Hk"]
    dk, dv = (ch.join(x).unflatten(1, (c["Hk"], G)).sum(2) for x in (dk, dv))
    t = s["q"].dtype
    return ch.join(dq).to(t), dk.to(t), dv.to(t), dg, d_h0


def _norm(s):
    x = s["x"].float()
    m = x - x.mean(-1, keepdim=True)
    return m * torch.rsqrt((m * m).mean(-1, keepdim=True) + EPS)


def _weights(s, name):
    w = s[name].float()
    return w[:, None] if s["case"]["heads"] else w


def _norm_backward(s):
    x, dy = s["x"].float(), s["dy"].float()
    m = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((m * m).mean(-1, keepdim=True) + EPS)
    n = m * r
    dn = dy * _weights(s, "weight")
    dx = r * (dn - dn.mean(-1, keepdim=True) - n * (dn * n).mean(-1, keepdim=True))
    over = (0, 2) if s["case"]["heads"] else (0, 1, 2)
    return dx.to(s["x"].dtype), (dy * n).sum(over, dtype=torch.float64).float(), dy.sum(over, dtype=torch.float64).float()


def _plain(s):
    c = s["case"]
    if c["kind"] == "norm":
        return (_norm(s) * _weights(s, "weight") + _weights(s, "bias")).to(s["x"].dtype)
    if c["kind"] == "norm_bwd":
        return _norm_backward(s)
    if c["kind"] == "bwd":
        out = _backward(s)
        return out if c["h0"] else out[:4]
    if c["kind"] == "step" and c["L"] == 1:
        G = c["H"] // c["Hk"]
        q = s["q"][:, :, 0].float()
        k, v = (s[x][:, :, 0].float().repeat_interleave(G, 1) for x in ("k", "v"))
        h = s["h0"]
        h.mul_(torch.exp(s["log_decay"])[..., None]).add_(k[..., None] * v[:, :, None])
        y = torch.matmul(q[:, :, None], h) * c["dk"] ** -0.5
        return y.to(s["q"].dtype), h
    y, h = _forward(s)
    if c["kind"] == "step":
        h = s["h0"].copy_(h)
    return (y, h) if c["final"] else y


# ---------------------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------------------
def _handles(lz, s):
    """What a program keeps between calls: dimensions, workspaces, outputs."""
    c = s["case"]
    dt = lz.LIZARD_BF16 if c["dtype"] == "bf16" else lz.LIZARD_F32
    h = s["handles"] = {}
    dev = (s["x"] if "x" in s else s["q"]).device
    if c["kind"] in ("norm", "norm_bwd"):
        h["dims"] = lz.lizard_norm_dims(c["N"], c["H"], c["T"], c["d"], c["heads"], dt, EPS)
        h["out"] = torch.empty_like(s["x"])
        if c["kind"] == "norm_bwd":
            h["out"] = [h["out"]] + [torch.empty(s["weight"].shape, dtype=torch.float32, device=dev) for _ in range(2)]
            h["ws"] = torch.zeros(lz.lizard_layer_norm_workspace_bytes(h["dims"]), dtype=torch.uint8, device=dev)
        return h
    h["dims"] = lz.lizard_decay_dims(c["B"], c["H"], c["Hk"], c["L"], c["dk"], c["dv"], dt, 0.0)
    final = torch.empty(c["B"], c["H"], c["dk"], c["dv"], device=dev)
    if c["kind"] == "bwd":
        h["out"] = [torch.empty_like(s[x]) for x in ("q", "k", "v")]
        h["out"] += [torch.empty(c["B"], c["H"], c["L"], device=dev), final if c["h0"] else None]
    else:
        h["y"] = torch.empty(s["q"].shape[:3] + (c["dv"],), dtype=s["q"].dtype, device=dev)
        h["final"] = final if c["final"] else None
    if c["kind"] != "step":
        size = lz.lizard_decay_attn_workspace_bytes(h["dims"], c["kind"] == "bwd")
        h["ws"] = torch.zeros(size, dtype=torch.uint8, device=dev)
    return h


def _own(s):
    import hybrid_gated_linear_gb300 as lz
    c = s["case"]
    h = s.get("handles") or _handles(lz, s)
    if c["kind"] == "norm":
        lz.lizard_layer_norm_fwd(h["dims"], s["x"], s["weight"], s["bias"], h["out"])
        return h["out"]
    if c["kind"] == "norm_bwd":
        lz.lizard_layer_norm_bwd(h["dims"], s["x"], s["weight"], s["dy"], *h["out"], h["ws"])
        return h["out"]
    if c["kind"] == "step":
        lz.lizard_decay_attn_step(h["dims"], s["q"], s["k"], s["v"], s["log_decay"], s["h0"], h["y"])
        return h["y"], s["h0"]
    if c["kind"] == "fwd":
        lz.lizard_decay_attn_fwd(h["dims"], s["q"], s["k"], s["v"], s["log_decay"], s["count"], s["h0"], h["y"],
                                 h["final"], h["ws"])
        return (h["y"], h["final"]) if c["final"] else h["y"]
    lz.lizard_decay_attn_bwd(h["dims"], s["q"], s["k"], s["v"], s["log_decay"], s["count"], s["h0"], s["dy"],
                             s["d_final"], *h["out"], h["ws"])
    return h["out"] if c["h0"] else h["out"][:4]


def run(s):
    return _own(s) if own else _plain(s)


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------
def _exact_norm(s):
    c = s["case"]
    x = s["x"].double()
    var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
    xhat = (x - mean) / torch.sqrt(var + EPS)
    shape = (1, c["H"], 1, c["d"]) if c["heads"] else (1, 1, 1, c["d"])
    w = s["weight"].double().view(shape)
    if c["kind"] == "norm":
        return xhat * w + s["bias"].double().view(shape)
    # the Jacobian of xhat = (x - mean) / sigma, applied from the left
    dy = s["dy"].double()
    a = dy * w
    d = c["d"]
    dx = (a - a.sum(-1, keepdim=True) / d - xhat * ((a * xhat).sum(-1, keepdim=True) / d)) / torch.sqrt(var + EPS)
    dw = torch.einsum("nhtd,nhtd->hd", dy, xhat)
    db = torch.einsum("nhtd->hd", dy)
    return [dx, dw if c["heads"] else dw.sum(0), db if c["heads"] else db.sum(0)]


def _tokens(s):
    """Per token: decay factors [L,B*H,1,1] and rows [L,B*H,d], in 64 bits; past a sequence's end
    the factor is 1 and every row 0, so that the state stays."""
    c = s["case"]
    H, L = c["H"], c["L"]
    live = torch.ones(c["B"], L, dtype=torch.float64, device=s["q"].device)
    for b, n in enumerate(_count(c)):
        live[b, n:] = 0
    a = torch.exp(s["log_decay"].double())
    a = torch.where(live[:, None] > 0, a, 1.0).permute(2, 0, 1).reshape(L, -1, 1, 1)
    rows = []
    for name in ("q", "k", "v", "dy"):
        if name in s:
            x = s[name].double()
            x = x if x.shape[1] == H else x.repeat_interleave(H // x.shape[1], 1)
            x = torch.where(live[:, None, :, None] > 0, x, 0.0)
            rows.append(x.permute(2, 0, 1, 3).reshape(L, c["B"] * H, -1).contiguous())
    return a, rows


def _state(s, name):
    c = s["case"]
    h = torch.zeros(c["B"], c["H"], c["dk"], c["dv"], dtype=torch.float64, device=s["q"].device)
    return (h if s.get(name) is None else h + s[name]).view(-1, c["dk"], c["dv"])


def _back(x, c):
    """[L,B*H,d] to [B,H,L,d]."""
    return x.view(c["L"], c["B"], c["H"], -1).permute(1, 2, 0, 3)


def _exact_forward(s):
    c = s["case"]
    a, (q, k, v) = _tokens(s)
    h = _state(s, "h0")
    y = torch.empty(c["L"], h.shape[0], 1, c["dv"], dtype=torch.float64, device=h.device)
    for t in range(c["L"]):
        h = torch.baddbmm(h * a[t], k[t].unsqueeze(2), v[t].unsqueeze(1))
        torch.bmm(q[t].unsqueeze(1), h, out=y[t])
    return _back(y, c) * c["dk"] ** -0.5, h.view(c["B"], c["H"], c["dk"], c["dv"])


def _exact_backward(s):
    c, scale, M = s["case"], s["case"]["dk"] ** -0.5, 64
    L = c["L"]
    a, (q, k, v, dy) = _tokens(s)
    q = q * scale
    h = _state(s, "h0")
    kept = []
    for t in range(L):
        if t % M == 0:
            kept.append(h)
        h = torch.baddbmm(h * a[t], k[t].unsqueeze(2), v[t].unsqueeze(1))
    dh = _state(s, "d_final")
    dq, dk, dv, da = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(a[..., 0])
    for block in range(len(kept) - 1, -1, -1):
        hs = [kept[block]]
        top = min(L, block * M + M)
        for t in range(block * M, top):
            hs.append(torch.baddbmm(hs[-1] * a[t], k[t].unsqueeze(2), v[t].unsqueeze(1)))
        for t in range(top - 1, block * M - 1, -1):
            dh = torch.baddbmm(dh, q[t].unsqueeze(2), dy[t].unsqueeze(1))
            dq[t] = torch.bmm(hs[t - block * M + 1], dy[t].unsqueeze(2))[..., 0] * scale
            dk[t] = torch.bmm(dh, v[t].unsqueeze(2))[..., 0]
            dv[t] = torch.bmm(k[t].unsqueeze(1), dh)[:, 0]
            before = hs[t - block * M] * a[t]
            da[t] = (before * dh).sum((1, 2))[:, None]
            dh = dh * a[t]
    G = c["H"] // c["Hk"]
    dq, dk, dv = _back(dq, c), *(_back(x, c).unflatten(1, (c["Hk"], G)).sum(2) for x in (dk, dv))
    # the decay past a sequence's end is not read: its gradient is 0
    live = torch.tensor(_count(c), device=q.device)[:, None, None] > torch.arange(L, device=q.device)
    dg = torch.where(live, _back(da, c)[..., 0], 0.0)
    out = [dq, dk, dv, dg, dh.view(c["B"], c["H"], c["dk"], c["dv"])]
    return out if c["h0"] else out[:4]


def exact(c, seed):
    s = prepare(c, seed)
    if c["kind"] in ("norm", "norm_bwd"):
        return _exact_norm(s)
    if c["kind"] == "bwd":
        return _exact_backward(s)
    y, h = _exact_forward(s)
    return (y, h) if c["final"] else y
