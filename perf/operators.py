"""The operators around an 8-bit key/value cache: their cases, plain forms and 64-bit values.

Rotary positions (forward and backward), the write and the read-back of a paged cache that
holds keys and values in 8 bits with one power-of-two scale per page and head, and the
attention that reads it (windows, meta tokens, grouped heads, one or many new tokens).
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
QMAX = {"e4m3": 448.0, "i8": 127.0}


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def listed():
    c = [
        # a serving step of 32 sequences rotates one new query and key per head, far into a
        # long context (frequencies scaled by parts): the call's latency counts
        dict(name="rope one token", kind="rope", dtype="bf16", N=32, H=32, Hk=8, T=1, d=128, rot=128,
             layout="half", scaling="parts", order="bhld"),
        # the training workload's queries and keys as the projections leave them (token-major)
        dict(name="rope training", kind="rope", dtype="bf16", N=8, H=32, Hk=32, T=2048, d=128, rot=128,
             layout="half", scaling="none", order="blhd"),
        # the gradients on their way back, fp32, interleaved pairs, half of each head rotated,
        # an odd length
        dict(name="rope backward", kind="rope_bwd", dtype="f32", N=2, H=24, Hk=6, T=1999, d=128, rot=64,
             layout="interleaved", scaling="linear", order="bhld"),
        # one new token of each of 64 sequences goes into the cache
        dict(name="store one token", kind="store", dtype="bf16", N=64, Hk=8, T=1, d=128, P=64, fmt="e4m3",
             len=5000, ragged=True, rope=False, order="bhld"),
        # four prompts of 4096 tokens, keys rotated on their way in
        dict(name="store prompts", kind="store", dtype="bf16", N=4, Hk=8, T=4096, d=128, P=64, fmt="e4m3",
             len=100, ragged=True, rope=True, order="blhd"),
        # uneven continuations in fp32, small pages, 8-bit integers
        dict(name="store ragged", kind="store", dtype="f32", N=7, Hk=5, T=333, d=64, P=16, fmt="i8",
             len=71, ragged=True, rope=False, order="bhld"),
        # one user, a short conversation, one token: latency
        dict(name="attend short", kind="attend", dtype="bf16", N=1, H=32, Hk=8, T=1, d=128, P=64, fmt="e4m3",
             len=500, ragged=False, W=0, M=0, rope=True, first=False, add=False, order="bhld"),
        # a serving batch of uneven lengths
        dict(name="attend batch", kind="attend", dtype="bf16", N=64, H=32, Hk=8, T=1, d=128, P=64, fmt="e4m3",
             len=8192, ragged=True, W=0, M=0, rope=True, first=False, add=False, order="bhld"),
        # the anchor window of 64 sequences x 32 heads over a ring of pages, meta tokens, added
        # to the gated branch's output
        dict(name="attend window", kind="attend", dtype="bf16", N=64, H=32, Hk=32, T=1, d=128, P=64, fmt="i8",
             len=20000, ragged=True, W=1024, M=4, rope=False, first=False, add=True, order="bhld"),
        # one very long context: the cache axis has to be split over the whole GPU
        dict(name="attend long", kind="attend", dtype="bf16", N=1, H=32, Hk=8, T=1, d=128, P=128, fmt="e4m3",
             len=131072, ragged=False, W=0, M=0, rope=True, first=False, add=False, order="bhld"),
        # drafted tokens to be verified: a few queries per sequence, uneven counts, left-padded
        # prompts of which one is all padding, fp32
        dict(name="attend drafted", kind="attend", dtype="f32", N=16, H=24, Hk=6, T=6, d=64, P=16, fmt="i8",
             len=3001, ragged=True, W=0, M=0, rope=True, first=True, add=False, order="blhd"),
        # a chunk of a long prompt against what came before it: matrix products bound it
        dict(name="attend prompt", kind="attend", dtype="bf16", N=2, H=32, Hk=8, T=2048, d=128, P=64, fmt="e4m3",
             len=14336, ragged=False, W=0, M=0, rope=True, first=False, add=False, order="blhd"),
    ]
    return c


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "rope_bwd", "store", "store", "attend", "attend", "attend"])
    c = dict(kind=kind, dtype=rng.choice(["bf16", "bf16", "f32"]), d=rng.choice([64, 128]),
             order=rng.choice(["bhld", "blhd"]))
    hk = rng.randint(1, 16)
    if kind in ("rope", "rope_bwd"):
        c.update(N=_log(rng, 1, 32), H=hk * rng.choice([1, 2, 4]), Hk=hk, rot=2 * rng.randint(4, c["d"] // 2),
                 layout=rng.choice(["half", "interleaved"]), scaling=rng.choice(["none", "linear", "parts"]))
        if rng.random() < 0.6:
            c["rot"] = c["d"]
        most = (1 << 25) // (c["N"] * (c["H"] + c["Hk"]))
        c["T"] = _log(rng, 1, max(2, min(16384, most // c["d"])))
        return c
    c.update(P=rng.choice([16, 32, 64, 128]), fmt=rng.choice(["e4m3", "i8"]), ragged=rng.random() < 0.7)
    if kind == "store":
        c.update(N=_log(rng, 1, 64), Hk=hk, len=_log(rng, 1, 20000), rope=c["dtype"] == "bf16" and rng.random() < 0.5)
        c["T"] = _log(rng, 1, max(2, min(8192, (1 << 24) // (c["N"] * hk * c["d"]))))
        return c
    c.update(H=hk * rng.choice([1, 2, 3, 4, 8]), Hk=hk, M=rng.choice([0, 0, 4, 7]), rope=rng.random() < 0.5,
             first=rng.random() < 0.3, add=rng.random() < 0.4)
    c["T"] = 1 if rng.random() < 0.5 else _log(rng, 2, 16) if rng.random() < 0.6 else _log(rng, 16, 1024)
    c["N"] = _log(rng, 1, 64 if c["T"] == 1 else 16 if c["T"] <= 16 else 3)
    c["len"] = _log(rng, 16, max(17, min(100000, (1 << 28) // (c["N"] * hk * c["d"]),
                                        (1 << 29) // (c["N"] * c["H"] * c["T"]))))
    c["W"] = _log(rng, 1, 4096) if rng.random() < 0.4 else 0
    return c


def _pos(c):
    """Tokens each sequence holds before the new ones: uneven lengths are spread evenly."""
    if not c["ragged"]:
        return [c["len"]] * c["N"]
    return [c["len"] * (n + 1) // c["N"] for n in range(c["N"])]


def _count(c):
    """New tokens of each sequence (uneven where there are several)."""
    return [c["T"] - (n * 5 % c["T"] if c["ragged"] else 0) for n in range(c["N"])]


def _first(c):
    """The first visible token of each sequence; the last of several sequences sees none."""
    if not c["first"]:
        return [0] * c["N"]
    p = _pos(c)
    return [p[n] + c["T"] if 0 < n == c["N"] - 1 else p[n] // 8 * (1 - n % 2) for n in range(c["N"])]


def _slots(c):
    """Pages a sequence's table holds: the whole context, or a ring that covers the window."""
    P = c["P"]
    if c["kind"] == "store":
        return (c["T"] + P - 2) // P + 3
    if c["W"]:
        return min((c["W"] + c["T"] - 2) // P + 2, (c["len"] + c["T"] + P - 1) // P)
    return (c["len"] + c["T"] + P - 1) // P


def work(c):
    es = 2 if c["dtype"] == "bf16" else 4
    if c["kind"] in ("rope", "rope_bwd"):
        n = c["N"] * (c["H"] + c["Hk"]) * c["T"]
        return {"bytes": n * c["d"] * 2 * es + 8 * c["N"] * c["T"], "flops": 3 * n * c["rot"]}
    hd = c["Hk"] * c["d"]
    if c["kind"] == "store":
        new = sum(_count(c))
        back = sum(k + min(p, c["P"]) for k, p in zip(_count(c), _pos(c)))
        return {"bytes": 2 * hd * (new * (es + 1) + back + c["N"] * (c["T"] + c["P"]) * es), "flops": 4 * hd * new}
    b = c["N"] * c["H"] * c["T"] * c["d"] * es * (3 if c["add"] else 2) + 2 * c["H"] * c["M"] * c["d"] * es
    f = 0
    for p, k, s in zip(_pos(c), _count(c), _first(c)):
        lo = max(s, p - c["W"] + 1 if c["W"] else 0, 0)
        seen = max(0, p + k - lo)
        b += 2 * seen * hd + 8 * c["Hk"] * ((seen + c["P"] - 1) // c["P"])
        pairs = sum(max(0, p + t + 1 - max(s, p + t - c["W"] + 1 if c["W"] else 0, 0)) for t in range(k))
        f += 4 * c["H"] * c["d"] * (pairs + k * c["M"])
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
BASE = 500000.0
SCALING = {"none": (1.0, 1.0, 1.0, 1, 1.0), "linear": (4.0, 1.0, 1.0, 1, 1.0),
           # factor, low, high, original length, factor on cos and sin
           "parts": (8.0, 1.0, 4.0, 8192, 1.2079)}


def _theta(rot, scaling, dev):
    """Angle per token of each pair, in 64 bits."""
    factor, low, high, orig, _ = SCALING[scaling]
    th = BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    if scaling == "linear":
        return th / factor
    if scaling == "parts":
        turns = orig * th / (2 * math.pi)
        keep = ((turns - low) / (high - low)).clamp(0, 1)
        return th * (keep + (1 - keep) / factor)
    return th


def _rows(g, dev, N, H, T, d, dtype, order, amp=1.0):
    """Rows of N sequences, H heads, T tokens: head-major, or a view of token-major memory."""
    shape = (N, H, T, d) if order == "bhld" else (N, T, H, d)
    x = (torch.randn(shape, generator=g, device=dev) * amp).to(DT[dtype])
    return x if order == "bhld" else x.permute(0, 2, 1, 3)


def _pool(g, dev, c, end, gain):
    """Codes and scales of a pool of pages in which every token before `end` is written; what
    no token was written to holds arbitrary bytes (and scales that are not numbers)."""
    N, S, P, Hk, d = c["N"], _slots(c), c["P"], c["Hk"], c["d"]
    x = torch.randn(N * S, Hk, P, d, generator=g, device=dev)
    x *= gain * torch.exp(0.4 * torch.randn(N * S, Hk, 1, 1, generator=g, device=dev))
    scale = torch.exp2(torch.ceil(torch.log2(x.abs().amax((2, 3)) / QMAX[c["fmt"]])))
    x /= scale[:, :, None, None]
    if c["fmt"] == "e4m3":
        codes = x.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        codes = x.round_().clamp_(-127, 127).to(torch.int8).view(torch.uint8)
    del x
    slot = torch.arange(S, device=dev)
    last = (end - 1).clamp(min=0)[:, None] // P
    page = last - (last - slot) % S  # the newest logical page that a slot can hold
    tok = page[:, :, None] * P + torch.arange(P, device=dev)
    live = ((tok >= 0) & (tok < end[:, None, None])).reshape(N * S, P)
    codes = codes.view(N * S, Hk, P, d)
    holes = (~live).nonzero()
    junk = torch.randint(0, 256, (holes.shape[0], Hk, d), generator=g, device=dev, dtype=torch.uint8)
    codes[holes[:, 0], :, holes[:, 1]] = junk
    scale[~live.any(1)] = float("nan")
    return codes, scale


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed * 7919 + 11)
    s = dict(case=c)
    N, T, d, dt = c["N"], c["T"], c["d"], c["dtype"]
    if c["kind"] in ("rope", "rope_bwd"):
        s["q"] = _rows(g, dev, N, c["H"], T, d, dt, c["order"])
        s["k"] = _rows(g, dev, N, c["Hk"], T, d, dt, c["order"])
        start = torch.randint(0, 120000 if T == 1 else 4096, (N, 1), generator=g, device=dev)
        s["positions"] = start + torch.arange(T, device=dev)
        s["theta"] = _theta(c["rot"], c["scaling"], dev)
        return s
    S, P, Hk = _slots(c), c["P"], c["Hk"]
    s["pos"] = torch.tensor(_pos(c), device=dev)
    s["count"] = torch.tensor(_count(c), device=dev, dtype=torch.int32)
    end = s["pos"] + (s["count"] if c["kind"] == "attend" else 0)
    pages = N * S + 3
    s["table"] = torch.randperm(pages, generator=g, device=dev)[:N * S].to(torch.int32).view(N, S)
    gain = torch.exp(0.5 * torch.randn(1, Hk, 1, d, generator=g, device=dev))
    for name in ("k", "v"):
        codes, scale = _pool(g, dev, c, end, gain if name == "k" else 1.0)
        s[name + "_codes"] = torch.zeros(pages, Hk, P, d, dtype=torch.uint8, device=dev)
        s[name + "_scale"] = torch.ones(pages, Hk, dtype=torch.float32, device=dev)
        at = s["table"].reshape(-1).long()
        s[name + "_codes"][at] = codes
        s[name + "_scale"][at] = scale
    s["theta"] = _theta(d, "parts", dev)
    if c["kind"] == "store":
        s["k"] = _rows(g, dev, N, Hk, T, d, dt, c["order"])
        # keys carry a few strong channels
        s["k"].mul_(gain.to(s["k"].dtype))
        s["v"] = _rows(g, dev, N, Hk, T, d, dt, c["order"])
        return s
    s["q"] = _rows(g, dev, N, c["H"], T, d, dt, c["order"], amp=1.5)
    s["first"] = torch.tensor(_first(c), device=dev) if c["first"] else None
    s["meta_k"] = _rows(g, dev, 1, c["H"], c["M"], d, dt, "bhld")[0] if c["M"] else None
    s["meta_v"] = _rows(g, dev, 1, c["H"], c["M"], d, dt, "bhld")[0] if c["M"] else None
    s["y_add"] = _rows(g, dev, N, c["H"], T, d, dt, c["order"]) if c["add"] else None
    s["alpha"] = 0.75 if c["add"] else 1.0
    return s


# ---------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------
def _rotate(x, positions, theta, layout, factor, sign):
    """x [N,H,T,d] in fp32 with the first 2 * len(theta) channels rotated."""
    ang = positions.double()[:, None, :, None] * theta
    co, si = (torch.cos(ang) * factor).float(), (torch.sin(ang) * (sign * factor)).float()
    rot = 2 * theta.numel()
    x = x.float()
    y = x.clone()
    if layout == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2] = a * co - b * si
        y[..., rot // 2:rot] = b * co + a * si
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = a * co - b * si
        y[..., 1:rot:2] = b * co + a * si
    return y


def _chunk_order(P, d, dev):
    """Where the 16-byte chunks of a page's rows are stored: chunk c of row r at place
    c ^ (r % 8) of rows of 128 bytes, c ^ (r / 2 % 4) of rows of 64."""
    r = torch.arange(P, device=dev)[:, None]
    x = r % 8 if d == 128 else r // 2 % 4
    return r, torch.arange(d // 16, device=dev) ^ x


def _values(codes, fmt):
    return codes.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8).float()


def _pages(s, name, ids):
    """Codes (rows in order) and scales of the pages ids [N,J]: [N,J,Hk,P,d], [N,J,Hk]."""
    c = s["case"]
    r, x = _chunk_order(c["P"], c["d"], ids.device)
    codes = s[name + "_codes"][ids.long()]
    codes = codes.unflatten(-1, (c["d"] // 16, 16))[:, :, :, r, x].flatten(-2)
    return codes, s[name + "_scale"][ids.long()]


def _table(s, page):
    """Page ids of logical pages [N,J]."""
    return torch.gather(s["table"], 1, page % s["table"].shape[1])


def _store(s, name, x):
    """x [N,Hk,T,d] fp32 into the pages of tokens pos .. pos + count - 1."""
    c = s["case"]
    P, T, dev = c["P"], c["T"], x.device
    J = (T + P - 2) // P + 1
    pos, cnt = s["pos"][:, None, None], s["count"][:, None, None]
    page = s["pos"][:, None] // P + torch.arange(J, device=dev)
    rel = page[:, :, None] * P + torch.arange(P, device=dev) - pos
    new = (rel >= 0) & (rel < cnt)
    touched = new.any(2)
    old = (rel < 0) & touched[:, :, None]
    ids = _table(s, page)
    codes, scale = _pages(s, name, ids)
    n = torch.arange(c["N"], device=dev)[:, None, None]
    rows = x[n, :, rel.clamp(0, T - 1)].permute(0, 1, 3, 2, 4)  # [N,J,Hk,P,d]
    rows = torch.where(new[:, :, None, :, None], rows, 0.0)
    need = torch.exp2(torch.ceil(torch.log2(rows.abs().amax((3, 4)) / QMAX[c["fmt"]]))).clamp(min=2.0 ** -126)
    fresh = torch.where(old.any(2)[:, :, None], torch.maximum(need, scale), need)
    kept = torch.where(old[:, :, None, :, None], _values(codes, c["fmt"]) * scale[..., None, None], 0.0)
    v = torch.where(new[:, :, None, :, None], rows, kept) / fresh[..., None, None]
    q = v.to(torch.float8_e4m3fn).view(torch.uint8) if c["fmt"] == "e4m3" else v.round().to(torch.int8).view(torch.uint8)
    q = torch.where((new | old)[:, :, None, :, None], q, codes)
    r, order = _chunk_order(P, c["d"], dev)
    out = torch.empty_like(q).unflatten(-1, (c["d"] // 16, 16))
    out[:, :, :, r, order] = q.unflatten(-1, (c["d"] // 16, 16))
    at = ids.long()[touched]
    s[name + "_codes"][at] = out.flatten(-2)[touched]
    s[name + "_scale"][at] = fresh[touched]


def _read(s, name, start, count, T):
    """Tokens start .. start + count - 1 as values, zeros up to T: [N,Hk,T,d]."""
    c = s["case"]
    P, dev = c["P"], start.device
    J = (T + P - 2) // P + 1
    page = start[:, None] // P + torch.arange(J, device=dev)
    codes, scale = _pages(s, name, _table(s, page))
    v = (_values(codes, c["fmt"]) * scale[..., None, None]).permute(0, 2, 1, 3, 4).flatten(2, 3)
    t = torch.arange(T, device=dev)
    v = torch.gather(v, 2, ((start % P)[:, None] + t)[:, None, :, None].expand(-1, v.shape[1], -1, v.shape[3]))
    return torch.where((t < count[:, None])[:, None, :, None], v, 0.0).to(DT[c["dtype"]])


def _attend(s):
    c = s["case"]
    N, H, Hk, T, d, P, W, dev = c["N"], c["H"], c["Hk"], c["T"], c["d"], c["P"], c["W"], s["q"].device
    G = H // Hk
    pos, cnt = s["pos"], s["count"]
    first = s["first"] if s["first"] is not None else torch.zeros_like(pos)
    J = s["table"].shape[1]
    last = (pos + cnt - 1).clamp(min=0) // P
    page = (last - J + 1).clamp(min=0)[:, None] + torch.arange(J, device=dev)
    tok = (page[:, :, None] * P + torch.arange(P, device=dev)).flatten(1)  # [N,J*P]
    at = pos[:, None] + torch.arange(T, device=dev)  # positions of the queries
    seen = (tok[:, None] <= at[:, :, None]) & (tok[:, None] >= first[:, None, None])
    if W:
        seen &= tok[:, None] > at[:, :, None] - W
    seen &= (torch.arange(T, device=dev) < cnt[:, None])[:, :, None]  # [N,T,J*P]
    live = seen.any(1)[:, None, :, None]
    ids = _table(s, page)
    kv = []
    for name in ("k", "v"):
        codes, scale = _pages(s, name, ids)
        x = (_values(codes, c["fmt"]) * scale[..., None, None]).permute(0, 2, 1, 3, 4).flatten(2, 3)
        kv.append(torch.where(live, x, 0.0))
        del codes, x
    q = s["q"].float()
    qr = _rotate(q, at, s["theta"], "half", SCALING["parts"][4], 1.0) if c["rope"] else q
    z = torch.matmul(qr.reshape(N, Hk, G * T, d), kv[0].transpose(2, 3)) / math.sqrt(d)
    z = z.view(N, H, T, J * P).masked_fill_(~seen[:, None], -math.inf)
    if c["M"]:
        zm = torch.matmul(q, s["meta_k"].float().transpose(1, 2)) / math.sqrt(d)
        z = torch.cat([zm, z], -1)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(m == -math.inf, 0.0, m))
    del z
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p[..., c["M"]:].reshape(N, Hk, G * T, J * P), kv[1]).view(N, H, T, d)
    if c["M"]:
        o = o + torch.matmul(p[..., :c["M"]], s["meta_v"].float())
    o = o / torch.where(total > 0, total, 1.0) * s["alpha"]
    if s["y_add"] is not None:
        o = o + s["y_add"].float()
    return torch.where((torch.arange(T, device=dev) < cnt[:, None])[:, None, :, None], o, 0.0).to(DT[c["dtype"]])


def _plain(s):
    c = s["case"]
    if c["kind"] in ("rope", "rope_bwd"):
        sign = 1.0 if c["kind"] == "rope" else -1.0
        f = SCALING[c["scaling"]][4]
        return [_rotate(s[n], s["positions"], s["theta"], c["layout"], f, sign).to(s[n].dtype) for n in ("q", "k")]
    if c["kind"] == "attend":
        return _attend(s)
    at = s["pos"][:, None] + torch.arange(c["T"], device=s["pos"].device)
    k = s["k"].float()
    if c["rope"]:
        k = _rotate(k, at, s["theta"], "half", SCALING["parts"][4], 1.0)
    _store(s, "k", k)
    _store(s, "v", s["v"].float())
    start = (s["pos"] - c["P"]).clamp(min=0)
    n = s["pos"] + s["count"] - start
    return [_read(s, "k", start, n, c["T"] + c["P"]), _read(s, "v", start, n, c["T"] + c["P"])]


# ---------------------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------------------
def _rope_handle(lz, s, rot, layout, scaling):
    factor, low, high, orig, attn = SCALING[scaling]
    kind = {"none": lz.LIZARD_ROPE_PLAIN, "linear": lz.LIZARD_ROPE_LINEAR, "parts": lz.LIZARD_ROPE_PARTS}[scaling]
    turns = lz.lizard_rope_table(lz.lizard_rope_spec(rot, kind, BASE, factor, low, high, orig)).to(s["theta"].device)
    return lz.lizard_rope(turns, rot, lz.LIZARD_ROPE_HALF if layout == "half" else lz.LIZARD_ROPE_INTERLEAVED, attn)


def _handles(lz, s):
    """What a serving program keeps between calls: tables, handles, workspaces, outputs."""
    c, dev = s["case"], s["theta"].device
    dt = lz.LIZARD_BF16 if c["dtype"] == "bf16" else lz.LIZARD_F32
    h = s["handles"] = {}
    if c["kind"] in ("rope", "rope_bwd"):
        h["rope"] = _rope_handle(lz, s, c["rot"], c["layout"], c["scaling"])
        h["dims"] = lz.lizard_rope_dims(c["N"], c["H"], c["Hk"], c["T"], c["d"], dt)
        h["out"] = [torch.empty_like(s["q"]), torch.empty_like(s["k"])]
        return h
    h["rope"] = _rope_handle(lz, s, c["d"], "half", "parts") if c["rope"] else None
    h["cache"] = lz.lizard_cache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], s["table"],
                                 lz.LIZARD_KV_E4M3 if c["fmt"] == "e4m3" else lz.LIZARD_KV_I8)
    if c["kind"] == "store":
        h["io"] = lz.lizard_cache_io(c["T"], dt)
        h["io_back"] = lz.lizard_cache_io(c["T"] + c["P"], dt)
        h["out"] = [torch.empty(c["N"], c["Hk"], c["T"] + c["P"], c["d"], dtype=DT[c["dtype"]], device=dev)
                    for _ in range(2)]
        h["ws"] = torch.zeros(lz.lizard_cache_workspace_bytes(), dtype=torch.uint8, device=dev)
        h["start"] = (s["pos"] - c["P"]).clamp(min=0)
        h["n"] = (s["pos"] + s["count"] - h["start"]).to(torch.int32)
        return h
    h["dims"] = lz.lizard_cache_attn_dims(c["H"], c["T"], c["M"], c["W"], dt, 0.0, s["alpha"])
    h["out"] = torch.empty_like(s["q"])
    h["ws"] = torch.zeros(lz.lizard_cache_attn_workspace_bytes(h["cache"], h["dims"]), dtype=torch.uint8, device=dev)
    return h


def _own(s):
    import hybrid_gated_linear_gb300 as lz
    c = s["case"]
    h = s.get("handles") or _handles(lz, s)
    out = h["out"]
    if c["kind"] == "rope":
        lz.lizard_rope_fwd(h["dims"], h["rope"], s["q"], s["k"], s["positions"], out[0], out[1])
    elif c["kind"] == "rope_bwd":
        lz.lizard_rope_bwd(h["dims"], h["rope"], s["q"], s["k"], s["positions"], out[0], out[1])
    elif c["kind"] == "store":
        lz.lizard_cache_write(h["cache"], h["io"], s["k"], s["v"], h["rope"], s["pos"], s["count"], h["ws"])
        lz.lizard_cache_read(h["cache"], h["io_back"], h["start"], h["n"], out[0], out[1], h["ws"])
    else:
        lz.lizard_cache_attn(h["cache"], h["dims"], s["q"], h["rope"], s["pos"], s["count"], s["first"],
                             s["meta_k"], s["meta_v"], s["y_add"], out, h["ws"])
    return out


def run(s):
    return _own(s) if own else _plain(s)


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------
def _turned(x, position, theta, layout, factor):
    """One token's heads [H,d] (or many tokens': position [T], x [H,T,d]) rotated, in 64 bits:
    the pair (a, b) as the complex number a + ib times factor e^{i position theta}."""
    h = theta.numel()
    x = x.double()
    pairs = torch.stack([x[..., :h], x[..., h:2 * h]], -1) if layout == "half" else x[..., :2 * h].unflatten(-1, (h, 2))
    z = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.full_like(theta, factor).expand(len(position), h), position.double()[:, None] * theta)
    z = torch.view_as_real(z)
    z = torch.cat([z[..., 0], z[..., 1]], -1) if layout == "half" else z.flatten(-2)
    return torch.cat([z, x[..., 2 * h:]], -1)


def _bytes_to_values(b, fmt):
    b = b.long()
    if fmt == "i8":
        return torch.where(b > 127, b - 256, b).double()
    e, m = b >> 3 & 15, b & 7
    v = torch.where(e > 0, (8 + m).double() * torch.exp2((e - 10).double()), m.double() * 2.0 ** -9)
    return torch.where(b > 127, -v, v)


def _token_values(s, name, n, t):
    """Values [Hk,len(t),d] of tokens t of sequence n, byte by byte by the storage rule."""
    c = s["case"]
    P, d = c["P"], c["d"]
    page = s["table"][n, t // P % s["table"].shape[1]].long()
    row, col = (t % P)[:, None], torch.arange(d, device=t.device)
    byte = row * d + ((col // 16) ^ (row % 8 if d == 128 else row // 2 % 4)) * 16 + col % 16
    raw = s[name + "_codes"].view(-1, c["Hk"], P * d)[page[:, None], :, byte]  # [T,d,Hk]
    v = _bytes_to_values(raw, c["fmt"]) * s[name + "_scale"].double()[page][:, None]
    return v.permute(2, 0, 1)


def _rounded(v, fmt):
    """v (within the range) to the nearest value that the format holds, ties to even."""
    if fmt == "i8":
        return torch.round(v)
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _exact_store(s):
    c = s["case"]
    P, T, dev = c["P"], c["T"], s["pos"].device
    out = [torch.zeros(c["N"], c["Hk"], T + P, c["d"], dtype=torch.float64, device=dev) for _ in range(2)]
    for n in range(c["N"]):
        pos, cnt = _pos(c)[n], _count(c)[n]
        start = max(0, pos - P)
        for o, name in zip(out, ("k", "v")):
            x = s[name][n, :, :cnt].double()
            if name == "k" and c["rope"]:
                x = _turned(x, pos + torch.arange(cnt, device=dev), s["theta"], "half", SCALING["parts"][4])
            if pos > start:
                o[n, :, :pos - start] = _token_values(s, name, n, torch.arange(start, pos, device=dev))
            o[n, :, pos - start:pos - start + cnt] = x
            for page in range(pos // P, (pos + cnt - 1) // P + 1):
                a, b = max(page * P, start) - start, min(page * P + P, pos + cnt) - start
                new = o[n, :, max(a, pos - start):b].abs().amax((1, 2))
                scale = torch.exp2(torch.ceil(torch.log2(new / QMAX[c["fmt"]])))
                if pos > page * P:
                    had = s[name + "_scale"][s["table"][n, page % s["table"].shape[1]].long()].double()
                    scale = torch.maximum(scale, had)
                o[n, :, a:b] = _rounded(o[n, :, a:b] / scale[:, None, None], c["fmt"]) * scale[:, None, None]
    return out


def _exact_attend(s):
    c = s["case"]
    dev, T, d, Hk = s["q"].device, c["T"], c["d"], c["Hk"]
    out = torch.zeros(c["N"], c["H"], T, d, dtype=torch.float64, device=dev)
    for n, (pos, cnt, first) in enumerate(zip(_pos(c), _count(c), _first(c))):
        lo = max(first, pos - c["W"] + 1 if c["W"] else 0, 0)
        at = pos + torch.arange(cnt, device=dev)
        tok = torch.arange(lo, max(lo, pos + cnt), device=dev)
        q = s["q"][n, :, :cnt].double()
        qr = _turned(q, at, s["theta"], "half", SCALING["parts"][4]) if c["rope"] else q
        k, v = _token_values(s, "k", n, tok), _token_values(s, "v", n, tok)
        no = (tok > at[:, None]) | ((tok <= at[:, None] - c["W"]) if c["W"] else False)
        for h in range(c["H"]):
            kk, vv, hide = k[h // (c["H"] // Hk)], v[h // (c["H"] // Hk)], no
            z = qr[h] @ kk.T
            if c["M"]:
                z = torch.cat([q[h] @ s["meta_k"][h].double().T, z], 1)
                vv = torch.cat([s["meta_v"][h].double(), vv], 0)
                hide = torch.cat([torch.zeros(cnt, c["M"], dtype=torch.bool, device=dev), no], 1)
            p = torch.softmax((z / math.sqrt(d)).masked_fill(hide, -math.inf), 1) if z.shape[1] else z
            out[n, h, :cnt] = s["alpha"] * torch.nan_to_num(p, nan=0.0) @ vv
            if s["y_add"] is not None:
                out[n, h, :cnt] += s["y_add"][n, h, :cnt].double()
    return out


def exact(c, seed):
    s = prepare(c, seed)
    if c["kind"] in ("rope", "rope_bwd"):
        sign = 1 if c["kind"] == "rope" else -1
        f = SCALING[c["scaling"]][4]
        return [torch.stack([_turned(s[x][n], sign * s["positions"][n], s["theta"], c["layout"], f) for n in range(c["N"])])
                for x in ("q", "k")]
    return _exact_attend(s) if c["kind"] == "attend" else _exact_store(s)
