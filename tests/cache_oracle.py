"""64-bit numpy oracle of the rotary positions, the 8-bit paged cache and the attention over
it (the formulas of include/lizard.h), for the parity tests."""
from __future__ import annotations

import math

import numpy as np

QMAX = {"e4m3": 448.0, "i8": 127.0}
# 2 pi in extended precision: far positions multiply an angle's relative error
TWO_PI = 2 * np.longdouble(math.pi) + np.longdouble(2.4492935982947064e-16)


def theta(rot, base=500000.0, scaling="plain", factor=1.0, low=1.0, high=4.0, original=8192):
    """Angles per token, in extended precision."""
    th = np.longdouble(base) ** (-np.arange(0, rot, 2).astype(np.longdouble) / rot)
    if scaling == "linear":
        th = th / np.longdouble(factor)
    if scaling == "parts":
        keep = np.clip((original * th / TWO_PI - low) / (np.longdouble(high) - low), 0, 1)
        th = th * (keep + (1 - keep) / np.longdouble(factor))
    return th


def rotate(x, pos, th, layout="half", factor=1.0, sign=1.0):
    """x [..., T, d] at positions pos [T] (or broadcastable [..., T])."""
    x = np.asarray(x, np.float64)
    rot = 2 * len(th)
    ang = np.fmod(np.asarray(pos)[..., None].astype(np.longdouble) * th, TWO_PI).astype(np.float64)
    c, s = factor * np.cos(ang), factor * sign * np.sin(ang)
    y = x.copy()
    if layout == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    return y


def e4m3_decode(b):
    b = np.asarray(b).astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e > 0, (8 + m) * 2.0 ** (e - 10.0), m * 2.0 ** -9)
    return np.where(b & 128, -v, v)


def decode(b, fmt):
    return e4m3_decode(b) if fmt == "e4m3" else np.asarray(b).astype(np.uint8).view(np.int8).astype(np.float64)


def encode(v, fmt):
    """Values in units of the scale to bytes: nearest, ties to even, saturating."""
    v = np.asarray(v, np.float64)
    if fmt == "i8":
        return np.clip(np.rint(v), -127, 127).astype(np.int8).view(np.uint8)
    a = np.minimum(np.abs(v), 448.0)
    e = np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -9))), -6)
    step = 2.0 ** (e - 3)
    q = np.minimum(np.rint(a / step) * step, 448.0)
    e = np.maximum(np.floor(np.log2(np.maximum(q, 2.0 ** -9))), -6)
    normal = q >= 2.0 ** -6
    byte = np.where(normal, (e + 7) * 8 + q / 2.0 ** (e - 3) - 8, q * 2.0 ** 9).astype(np.int64)
    return (byte | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def scale_of(amax, fmt):
    if not amax > 0:
        return 2.0 ** -126
    return max(2.0 ** math.ceil(math.log2(amax / QMAX[fmt])), 2.0 ** -126)


class Cache:
    """Pools in the stored byte order.  Bytes and scales nothing was written to are junk
    (every byte value, NaN scales)."""

    def __init__(self, N, Hk, P, d, max_pages, fmt, rng, extra=2):
        self.N, self.Hk, self.P, self.d, self.S, self.fmt = N, Hk, P, d, max_pages, fmt
        self.pages = N * max_pages + extra
        shape = (self.pages, Hk, P, d)
        self.codes = {x: rng.integers(0, 256, shape).astype(np.uint8) for x in "kv"}
        self.scale = {x: np.full((self.pages, Hk), np.nan, np.float32) for x in "kv"}
        self.table = rng.permutation(self.pages)[:N * max_pages].astype(np.int32).reshape(N, max_pages)

    def place(self, r):
        """Byte positions of the d channels of row r of a page."""
        c = np.arange(self.d)
        x = r % 8 if self.d == 128 else r // 2 % 4
        return (c // 16 ^ x) * 16 + c % 16

    def write(self, x, n, pos, rows):
        """rows [Hk, count, d] of sequence n at positions pos ..; x is "k" or "v"."""
        cnt = rows.shape[1]
        for page in range(pos // self.P, (pos + cnt - 1) // self.P + 1 if cnt else 0):
            pid = self.table[n, page % self.S]
            t0 = page * self.P
            r0, r1 = max(0, pos - t0), min(self.P, pos + cnt - t0)
            for h in range(self.Hk):
                new = np.asarray(rows[h, t0 + r0 - pos:t0 + r1 - pos], np.float64)
                fin = np.where(np.isfinite(new), np.abs(new), 0.0)
                s = scale_of(fin.max(), self.fmt)
                if r0:
                    had = float(self.scale[x][pid, h])
                    s = max(s, had)
                    for r in range(r0):
                        at = self.place(r)
                        v = decode(self.codes[x][pid, h, r, at], self.fmt) * had
                        self.codes[x][pid, h, r, at] = encode(v / s, self.fmt)
                new = np.where(np.isnan(new), 0.0, new)
                for r in range(r0, r1):
                    self.codes[x][pid, h, r, self.place(r)] = encode(new[r - r0] / s, self.fmt)
                self.scale[x][pid, h] = s

    def read(self, x, n, tokens):
        """Values [Hk, len(tokens), d]."""
        out = np.zeros((self.Hk, len(tokens), self.d))
        for i, t in enumerate(tokens):
            pid, r = self.table[n, t // self.P % self.S], t % self.P
            raw = self.codes[x][pid][:, r][:, self.place(r)]
            out[:, i] = decode(raw, self.fmt) * self.scale[x][pid].astype(np.float64)[:, None]
        return out


def attend(cache, q, pos, count, W=0, first=None, meta_k=None, meta_v=None, y_add=None, alpha=1.0,
           scale=None, rope=None):
    """q [N,H,T,d]; rope: None or (theta, layout, factor).  Returns y, and the sums the error
    bounds are made of: A = sum p |v| per channel and Z = max_t scale sum |q'||k| per row."""
    N, H, T, d = q.shape
    scale = scale or 1 / math.sqrt(d)
    y, A = np.zeros((N, H, T, d)), np.zeros((N, H, T, d))
    Z = np.zeros((N, H, T, 1))
    for n in range(N):
        cnt = T if count is None else int(count[n])
        p0, f0 = int(pos[n]), 0 if first is None else max(0, int(first[n]))
        lo0 = max(f0, p0 - W + 1 if W else 0, 0)
        toks = np.arange(lo0, max(lo0, p0 + cnt))
        K, V = cache.read("k", n, toks), cache.read("v", n, toks)
        for h in range(H):
            kh, vh = K[h // (H // cache.Hk)], V[h // (H // cache.Hk)]
            for t in range(cnt):
                see = (toks <= p0 + t) & (toks > p0 + t - W if W else True)
                qv = np.asarray(q[n, h, t], np.float64)
                qr = rotate(qv[None], [p0 + t], *rope)[0] if rope else qv
                kk, vv, qk = kh[see], vh[see], np.broadcast_to(qr, kh[see].shape)
                if meta_k is not None:
                    kk, vv = np.concatenate([meta_k[h], kk]), np.concatenate([meta_v[h], vv])
                    qk = np.concatenate([np.broadcast_to(qv, meta_k[h].shape), qk])
                if len(kk):
                    z = scale * (qk * kk).sum(1)
                    p = np.exp(z - z.max())
                    p /= p.sum()
                    y[n, h, t], A[n, h, t] = alpha * p @ vv, abs(alpha) * p @ np.abs(vv)
                    Z[n, h, t] = scale * (np.abs(qk) * np.abs(kk)).sum(1).max()
                if y_add is not None:
                    y[n, h, t] += y_add[n, h, t]
    return y, A, Z


def attend_bound(y, A, Z, dtype, d, L):
    """Elementwise bound of the attention's error.  Logits: the query's rounding (2^-11, in two
    parts 2^-22), d products summed in fp32, the rotation's 2^-21; a logit error e moves a
    probability by a factor 1 +- 2e.  Probabilities: rounding as the query's, exp2's 2^-21, L
    products summed in fp32.  Output: one rounding to its type."""
    part = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -22
    out = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -23
    dz = (part + 2.0 ** -21 + (d + 8) * 2.0 ** -23) * Z
    return out * np.abs(y) + (part + 2.0 ** -20 + (L + 8) * 2.0 ** -23 + 2 * dz) * A * 1.01 + 1e-30
