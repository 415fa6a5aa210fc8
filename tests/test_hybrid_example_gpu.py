"""The example's hybrid layer end to end on the GPU: prompt in chunks and decode agree with the
gated recurrence plus the 64-bit softmax over the cache's values.

Tolerance: the operator's bf16 parity bound (relative L2 2e-2), with the keys and values taken
from the cache itself, so that the quantisation is not part of the difference."""
import os
import sys

import numpy as np
import pytest

import cache_oracle as co
import hybrid_gated_linear_gb300 as lz
import oracle
from gpu_util import rel_l2

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("fmt,W,L", [(0, 0, 150), (1, 100, 150), (0, 70, 1100)])
def test_hybrid_layer(fmt, W, L):
    import hybrid_decode as ex
    import torch
    N, H, Hk, S = 2, 4, 2, 3
    layer = ex.HybridLayer(N, H, Hk, W, longest=2048, fmt=fmt, alpha=0.5)
    x = ex.tokens(N, H, Hk, L + S, 3)
    y = [layer.prompt(**{n: t[:, :, :L].contiguous() for n, t in x.items()})]
    for i in range(S):
        y.append(layer.step(**{n: t[:, :, L + i].contiguous() for n, t in x.items()})[:, :, None])
    layer.check()
    got = _np(torch.cat(y, 2))
    rep = {n: np.repeat(_np(x[n]), H // Hk, 1) for n in ("v",)}
    zero = np.zeros((H, 0, 128), np.float32)
    f = {n: _np(x[n]).astype(np.float32) for n in ("phi_q", "phi_k", "log_gamma", "q")}
    gla = oracle.fwd(f["phi_q"], f["phi_k"], rep["v"].astype(np.float32), f["log_gamma"], f["q"], f["q"], zero, zero,
                     W=1, alpha=0.0)["y"]
    # the cache's own values (a window's ring holds the last tokens only: check those)
    first = 0 if not W else L + S - W - 4
    T = L + S - first
    vals = [torch.empty(N, Hk, T, 128, device="cuda") for _ in "kv"]
    pos = torch.full((N,), first, dtype=torch.int64, device="cuda")
    lz.lizard_cache_read(layer.cache, lz.lizard_cache_io(T, lz.LIZARD_F32), pos, None, *vals, layer.cache_ws)
    K, V = (np.repeat(_np(t), H // Hk, 1) for t in vals)
    th, mk, mv = co.theta(128), _np(layer.meta_k), _np(layer.meta_v)
    q = _np(x["q"])
    for t in range(L + S - 4, L + S):
        lo = max(0, t - W + 1) if W else 0
        qr = co.rotate(q[:, :, t:t + 1], [t], th)
        for n in range(N):
            for h in range(H):
                k, v = K[n, h, lo - first:t + 1 - first], V[n, h, lo - first:t + 1 - first]
                z = np.concatenate([mk[h] @ q[n, h, t], k @ qr[n, h, 0]]) / np.sqrt(128)
                p = np.exp(z - z.max())
                want = gla[n, h, t] + 0.5 * (p / p.sum()) @ np.concatenate([mv[h], v])
                assert rel_l2(got[n, h, t], want) < 2e-2
