"""Prompt and decode of one hybrid layer: the gated branch next to softmax attention over an
8-bit paged cache.

A prompt runs through lizard_attn_fwd for the gated branch alone (alpha = 0) and leaves its
state; its keys go into the cache, rotated and in 8 bits, and the prompt's own queries attend
to them.  Then tokens are decoded one by one: lizard_decode_step advances the state and writes
the gated output, lizard_cache_write adds the token, and lizard_cache_attn reads the window and
adds it to the gated output in place,

    y = y_gla + alpha * softmax([q . meta_k ; rotate(q) . k]) [meta_v ; v].

Run on a GB300 after building the library:  python examples/hybrid_decode.py [--format i8]
[--window 512] [--steps 64]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import hybrid_gated_linear_gb300 as lz  # noqa: E402

BF = torch.bfloat16


class HybridLayer:
    """N sequences, H query heads over Hk key heads of 128 channels; W = 0: no window."""

    def __init__(self, N, H, Hk, W, M=4, page=64, longest=4096, fmt=lz.LIZARD_KV_E4M3, alpha=1.0, seed=0):
        self.N, self.H, self.Hk, self.W, self.M, self.d, self.alpha = N, H, Hk, W, M, 128, alpha
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.meta_k, self.meta_v = (torch.randn(H, M, 128, generator=g, device="cuda").to(BF) for _ in "kv")
        # a window needs only the pages it overlaps, used as a ring
        span = min(W, longest) if W else longest
        self.max_new = min(longest, 1024)  # tokens of a prompt chunk
        slots = (span + self.max_new + page - 2) // page + 1
        pages = N * slots
        self.table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(N, slots)
        self.codes = [torch.empty(pages, Hk, page, 128, dtype=torch.uint8, device="cuda") for _ in "kv"]
        self.scales = [torch.empty(pages, Hk, device="cuda") for _ in "kv"]
        self.cache = lz.lizard_cache(*self.codes, *self.scales, self.table, fmt)
        spec = lz.lizard_rope_spec(128, lz.LIZARD_ROPE_PLAIN, 500000.0, 1.0, 1.0, 4.0, 8192)
        self.rope = lz.lizard_rope(lz.lizard_rope_table(spec).cuda(), 128, lz.LIZARD_ROPE_HALF)
        self.pos = torch.zeros(N, dtype=torch.int64, device="cuda")
        # the gated branch's state; its own one-slot ring is not used (alpha = 0)
        self.h = torch.zeros(N, H, 128, 128, device="cuda")
        self.ring = [torch.zeros(N, H, 1, 128, dtype=BF, device="cuda") for _ in "kv"]
        self.gla_pos = torch.zeros(N, dtype=torch.int64, device="cuda")
        self.step_dims = lz.lizard_decode_dims(N, H, 128, 128, 0, lz.LIZARD_BF16, 0.0)
        self.step_ws = torch.zeros(lz.lizard_decode_workspace_bytes(self.step_dims), dtype=torch.uint8, device="cuda")
        self.cache_ws = torch.zeros(lz.lizard_cache_workspace_bytes(), dtype=torch.uint8, device="cuda")
        self.attn = {}

    def _attend(self, q, k, v, y, T):
        """Adds the tokens to the cache and their attention to y."""
        if T not in self.attn:
            dims = lz.lizard_cache_attn_dims(self.H, T, self.M, self.W, lz.LIZARD_BF16, 0.0, self.alpha)
            ws = torch.zeros(lz.lizard_cache_attn_workspace_bytes(self.cache, dims), dtype=torch.uint8, device="cuda")
            self.attn[T] = (dims, ws, lz.lizard_cache_io(T, lz.LIZARD_BF16))
        dims, ws, io = self.attn[T]
        lz.lizard_cache_write(self.cache, io, k, v, self.rope, self.pos, None, self.cache_ws)
        lz.lizard_cache_attn(self.cache, dims, q, self.rope, self.pos, None, None, self.meta_k, self.meta_v, y, y, ws)
        self.pos += T

    def prompt(self, phi_q, phi_k, log_gamma, q, k, v):
        """phi_q, phi_k, q [N,H,L,128], k, v [N,Hk,L,128] bf16, log_gamma fp32; returns y."""
        L = q.shape[2]
        y = torch.empty_like(q)
        dims = lz.lizard_dims(self.N, self.H, L, 128, 128, 0, lz.LIZARD_BF16, 0.0)
        ws = torch.zeros(lz.lizard_fwd_workspace_bytes(dims, 1), dtype=torch.uint8, device="cuda")
        vq = v.repeat_interleave(self.H // self.Hk, 1).contiguous()
        h0 = self.h.clone()
        # window 1 with weight 0: the gated branch alone
        lz.lizard_attn_fwd(dims, phi_q, phi_k, vq, log_gamma, q, q, None, None, 1, 0.0, y, h0, self.h, ws)
        assert lz.lizard_check_device_errors(ws) == 0
        for a in range(0, L, self.max_new):
            b = min(L, a + self.max_new)
            self._attend(q[:, :, a:b], k[:, :, a:b], v[:, :, a:b], y[:, :, a:b], b - a)
        self.gla_pos += L
        return y

    def step(self, phi_q, phi_k, log_gamma, q, k, v):
        """One token: phi_q, phi_k, q [N,H,128], k, v [N,Hk,128]; returns y [N,H,128]."""
        y = torch.empty_like(q)
        vq = v.repeat_interleave(self.H // self.Hk, 1).contiguous()
        lz.lizard_decode_step(self.step_dims, phi_q, phi_k, vq, log_gamma, q, q, None, None, 1, 0.0, self.h,
                              *self.ring, self.gla_pos, y, self.step_ws)
        self._attend(q[:, :, None], k[:, :, None], v[:, :, None], y[:, :, None], 1)
        return y

    def check(self):
        """Raises if a call found a bad page, position or value."""
        for ws in [self.step_ws, self.cache_ws] + [ws for _, ws, _ in self.attn.values()]:
            status = lz.lizard_check_device_errors(ws)
            if status:
                raise lz.LizardError(status, "hybrid layer")


def tokens(N, H, Hk, L, seed):
    """Random inputs of L tokens with the distributions of a layer."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda h: torch.randn(N, h, L, 128, generator=g, device="cuda")  # noqa: E731
    phi = lambda: (0.1 * torch.exp(0.5 * r(H))).to(BF)  # noqa: E731
    return dict(phi_q=phi(), phi_k=phi(), log_gamma=torch.nn.functional.logsigmoid(r(H) + 2) / 16,
                q=r(H).to(BF), k=r(Hk).to(BF), v=r(Hk).to(BF))


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--format", choices=("e4m3", "i8"), default="e4m3")
    p.add_argument("--window", type=int, default=0)
    p.add_argument("--prompt", type=int, default=1500)
    p.add_argument("--steps", type=int, default=64)
    a = p.parse_args()
    N, H, Hk = 8, 32, 8
    layer = HybridLayer(N, H, Hk, a.window, fmt=lz.LIZARD_KV_E4M3 if a.format == "e4m3" else lz.LIZARD_KV_I8)
    x = tokens(N, H, Hk, a.prompt + a.steps, 1)
    y = layer.prompt(**{n: t[:, :, :a.prompt].contiguous() for n, t in x.items()})
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    steps = [{n: t[:, :, a.prompt + i].contiguous() for n, t in x.items()} for i in range(a.steps)]
    warm = min(4, a.steps // 2)  # first calls load kernels
    for s in steps[:warm]:
        y = layer.step(**s)
    start.record()
    for s in steps[warm:]:
        y = layer.step(**s)
    end.record()
    torch.cuda.synchronize()
    layer.check()
    assert torch.isfinite(y).all()
    held = sum(c.numel() for c in layer.codes) + 4 * sum(s.numel() for s in layer.scales)
    print(f"{N} sequences at position {int(layer.pos[0])}: {start.elapsed_time(end) / (a.steps - warm) * 1e3:.1f} us per step, "
          f"cache {held / 2 ** 20:.0f} MiB in {a.format}")


if __name__ == "__main__":
    main()
