"""One attention workspace for calls of different shapes, one after the other."""
import pytest

import hybrid_gated_linear_gb300 as lz
from cache_gpu_util import Filled, attend, gaussian, workspace

pytestmark = pytest.mark.gpu

SHAPES = [  # N, H, Hk, d, T, dtype, tokens held
    (1, 32, 8, 128, 1, "bf16", [4000]),                             # one sequence in many parts
    (16, 32, 8, 128, 1, "bf16", [500 + 37 * n for n in range(16)]),  # a batch that has grown
    (2, 8, 2, 128, 200, "bf16", [2000, 900]),                       # a chunk of a prompt
    (2, 8, 2, 64, 40, "f32", [1000, 3000]),                         # many rows in fp32
    (40, 8, 8, 64, 1, "bf16", [60 * n + 1 for n in range(40)]),     # a warp per sequence and head
    (80, 32, 32, 64, 1, "bf16", [1 + 5 * n for n in range(80)]),     # more of them than warps
    (100, 32, 8, 64, 1, "bf16", [1 + 30 * n for n in range(100)]),  # grouped heads
    (3, 6, 3, 64, 20, "bf16", [1500, 20, 700]),
    (8, 16, 8, 64, 600, "bf16", [600 + 150 * n for n in range(8)]),  # prompts in many tiles
]


def test_calls_of_any_shape_may_share_a_workspace():
    """Every shape after every other: what a call leaves in the workspace (parts of results of
    another shape) must not be taken for this call's own bookkeeping.  Equal bit for bit to the
    same call with a workspace of its own."""
    import torch
    calls = []
    for i, (N, H, Hk, d, T, dtype, held) in enumerate(SHAPES):
        k, v = (gaussian((N, Hk, max(held), d), 2 * i + j) for j in range(2))
        f = Filled(k, v, [0] * N, held, 64, "e4m3")
        q = gaussian((N, H, T, d), 100 + i, 1.5).to(torch.float32 if dtype == "f32" else torch.bfloat16)
        pos = [h - T for h in held]
        calls.append((f, q, pos, attend(f, q, pos)))
    size = 0
    for f, q, pos, _ in calls:
        dims = lz.lizard_cache_attn_dims(q.shape[1], q.shape[2], 0, 0, int(q.dtype == torch.bfloat16), 0.0, 1.0)
        size = max(size, workspace(f, dims).numel())
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    order = [0]
    for a in range(len(calls)):
        for b in range(len(calls)):
            order += [a, b]
    for i in order:
        f, q, pos, want = calls[i]
        assert torch.equal(attend(f, q, pos, ws=ws), want), SHAPES[i]
