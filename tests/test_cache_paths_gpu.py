"""The ways in which cache attention shares out its work, against the definition in 64 bits over the
cache's own values: a warp per (sequence, head) and a CTA per block of rows, equal pieces and equal
shares of one list (more segments than teams, or one far longer than the rest), several pieces and
two partial results per team, a ring of pages under a window, uneven counts and hidden rows.
Tolerance: cache_oracle.attend_bound."""
import pytest

from cache_gpu_util import Filled, check_attention, gaussian
from test_rope_gpu import make_rope

pytestmark = pytest.mark.gpu


def lengths(kind, N, most):
    if kind == "even":
        return [most] * N
    if kind == "one long":
        return [most if n == N // 2 else 1 + 37 * n % 90 for n in range(N)]
    return [1 + (most - 1) * (n * 13 % N) // N for n in range(N)]  # spread


CASES = {
    # name: N, H, Hk, P, d, T, dtype, fmt, lengths, most, W, M, rope, first, counts, add
    # a warp per (sequence, head)
    "warps, pieces": (40, 16, 8, 64, 128, 1, "bf16", "e4m3", "spread", 900, 0, 0, True, False, False, False),
    "warps, pieces, one long": (33, 8, 8, 16, 64, 1, "bf16", "i8", "one long", 9000, 0, 3, False, True, False, True),
    "warps, pieces, fp32": (16, 32, 16, 32, 128, 3, "f32", "i8", "spread", 500, 0, 0, True, False, True, False),
    "warps, list": (80, 32, 32, 64, 64, 1, "bf16", "e4m3", "spread", 400, 0, 0, True, False, False, False),
    "warps, list, one long": (80, 32, 32, 16, 64, 1, "bf16", "e4m3", "one long", 6000, 0, 2, True, True, False, True),
    "warps, list, window": (80, 32, 32, 32, 128, 1, "bf16", "i8", "spread", 700, 150, 4, False, False, False, True),
    "warps, list, fp32": (43, 60, 30, 64, 128, 4, "f32", "e4m3", "spread", 1500, 0, 1, True, False, True, True),
    # a CTA per 16 rows
    "16 rows, pieces": (5, 20, 4, 64, 128, 3, "bf16", "e4m3", "spread", 20000, 0, 2, True, True, True, False),
    "16 rows, list": (30, 16, 8, 64, 64, 1, "bf16", "i8", "even", 4700, 0, 0, True, False, False, True),
    "16 rows, list, fp32": (30, 8, 8, 128, 64, 5, "f32", "e4m3", "even", 4700, 0, 0, False, False, True, False),
    # 32, 64 and 128 rows
    "32 rows, pieces": (2, 8, 2, 64, 64, 7, "bf16", "e4m3", "spread", 5000, 0, 0, True, False, False, False),
    "32 rows, list": (40, 32, 8, 16, 64, 6, "bf16", "i8", "spread", 900, 0, 3, True, True, True, True),
    "32 rows, list, fp32": (41, 8, 8, 64, 128, 25, "f32", "e4m3", "one long", 4000, 33, 0, True, False, True, False),
    "64 rows, pieces": (3, 12, 3, 32, 128, 15, "bf16", "i8", "spread", 2500, 0, 4, True, False, True, True),
    "64 rows, list": (45, 32, 8, 64, 64, 12, "bf16", "e4m3", "spread", 800, 0, 0, True, True, True, False),
    "64 rows, list, fp32": (45, 16, 8, 64, 128, 30, "f32", "i8", "spread", 900, 0, 2, False, False, True, True),
    "128 rows, pieces, fp32": (1, 6, 2, 128, 64, 70, "f32", "e4m3", "even", 3000, 0, 0, True, False, False, False),
    "128 rows, list, fp32": (12, 16, 8, 64, 128, 100, "f32", "e4m3", "spread", 900, 0, 3, True, True, True, True),
    # tcgen05
    "tcgen05, pieces": (2, 8, 2, 64, 128, 300, "bf16", "i8", "spread", 5000, 0, 2, True, False, True, True),
    "tcgen05, list": (7, 16, 8, 64, 128, 300, "bf16", "e4m3", "spread", 3000, 0, 0, True, False, False, False),
    "tcgen05, list, one long": (40, 8, 8, 16, 64, 90, "bf16", "i8", "one long", 9000, 0, 4, True, True, True, True),
    "tcgen05, list, window": (40, 16, 4, 32, 64, 130, "bf16", "e4m3", "spread", 3000, 200, 1, False, False, False, True),
}


@pytest.mark.parametrize("name", CASES)
def test_attention_work_sharing(name):
    import torch
    N, H, Hk, P, d, T, dtype, fmt, kind, most, W, M, rope, first, counts, add = CASES[name]
    pos = lengths(kind, N, most)
    count = [n * 11 % (T + 1) for n in range(N)] if counts else None
    end = [p + (T if count is None else c) for p, c in zip(pos, count or pos)]
    lo = [max(0, p - W + 1) // P * P if W else 0 for p in pos]
    # a window's table is a ring of the pages that the new tokens and their windows touch
    slots = max((e - 1) // P - a // P + 1 for a, e in zip(lo, end)) if W else None
    rows = max(e - a for a, e in zip(lo, end))
    k, v = gaussian((N, Hk, rows, d), 1), gaussian((N, Hk, rows, d), 2)
    f = Filled(k, v, lo, end, P, fmt, slots)
    typed = [x.to(torch.float32 if dtype == "f32" else torch.bfloat16)
             for x in (gaussian((N, H, T, d), 3, 1.5), gaussian((N, H, T, d), 4), gaussian((2, H, M, d), 5))]
    kw = dict(W=W, count=count, alpha=0.7)
    if first:  # some sequences see nothing, some a part
        kw["first"] = [p + T if n % 5 == 4 else p * (n % 3) // 3 for n, p in enumerate(pos)]
    if M:
        kw["meta"] = (typed[2][0], typed[2][1])
    if add:
        kw["y_add"] = typed[1]
    if rope:
        kw["rope"] = make_rope(d)
    y = check_attention(f, typed[0], pos, **kw)
    again = check_attention(f, typed[0], pos, **kw)
    assert torch.equal(y, again)
