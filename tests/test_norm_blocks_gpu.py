"""The norm's backward where every block of a round takes many rows: widths on both sides of the rule for the
blocks that an SM holds, each type, with as many rows as need several turns of every block."""
import pytest

torch = pytest.importorskip("torch")

import hybrid_gated_linear_gb300 as lz
from test_norm_gpu import In

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [272, 512, 520, 544, 768, 776, 1024, 1096, 2048])
def test_many_rows(d, dtype):
    In(1, 1, 3000 if d < 1000 else 1700, d, dtype).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sums_follow_the_last_row(dtype):
    """The sums of a block's rows lie where its rows did: the same bits call after call, a workspace's
    content and other calls in between notwithstanding."""
    x, z = In(1, 1, 2500, 512, dtype), In(2, 5, 300, 128, dtype, per_head=True)
    ws = torch.full((max(lz.lizard_layer_norm_workspace_bytes(i.dims) for i in (x, z)),), 255, dtype=torch.uint8, device="cuda")
    want = x.bwd(), z.bwd()
    for _ in range(5):
        for i, w in zip((x, z), want):
            assert all(torch.equal(p, q) for p, q in zip(w, i.bwd(ws=ws)))
