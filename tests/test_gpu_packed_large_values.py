"""Values of v so large that a weight taken against an early reference carries them
out of float32, though the row itself stays inside (bounds in seq_util.py)."""
import pytest
import torch

from adaptive_block_sparse_fractal_b200 import nabla

import seq_util

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("scale_v", [1e18, 1e24, 1e32])
@pytest.mark.parametrize("step", [10.0, 36.0, 40.0])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,keys", [(1, 512), (1, 9000), (300, 700)])
def test_rising_scores_and_large_values(scale_v, step, D, rows, keys):
    """Scores rise by `step` behind the first tile: up to 2^58 of weight, below what the
    row's sum is tested for.  (One row on 9,000 keys: the key range is split.)"""
    g = torch.Generator(device="cuda").manual_seed(int(step))
    q = torch.zeros(rows, 2, D, dtype=BF, device="cuda")
    q[:, :, 0] = 1.0
    k = torch.zeros(keys, 1, D, dtype=BF, device="cuda")
    k[keys // 2:, :, 0] = step
    v = (torch.randn(keys, 1, D, generator=g, device="cuda") * scale_v).to(BF)
    cu = lambda n: torch.tensor([0, n], dtype=torch.int32, device="cuda")
    ws = nabla.packed_workspace(q, k, 1)
    for causal in (False, True):
        o, lse = nabla.attn_packed_fwd(q, k, v, cu(rows), cu(keys), causal=causal, scale=1.0, ws=ws)
        assert nabla.status(ws) == nabla.OK
        r = seq_util.packed(q, k, v, [0, rows], [0, keys], causal, scale=1.0)
        seq_util.check(o, r["o"], r["o_tol"], "o")
        seq_util.check_lse(lse, r["lse"])
