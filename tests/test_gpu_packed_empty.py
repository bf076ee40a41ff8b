"""The packed backward without queries, behind a call that left an error in the workspace."""
import pytest
import torch

from adaptive_block_sparse_fractal_b200 import nabla

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("keys", [1, 64, 700])
def test_no_query_after_an_error(keys, D):
    k, v = (torch.randn(keys, 2, D, device="cuda").to(BF) for _ in range(2))
    q = torch.empty(0, 4, D, dtype=BF, device="cuda")
    lse = torch.empty(4, 0, device="cuda")
    none = torch.zeros(2, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, keys], dtype=torch.int32, device="cuda")
    bad = torch.tensor([keys, 0], dtype=torch.int32, device="cuda")
    ws = nabla.packed_workspace(q, k, 1, back=True)
    for _ in range(20):
        dk, dv = (torch.full_like(t, 7.0) for t in (k, v))
        nabla.attn_packed_bwd(q, k, v, q, q, lse, none, bad, dk=dk, dv=dv, ws=ws)
        # (not waited for: the next call clears what this one leaves)
        dk2, dv2 = (torch.full_like(t, 7.0) for t in (k, v))
        nabla.attn_packed_bwd(q, k, v, q, q, lse, none, cu, dk=dk2, dv=dv2, ws=ws)
        assert nabla.status(ws) == nabla.OK
        assert bool((dk == 7).all()) and bool((dv == 7).all())
        assert bool((dk2 == 0).all()) and bool((dv2 == 0).all())
