"""Pools whose K and V are slices of one buffer, in every place that K and V can
take in it, and pools that overlap."""
import pytest
import torch

from adaptive_block_sparse_fractal_b200 import nabla

import seq_util

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
PAGES, PAGE, HEADS, D = 12, 16, 2, 64


def pools(layout):
    """k, v [pages, page, heads, D] and the buffer that holds them."""
    if layout == "pools":
        x = torch.randn(2, PAGES, PAGE, HEADS, D, device="cuda").to(BF)
        return x[0], x[1], x
    if layout == "pages":
        x = torch.randn(PAGES, 2, PAGE, HEADS, D, device="cuda").to(BF)
        return x[:, 0], x[:, 1], x
    if layout == "heads first":
        x = torch.randn(PAGES, HEADS, 2, PAGE, D, device="cuda").to(BF)
        return x[:, :, 0].transpose(1, 2), x[:, :, 1].transpose(1, 2), x
    if layout == "tokens":
        x = torch.randn(PAGES, PAGE, 2, HEADS, D, device="cuda").to(BF)
        return x[:, :, 0], x[:, :, 1], x
    x = torch.randn(PAGES, PAGE, HEADS, 2, D, device="cuda").to(BF)
    return x[..., 0, :], x[..., 1, :], x


@pytest.mark.parametrize("layout", ["pools", "pages", "heads first", "tokens", "rows"])
def test_append_then_attend(layout):
    kc, vc, whole = pools(layout)
    lens = [40, 1, 70]
    table = torch.randperm(PAGES, device="cuda").to(torch.int32)[:9].view(3, 3).contiguous()
    table = torch.cat([table, table[:, :2] * 0 - 1], 1).contiguous()
    table[2, 3:] = torch.tensor([p for p in range(PAGES) if p not in table[:, :3].flatten().tolist()][:2],
                                dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 40, 41, 111], dtype=torch.int32, device="cuda")
    k, v = (torch.randn(111, HEADS, D, device="cuda").to(BF) for _ in range(2))
    before = whole.clone()
    ws = nabla.cache_workspace("cuda")
    nabla.cache_append(k, v, kc, vc, table, torch.zeros(3, dtype=torch.int32, device="cuda"), cu=cu, ws=ws)
    assert nabla.status(ws) == nabla.OK
    for s, (a, n) in enumerate(zip(cu.tolist(), lens)):
        p = torch.arange(n, device="cuda")
        at = table[s, p // PAGE].long(), p % PAGE
        assert torch.equal(kc[at], k[a:a + n]) and torch.equal(vc[at], v[a:a + n])
    assert int((whole != before).any(-1).sum()) <= 2 * 111 * HEADS  # nothing but those rows
    q = torch.randn(3, 4, D, device="cuda").to(BF)
    o, lse = nabla.attn_paged(q, kc, vc, table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    for s, (a, n) in enumerate(zip(cu.tolist(), lens)):
        for h in range(4):
            x = seq_util.attention(q[s, h:h + 1].double(), k[a:a + n, h // 2].double(), v[a:a + n, h // 2].double(),
                                   D ** -0.5, torch.ones(1, n, dtype=torch.bool, device="cuda"))
            seq_util.check(o[s, h:h + 1], x["o"], x["o_tol"], "o")


def test_pools_that_share_rows_are_refused():
    x = torch.zeros(2 * PAGES * PAGE * HEADS * D + 64, dtype=BF, device="cuda")
    shape, stride = (PAGES, PAGE, HEADS, D), (PAGE * HEADS * D, HEADS * D, D, 1)
    at = lambda first: torch.as_strided(x, shape, stride, first)
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    k, v = (torch.randn(1, HEADS, D, device="cuda").to(BF) for _ in range(2))
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    for first in (0, 8, D, HEADS * D, PAGE * HEADS * D, (PAGES - 1) * PAGE * HEADS * D, PAGES * PAGE * HEADS * D - 8):
        with pytest.raises(nabla.NablaError) as e:
            nabla.cache_append(k, v, at(0), at(first), table, start)
        assert e.value.status == nabla.ERR_PARAM
    nabla.cache_append(k, v, at(0), at(PAGES * PAGE * HEADS * D), table, start)
    # rows given that lie in a pool
    for rows in (at(0)[3, 2:3], at(PAGES * PAGE * HEADS * D)[0, 0:1]):
        with pytest.raises(nabla.NablaError) as e:
            nabla.cache_append(rows, v, at(0), at(PAGES * PAGE * HEADS * D), table, start)
        assert e.value.status == nabla.ERR_PARAM
