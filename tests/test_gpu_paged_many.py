"""Attention of one token for many sequences: empty, short and shared ones."""
import math
import random

import pytest
import torch

from adaptive_block_sparse_fractal_b200 import nabla

import seq_util

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


# 257 x 10 and more have more (sequence, head) rows than CTAs that run at once
@pytest.mark.parametrize("seqs,longest,heads,heads_kv", [(256, 300, 10, 2), (257, 300, 10, 2), (700, 90, 20, 1),
                                                         (3000, 40, 4, 2), (20000, 3, 2, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_many_sequences(seqs, longest, heads, heads_kv, D):
    rng = random.Random(seqs)
    lens = [rng.choice([0, 1, rng.randrange(longest + 1)]) for _ in range(seqs)]
    for s in (0, seqs // 2, seqs - 1):
        lens[s] = 4 * longest + 5
    lens[1] = lens[seqs - 2] = 0
    page, G = 16, heads // heads_kv
    width = -(-max(lens) // page)
    pages = 400
    g = torch.Generator(device="cuda").manual_seed(seqs)
    kc, vc = (torch.randn(pages, page, heads_kv, D, generator=g, device="cuda").to(BF) for _ in range(2))
    table = torch.randint(0, pages, (seqs, width), generator=g, device="cuda").to(torch.int32)  # pages are shared
    q = torch.randn(seqs, heads, D, generator=g, device="cuda").to(BF)
    dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = nabla.paged_workspace(q, kc)
    ws.fill_(255)
    o, lse = torch.full_like(q, 7.0), torch.full((seqs, heads), 7.0, device="cuda")
    nabla.attn_paged(q, kc, vc, table, dl, o=o, lse=lse, ws=ws)
    assert nabla.status(ws) == nabla.OK
    empty = dl == 0
    assert bool((o[empty] == 0).all()) and bool((lse[empty] == -math.inf).all())
    assert bool(torch.isfinite(o).all()) and bool((o[~empty] != 7).any(-1).all())
    for s in {0, 2, 3, seqs // 2, seqs // 2 + 1, seqs - 3, seqs - 1} | {rng.randrange(seqs) for _ in range(25)}:
        n = lens[s]
        if n == 0:
            continue
        p = torch.arange(n, device="cuda")
        at = table[s, p // page].long(), p % page
        keep = torch.ones(1, n, dtype=torch.bool, device="cuda")
        for h in range(heads):
            x = seq_util.attention(q[s, h:h + 1].double(), kc[at][:, h // G].double(), vc[at][:, h // G].double(),
                                   D ** -0.5, keep)
            seq_util.check(o[s, h:h + 1], x["o"], x["o_tol"], "o")
            seq_util.check_lse(lse[s, h:h + 1], x["lse"])
    again = nabla.attn_paged(q, kc, vc, table, dl, ws=ws)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)
    dl[seqs - 5] = -1
    bad, _ = nabla.attn_paged(q, kc, vc, table, dl, ws=ws)
    assert nabla.status(ws) == nabla.ERR_PARAM and bool((bad[seqs - 5] == 0).all())
