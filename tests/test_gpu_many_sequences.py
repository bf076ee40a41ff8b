"""Thousands of short sequences: the work of a call grows with them, not with their square."""
import random

import pytest
import torch

from adaptive_block_sparse_fractal_b200 import nabla

import seq_util

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def borders(lens, first):
    out = [first]
    for n in lens:
        out.append(out[-1] + n)
    return out


@pytest.mark.parametrize("seqs,longest,same", [(33, 200, True), (1025, 70, False), (5000, 30, True), (5000, 30, False),
                                               (60000, 4, True)])
@pytest.mark.parametrize("D,heads,heads_kv", [(64, 2, 1), (128, 3, 3)])
def test_packed(seqs, longest, same, D, heads, heads_kv):
    rng = random.Random(seqs + D)
    lens_q = [rng.randrange(0, longest + 1) for _ in range(seqs)]
    lens_k = lens_q if same else [rng.randrange(0, longest + 1) for _ in range(seqs)]
    cq, ck = borders(lens_q, 7), borders(lens_k, 7 if same else 100)
    g = torch.Generator(device="cuda").manual_seed(seqs)
    new = lambda n, h: torch.randn(n + 5, h, D, generator=g, device="cuda").to(BF)  # 5 rows behind the last
    q, k, v, dout = new(cq[-1], heads), new(ck[-1], heads_kv), new(ck[-1], heads_kv), new(cq[-1], heads)
    cu_q, cu_k = dev(cq), dev(ck)
    ws = nabla.packed_workspace(q, k, seqs, back=True)
    full = lambda t: torch.full_like(t, 7.0)
    o, dq, dk, dv = full(q), full(q), full(k), full(k)
    _, lse = nabla.attn_packed_fwd(q, k, v, cu_q, cu_k, causal=True, o=o, ws=ws)
    assert nabla.status(ws) == nabla.OK
    nabla.attn_packed_bwd(q, k, v, o, dout, lse, cu_q, cu_k, causal=True, dq=dq, dk=dk, dv=dv, ws=ws)
    assert nabla.status(ws) == nabla.OK
    n = 25
    for at in (0, seqs // 3, seqs - n):
        r = seq_util.packed(q, k, v, cq[at:at + n + 1], ck[at:at + n + 1], True, dout=dout)
        seq_util.check(o, r["o"], r["o_tol"], "o")
        for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
            seq_util.check(t, r[name], r[name + "_tol"], name)
    for t, c in ((o, cq), (dq, cq), (dk, ck), (dv, ck)):
        assert bool((t[:c[0]] == 7).all()) and bool((t[c[-1]:] == 7).all())
        assert bool((t[c[0]:c[-1]] != 7).any(-1).all())  # each row was written (none is all sevens)
    # one bad border among them
    for c, name in ((cq, "q"), (ck, "k")):
        for at in (1, seqs // 2, seqs):
            bad = list(c)
            bad[at] = c[-1] + 6 if at != 1 else -1
            o2, g2 = full(q), [full(q), full(k), full(k)]
            b = (dev(bad), cu_k) if name == "q" else (cu_q, dev(bad))
            nabla.attn_packed_fwd(q, k, v, *b, causal=True, o=o2, ws=ws)
            assert nabla.status(ws) == nabla.ERR_PARAM and bool((o2 == 7).all())
            nabla.attn_packed_bwd(q, k, v, o, dout, lse, *b, causal=True, dq=g2[0], dk=g2[1], dv=g2[2], ws=ws)
            assert nabla.status(ws) == nabla.ERR_PARAM and all(bool((t == 7).all()) for t in g2)


def test_bad_borders_without_queries():
    k, v = (torch.randn(50, 2, 64, device="cuda").to(BF) for _ in range(2))
    q, lse = torch.empty(0, 2, 64, dtype=BF, device="cuda"), torch.empty(2, 0, device="cuda")
    ws = nabla.packed_workspace(q, k, 2, back=True)
    for cq, ck, want in (([0, 0, 0], [0, 51, 50], nabla.ERR_PARAM), ([0, 1, 0], [0, 20, 50], nabla.ERR_PARAM),
                         ([0, 0, 0], [10, 20, 50], nabla.OK)):
        dk, dv = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
        nabla.attn_packed_bwd(q, k, v, q, q, lse, dev(cq), dev(ck), dk=dk, dv=dv, ws=ws)
        assert nabla.status(ws) == want
        for t in (dk, dv):
            assert bool((t[:10] == 7).all())
            assert bool((t[10:] == (7 if want else 0)).all())
