"""Gradients of rows that keep few keys inside longer sequences: delta = dout . o
must not carry the rounding of o there, whatever tile the row shares.  Bounds:
dS is rounded to bf16 once (H |dS|) and P (dP - delta) has float32 errors E against
its terms; only rows of more than 64 keys have P |ddelta| besides, ddelta being
|dout| times the bound of o.  The constants are derived in seq_util.py."""
import math

import pytest
import torch

from adaptive_block_sparse_fractal_b200 import nabla

import seq_util

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
FEW = 64

CASES = [
    # lens_q, lens_k: one behind another, causal
    ([65], [65]), ([128], [128]), ([129], [129]), ([1000], [1000]), ([65, 3, 1000, 128, 64], [65, 3, 1000, 128, 64]),
    ([300], [340]),       # rows keep 41 and more
    ([300], [364]),       # none keeps fewer than 65
    ([400], [150]),       # 250 rows keep nothing, the next 64 few
    ([330, 70], [90, 200]),
]


def grads(q, k, v, dout, cu_q, cu_k, seqs):
    ws = nabla.packed_workspace(q, k, seqs, back=True)
    o, lse = nabla.attn_packed_fwd(q, k, v, cu_q, cu_k, causal=True, ws=ws)
    out = nabla.attn_packed_bwd(q, k, v, o, dout, lse, cu_q, cu_k, causal=True, ws=ws)
    assert nabla.status(ws) == nabla.OK
    return out


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("heads,heads_kv", [(2, 2), (6, 2), (5, 1)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("only_few", [False, True])
def test_rows_with_few_keys(case, heads, heads_kv, D, only_few):
    lens_q, lens_k = CASES[case]
    G = heads // heads_kv
    g = torch.Generator(device="cuda").manual_seed(31 + case)
    borders = lambda lens: [sum(lens[:i]) for i in range(len(lens) + 1)]
    cq, ck = borders(lens_q), borders(lens_k)
    new = lambda n, h: torch.randn(n, h, D, generator=g, device="cuda").to(BF)
    q, k, v, dout = new(cq[-1], heads), new(ck[-1], heads_kv), new(ck[-1], heads_kv), new(cq[-1], heads)
    kept = torch.cat([torch.arange(1, n + 1, device="cuda") + m - n for n, m in zip(lens_q, lens_k)])
    if only_few:  # dk is then made by the rows with few keys alone
        dout[kept > FEW] = 0
    cu_q, cu_k = (torch.tensor(c, dtype=torch.int32, device="cuda") for c in (cq, ck))
    dq, dk, _ = grads(q, k, v, dout, cu_q, cu_k, len(lens_q))
    sc, H, E = D ** -0.5, seq_util.H, seq_util.E
    for a, b, c, e in zip(cq, cq[1:], ck, ck[1:]):
        want, tol = {}, {}
        keep = seq_util.keep_mask(b - a, e - c, True, "cuda")
        many = (kept[a:b] > FEW).double()[:, None]
        for h in range(heads):
            Q, K, V, Y = q[a:b, h].double(), k[c:e, h // G].double(), v[c:e, h // G].double(), dout[a:b, h].double()
            x = seq_util.attention(Q, K, V, sc, keep, Y)
            p = ((Q @ K.T) * sc).masked_fill(~keep, -math.inf)
            p = torch.where(keep, torch.softmax(p, 1), torch.zeros_like(p))  # (a row that keeps nothing has p = 0)
            dp, delta = Y @ V.T, (Y * x["o"]).sum(1, keepdim=True)
            ds = p * (dp - delta)
            dds = H * ds.abs() + E * p * (Y.abs() @ V.abs().T + (Y * x["o"]).abs().sum(1, keepdim=True))
            dds = dds + many * (E * ds.abs() + p * (Y.abs() * x["o_tol"]).sum(1, keepdim=True))
            seq_util.check(dq[a:b, h], x["dq"], (dds @ K.abs()) * sc + H * x["dq"].abs(), "dq")
            j = h // G
            want[j] = want.get(j, 0) + x["dk"]
            tol[j] = tol.get(j, 0) + (dds.T @ Q.abs()) * sc
        for j in want:
            seq_util.check(dk[c:e, j], want[j], tol[j] + H * want[j].abs(), "dk")
