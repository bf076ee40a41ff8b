"""Captured calls replayed on other inputs, borders and lengths: what lives on the
device may change between replays, bad values among it."""
import pytest
import torch

from adaptive_block_sparse_fractal_b200 import nabla

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def capture(f):
    f()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f()
    return g


@pytest.mark.parametrize("D", [64, 128])
def test_split_forward(D):
    """Few rows on many keys: two launches, the second beside the first."""
    q, k, v = (torch.randn(n, h, D, device="cuda").to(BF) for n, h in ((4, 4), (9000, 2), (9000, 2)))
    cq, ck = dev([0, 1, 4]), dev([0, 4000, 9000])
    ws = nabla.packed_workspace(q, k, 2)
    assert ws.numel() > 256
    o, lse = torch.empty_like(q), torch.empty(4, 4, device="cuda")
    call = lambda ws, **kw: nabla.attn_packed_fwd(q, k, v, cq, ck, causal=True, ws=ws, **kw)
    g = capture(lambda: call(ws, o=o, lse=lse))
    for b_q, b_k, want in (([0, 1, 4], [0, 4000, 9000], nabla.OK), ([0, 3, 3], [8000, 8001, 9000], nabla.OK),
                           ([0, 5, 4], [0, 4000, 9000], nabla.ERR_PARAM), ([1, 2, 4], [0, 0, 9000], nabla.OK)):
        cq.copy_(dev(b_q))
        ck.copy_(dev(b_k))
        q.copy_(torch.randn_like(q, dtype=torch.float32))
        o.fill_(7.0)
        lse.fill_(7.0)
        for _ in range(2):
            g.replay()
        assert nabla.status(ws) == want
        other = nabla.packed_workspace(q, k, 2)
        o2, lse2 = torch.full_like(o, 7.0), torch.full_like(lse, 7.0)
        call(other, o=o2, lse=lse2)
        assert nabla.status(other) == want
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("D", [64, 128])
def test_training_step(D):
    total = 900
    q, k, v, dout = (torch.randn(total, h, D, device="cuda").to(BF) for h in (6, 2, 2, 6))
    cu = dev([0, 300, 900, 900, 900])
    ws = nabla.packed_workspace(q, k, 4, back=True)
    o, lse = torch.empty_like(q), torch.empty(6, total, device="cuda")
    grads = [torch.empty_like(t) for t in (q, k, v)]

    def step(ws, o, lse, dq, dk, dv):
        nabla.attn_packed_fwd(q, k, v, cu, cu, causal=True, o=o, lse=lse, ws=ws)
        nabla.attn_packed_bwd(q, k, v, o, dout, lse, cu, cu, causal=True, dq=dq, dk=dk, dv=dv, ws=ws)
    g = capture(lambda: step(ws, o, lse, *grads))
    for b, want in (([0, 300, 900, 900, 900], nabla.OK), ([0, 30, 31, 33, 900], nabla.OK),
                    ([10, 60, 50, 70, 900], nabla.ERR_PARAM), ([5, 5, 5, 5, 5], nabla.OK),
                    ([5, 64, 128, 200, 264], nabla.OK)):
        cu.copy_(dev(b))
        q.copy_(torch.randn_like(q, dtype=torch.float32))
        mine = [torch.full_like(t, 7.0) for t in (o, lse, *grads)]
        for t in (o, lse, *grads):
            t.fill_(7.0)
        for _ in range(2):
            g.replay()
        assert nabla.status(ws) == want
        other = nabla.packed_workspace(q, k, 4, back=True)
        step(other, *mine)
        assert nabla.status(other) == want
        for a, b2 in zip((o, lse, *grads), mine):
            assert torch.equal(a, b2)


@pytest.mark.parametrize("total", [200, 3000])  # the status by the kernel, and by a memset in front of it
def test_prompts_into_the_cache_and_a_token(total):
    heads_kv, D, page, width = 2, 128, 16, 300
    k, v = (torch.randn(total, heads_kv, D, device="cuda").to(BF) for _ in range(2))
    kc, vc = (torch.zeros(2 * width, page, heads_kv, D, dtype=BF, device="cuda") for _ in range(2))
    table = torch.randperm(2 * width, device="cuda").to(torch.int32).view(2, width)
    starts, cu, lens = dev([0, 0]), dev([0, 100, total]), dev([100, total - 100])
    q = torch.randn(2, 8, D, device="cuda").to(BF)
    ws, pws, o = nabla.cache_workspace("cuda"), nabla.paged_workspace(q, kc), torch.empty_like(q)

    def step():
        nabla.cache_append(k, v, kc, vc, table, starts, cu=cu, ws=ws)
        nabla.attn_paged(q, kc, vc, table, lens, o=o, ws=pws)
    g = capture(step)
    for s, c, n, want in (([0, 0], [0, 100, total], [100, total - 100], nabla.OK),
                          ([5, 900], [0, 1, 90], [6, 0], nabla.OK), ([0, 0], [0, 101, 100], [7, 9], nabla.ERR_PARAM),
                          ([3, 16 * width - 5], [0, 10, 30], [13, 16 * width], nabla.ERR_PARAM)):
        for t, x in ((starts, s), (cu, c), (lens, n)):
            t.copy_(dev(x))
        kc.zero_()
        vc.zero_()
        g.replay()
        g.replay()
        assert nabla.status(ws) == want and nabla.status(pws) == nabla.OK
        got = kc.clone(), vc.clone(), o.clone()
        kc.zero_()
        vc.zero_()
        step()
        for a, b in zip(got, (kc, vc, o)):
            assert torch.equal(a, b)
