"""The rotary, cache and packed calls together, as a model runs them: a prompt
and the tokens after it against attention over the whole sequence, and the video
path through the rotation into the block mask and the block-sparse attention.
Bounds are derived in seq_util.py."""
import math

import pytest
import torch

from adaptive_block_sparse_fractal_b200 import nabla

import seq_util

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rotate(x, pairs, pos, offset=0.0):
    """Adjacent-pair rotation of [N, heads, D] float64 by int positions [N, 3]."""
    ang = torch.cat([(pos[:, a].double() + offset)[:, None] * torch.tensor(
        [10000.0 ** (-i / n) for i in range(n)], dtype=torch.float64, device=x.device)
        for a, n in enumerate(pairs)], 1)[:, None]
    R = sum(pairs)
    y = x.clone()
    a, b = x[..., 0:2 * R:2], x[..., 1:2 * R:2]
    y[..., 0:2 * R:2] = a * ang.cos() - b * ang.sin()
    y[..., 1:2 * R:2] = b * ang.cos() + a * ang.sin()
    return y


@pytest.mark.parametrize("D,heads,heads_kv,page", [(64, 6, 2, 16), (128, 5, 1, 64), (128, 8, 4, 24)])
def test_prompt_then_tokens(D, heads, heads_kv, page):
    """Projection -> rope in place -> cache -> prompt attention, then tokens one by
    one (rope, append, attention over the pages, captured in a graph)."""
    lens, extra, pairs = [130, 1, 77, 200], 5, (8, 8, D // 2 - 16)
    n, cu = len(lens), [0]
    for L in lens:
        cu.append(cu[-1] + L)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(D + heads)
    width = heads + 2 * heads_kv
    qkv = torch.randn(cu[-1], width, D, generator=g, device="cuda").to(BF)
    raw = qkv.clone()
    pos = torch.cat([torch.arange(L) for L in lens]).to("cuda", torch.int32)[:, None].repeat(1, 3).contiguous()
    prm = nabla.rope_params_of(pairs)
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + heads_kv], qkv[:, heads + heads_kv:]
    nabla.rope(prm, q.transpose(0, 1), k.transpose(0, 1), pos=pos, q_out=q.transpose(0, 1),
               k_out=k.transpose(0, 1))
    for part, want in ((q, rotate(raw[:, :heads].double(), pairs, pos)),
                       (k, rotate(raw[:, heads:heads + heads_kv].double(), pairs, pos))):
        assert float(((part.double() - want).abs() - want.abs() * 2.0 ** -8 - 2.0 ** -16).max()) <= 0
    assert torch.equal(v, raw[:, heads + heads_kv:])
    # the prompt's rows into the pages, and its attention
    per = -(-(max(lens) + extra) // page)
    table = torch.randperm(n * per, generator=g, device="cuda").to(torch.int32).view(n, per).contiguous()
    kc = torch.full((n * per, page, heads_kv, D), math.nan, device="cuda").to(BF)
    vc = torch.full_like(kc, math.nan)
    nabla.cache_append(k, v, kc, vc, table, dev([0] * n), cu=dev(cu))
    ws = nabla.packed_workspace(q, k, n, back=True)
    o, lse = nabla.attn_packed_fwd(q, k, v, dev(cu), dev(cu), causal=True, ws=ws)
    assert nabla.status(ws) == nabla.OK
    r = seq_util.packed(q, k, v, cu, cu, True)
    seq_util.check(o, r["o"], r["o_tol"], "o")
    # tokens after it
    seen = [[k[a:b].clone(), v[a:b].clone()] for a, b in zip(cu, cu[1:])]
    used = dev(lens)
    new = torch.empty(n, width, D, dtype=BF, device="cuda")
    at = torch.empty(n, 3, dtype=torch.int32, device="cuda")
    nq, nk, nv = new[:, :heads], new[:, heads:heads + heads_kv], new[:, heads + heads_kv:]
    pws, out = nabla.paged_workspace(nq, kc), torch.empty(n, heads, D, dtype=BF, device="cuda")

    def step():
        at.copy_(used[:, None].expand(n, 3))
        nabla.rope(prm, nq.transpose(0, 1), nk.transpose(0, 1), pos=at, q_out=nq.transpose(0, 1),
                   k_out=nk.transpose(0, 1))
        nabla.cache_append(nk, nv, kc, vc, table, used)
        used.add_(1)
        nabla.attn_paged(nq, kc, vc, table, used, o=out, ws=pws)
    graph = None
    for t in range(extra):
        new.copy_(torch.randn(n, width, D, generator=g, device="cuda").to(BF))
        if t == 1:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        if graph is None:
            step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert nabla.status(pws) == nabla.OK
        for s in range(n):
            for i, x in enumerate((nk, nv)):
                seen[s][i] = torch.cat([seen[s][i], x[s:s + 1]])
            keys = seen[s][0].shape[0]
            keep = torch.ones(1, keys, dtype=torch.bool, device="cuda")
            for h in range(heads):
                c = h // (heads // heads_kv)
                x = seq_util.attention(nq[s, h:h + 1].double(), seen[s][0][:, c].double(),
                                       seen[s][1][:, c].double(), D ** -0.5, keep)
                seq_util.check(out[s, h:h + 1], x["o"], x["o_tol"], "o")
    assert used.tolist() == [L + extra for L in lens]
    # the same rows by prompt attention of the last token against everything cached
    kk, vv = torch.cat([x[0] for x in seen]), torch.cat([x[1] for x in seen])
    ck = [0]
    for x in seen:
        ck.append(ck[-1] + x[0].shape[0])
    last, _ = nabla.attn_packed_fwd(nq, kk, vv, dev(range(n + 1)), dev(ck), causal=True)
    r = seq_util.packed(nq, kk, vv, list(range(n + 1)), ck, True)
    seq_util.check(last, r["o"], r["o_tol"], "o")
    seq_util.check(out, r["o"], r["o_tol"], "o")


@pytest.mark.parametrize("D", [64, 128])
def test_video_path(D):
    """Rotation fused with the flattening -> mask -> block-sparse attention and its
    gradients -> rotation back to grid order.  With every block kept the
    attention is dense: the packed calls compute the same."""
    T, H, W, heads = 3, 16, 24, 2
    N, pairs = T * H * W, (8, 8, D // 2 - 16)
    g = torch.Generator(device="cuda").manual_seed(D)
    q, k, v, dout = (torch.randn(heads, N, D, generator=g, device="cuda").to(BF) for _ in range(4))
    fwd, back = nabla.rope_params_of(pairs), nabla.rope_params_of(pairs, inverse=True)
    qf, kf = nabla.rope(fwd, q, k, grid=(T, H, W), flat_out=True)
    q2, k2 = nabla.rope(fwd, q, k, grid=(T, H, W))
    assert torch.equal(qf, nabla.flatten(q2, T, H, W)) and torch.equal(kf, nabla.flatten(k2, T, H, W))
    vf = nabla.flatten(v, T, H, W)
    shape = nabla.shape_of(1, heads, T, H, W, D)
    prm = nabla.params_of(0.8, (3, 3, 3), D=D, flags=nabla.EMIT_COLS)
    a = nabla.build_mask(shape, prm, qf, kf)
    _, _, b = nabla.build_mask_grid(shape, prm, q2, k2)
    assert torch.equal(a["bits"], b["bits"])
    dense = nabla.params_of(1.0, (3, 3, 3), D=D, flags=nabla.EMIT_COLS)
    m = nabla.build_mask(shape, dense, qf, kf)
    o, lse = nabla.attn_fwd(shape, dense, qf, kf, vf, m)
    dq, dk, dv = nabla.attn_bwd(shape, dense, qf, kf, vf, o, dout, lse, m)
    rows = lambda t: t.transpose(0, 1)
    cu = torch.tensor([0, N], dtype=torch.int32, device="cuda")
    po, pl = nabla.attn_packed_fwd(rows(qf), rows(kf), rows(vf), cu, cu)
    pq, pk, pv = nabla.attn_packed_bwd(rows(qf), rows(kf), rows(vf), po, rows(dout), pl, cu, cu)
    r = seq_util.packed(rows(qf), rows(kf), rows(vf), [0, N], [0, N], False, dout=rows(dout))
    for n, one, other in (("o", o, po), ("dq", dq, pq), ("dk", dk, pk), ("dv", dv, pv)):
        seq_util.check(rows(one), r[n], r[n + "_tol"], n)
        seq_util.check(other, r[n], r[n + "_tol"], n)
    gq, gk = nabla.rope(back, dq, dk, grid=(T, H, W), flat_in=True)
    wq = nabla.rope(back, nabla.flatten(dq, T, H, W, inverse=True), grid=(T, H, W))
    assert torch.equal(gq, wq) and gk.shape == k.shape


def test_two_streams_with_their_own_workspaces():
    """The same calls on two streams at once give the bits that they give alone."""
    lens = [300, 5, 1000, 64]
    cu = [0]
    for L in lens:
        cu.append(cu[-1] + L)
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    new = lambda h: torch.randn(cu[-1], h, 128, generator=g, device="cuda").to(BF)
    sets = [(new(6), new(2), new(2), new(6)) for _ in range(2)]

    def run(q, k, v, dout, ws):
        o, lse = nabla.attn_packed_fwd(q, k, v, cud, cud, causal=True, ws=ws)
        return (o,) + nabla.attn_packed_bwd(q, k, v, o, dout, lse, cud, cud, causal=True, ws=ws)
    spaces = [nabla.packed_workspace(x[0], x[1], len(lens), back=True) for x in sets]
    want = [run(*x, ws) for x, ws in zip(sets, spaces)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = run(*sets[i], spaces[i])
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


# ---------------------------------------------------------------------------
# offsets beyond 2^31 elements
# ---------------------------------------------------------------------------
FAR = 2 ** 31


def test_far_rows_of_packed_tensors():
    """Sequences whose rows lie behind the first 2^31 elements of every tensor."""
    heads, D = 40, 128
    total = FAR // (heads * D) + 700
    cu = [total - 650, total - 350, total - 349, total - 5]
    g = torch.Generator(device="cuda").manual_seed(3)

    def make():
        t = torch.empty(total, heads, D, dtype=BF, device="cuda")
        t[total - 700:] = torch.randn(700, heads, D, generator=g, device="cuda").to(BF)
        return t
    q, k, v, dout = make(), make(), make(), make()
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    ws = nabla.packed_workspace(q, k, 3, back=True)
    o, lse = nabla.attn_packed_fwd(q, k, v, cud, cud, causal=True, ws=ws)
    assert nabla.status(ws) == nabla.OK
    dq, dk, dv = nabla.attn_packed_bwd(q, k, v, o, dout, lse, cud, cud, causal=True, ws=ws)
    assert nabla.status(ws) == nabla.OK
    a = total - 700
    near = [c - a for c in cu]
    pick = lambda t: t[a:, 17:18].contiguous()
    r = seq_util.packed(pick(q), pick(k), pick(v), near, near, True, dout=pick(dout))
    for n, t in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
        seq_util.check(pick(t), r[n], r[n + "_tol"], n)
    seq_util.check_lse(lse[17:18, a:], r["lse"])


def test_far_pages_and_far_rope_rows():
    page, heads_kv, D = 64, 4, 128
    pages = FAR // (page * heads_kv * D) + 20
    kc = torch.empty(pages, page, heads_kv, D, dtype=BF, device="cuda")
    vc = torch.empty_like(kc)
    table = torch.tensor([[pages - 1, pages - 3, 0], [pages - 2, pages - 7, pages - 5]], dtype=torch.int32,
                         device="cuda")
    lens = [130, 190]
    cu = torch.tensor([0, 130, 320], dtype=torch.int32, device="cuda")
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    k, v = (torch.randn(320, heads_kv, D, device="cuda").to(BF) for _ in range(2))
    nabla.cache_append(k, v, kc, vc, table, zero, cu=cu)
    q = torch.randn(2, 8, D, device="cuda").to(BF)
    o, _ = nabla.attn_paged(q, kc, vc, table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    for s, (a, b) in enumerate(((0, 130), (130, 320))):
        for h in range(8):
            x = seq_util.attention(q[s, h:h + 1].double(), k[a:b, h // 2].double(), v[a:b, h // 2].double(),
                                   D ** -0.5, torch.ones(1, b - a, dtype=torch.bool, device="cuda"))
            seq_util.check(o[s, h:h + 1], x["o"], x["o_tol"], "o")
    del kc, vc
    # rotation in place of rows behind 2^31 elements, tokens first
    heads = 20
    total = FAR // (heads * D) + 300
    x = torch.empty(total, heads, D, dtype=BF, device="cuda")
    tail = torch.randn(300, heads, D, device="cuda").to(BF)
    x[total - 300:] = tail
    prm = nabla.rope_params_of((64,))
    pos = torch.arange(total, dtype=torch.int32, device="cuda")[:, None].contiguous()
    y = x.transpose(0, 1)
    nabla.rope(prm, y, pos=pos, q_out=y)
    want = nabla.rope(prm, tail.transpose(0, 1), pos=pos[total - 300:].contiguous())
    assert torch.equal(x[total - 300:].transpose(0, 1), want)
