"""The paged cache: appending rows and the attention of one new token
(bounds derived in seq_util.py)."""
import math

import pytest
import torch

from adaptive_block_sparse_fractal_b200 import nabla

import seq_util

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def make_cache(lens, page, heads_kv, D, seed=0, extra_cols=2, spare=3, heads_first=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g, device="cuda").tolist()
    width = max(need + [1]) + extra_cols
    table = torch.full((len(lens), width), -7, dtype=torch.int32)  # never looked at behind a length
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    if heads_first:
        shape = (pages, heads_kv, page, D)
        new = lambda: torch.randn(shape, generator=g, device="cuda").to(BF).transpose(1, 2)
    else:
        shape = (pages, page, heads_kv, D)
        new = lambda: torch.randn(shape, generator=g, device="cuda").to(BF)
    return new(), new(), table.cuda()


def rows_of(cache, table, s, n):
    page = cache.shape[1]
    p = torch.arange(n, device="cuda")
    return cache[table[s, p // page].long(), p % page]


def reference(q, kc, vc, table, lens):
    n, hq, D = q.shape
    G = hq // kc.shape[2]
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(o)
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device="cuda")
    for s, L in enumerate(lens):
        if L == 0:
            continue
        k, v = rows_of(kc, table, s, L).double(), rows_of(vc, table, s, L).double()
        keep = torch.ones(1, L, dtype=torch.bool, device="cuda")
        for h in range(hq):
            x = seq_util.attention(q[s, h:h + 1].double(), k[:, h // G], v[:, h // G], D ** -0.5, keep)
            o[s, h], tol[s, h], lse[s, h] = x["o"][0], x["o_tol"][0], x["lse"][0]
    return o, tol, lse


def run_paged(q, kc, vc, table, lens, want_status=nabla.OK, **kw):
    ws = nabla.paged_workspace(q, kc)
    ws.fill_(255)  # nothing of it needs a start value
    dev = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = nabla.attn_paged(q, kc, vc, table, dev, ws=ws, **kw)
    assert nabla.status(ws) == want_status
    return o, lse


@pytest.mark.parametrize("lens", [[1], [0], [16], [17], [63, 64, 65], [1000], [0, 5, 0, 0, 300, 1, 0],
                                  [7, 2000, 1, 129, 64]])
@pytest.mark.parametrize("heads,heads_kv", [(1, 1), (6, 2), (5, 1), (16, 1), (8, 8), (34, 2)])
@pytest.mark.parametrize("D", [64, 128])
def test_paged(lens, heads, heads_kv, D):
    for page in (1, 16, 24, 64):
        kc, vc, table = make_cache(lens, page, heads_kv, D, seed=page, heads_first=page == 64)
        q = torch.randn(len(lens), heads, D, device="cuda").to(BF)
        o, lse = run_paged(q, kc, vc, table, lens)
        ro, tol, rl = reference(q, kc, vc, table, lens)
        seq_util.check(o, ro, tol, "o")
        seq_util.check_lse(lse, rl)


def test_paged_long_and_many():
    for lens, heads, heads_kv, page in (([70000, 3], 12, 4, 128), ([(i * 131) % 700 for i in range(300)], 4, 2, 32)):
        kc, vc, table = make_cache(lens, page, heads_kv, 64, seed=1)
        q = torch.randn(len(lens), heads, 64, device="cuda").to(BF)
        o, lse = run_paged(q, kc, vc, table, lens)
        ro, tol, rl = reference(q, kc, vc, table, lens)
        seq_util.check(o, ro, tol, "o")
        seq_util.check_lse(lse, rl)


def test_paged_rising_scores():
    L = 900
    kc, vc, table = make_cache([L], 16, 1, 128, seed=2)
    ramp = torch.linspace(0.01, 4, L, device="cuda")
    page = kc.shape[1]
    p = torch.arange(L, device="cuda")
    kc[table[0, p // page].long(), p % page] *= ramp[:, None, None].to(BF)
    q = torch.randn(1, 3, 128, device="cuda").to(BF)
    o, lse = run_paged(q, kc, vc, table, [L])
    ro, tol, rl = reference(q, kc, vc, table, [L])
    seq_util.check(o, ro, tol, "o")
    seq_util.check_lse(lse, rl)


def test_rows_behind_a_length_do_not_leak():
    lens = [37, 64, 1]
    kc, vc, table = make_cache(lens, 16, 2, 128, seed=3)
    clean = [(rows_of(kc, table, s, n).clone(), rows_of(vc, table, s, n).clone()) for s, n in enumerate(lens)]
    q = torch.randn(3, 4, 128, device="cuda").to(BF)
    want, _ = run_paged(q, kc, vc, table, lens)
    kc.fill_(math.nan)
    vc.fill_(math.inf)
    for s, n in enumerate(lens):
        p = torch.arange(n, device="cuda")
        at = table[s, p // 16].long(), p % 16
        kc[at], vc[at] = clean[s]
    got, _ = run_paged(q, kc, vc, table, lens)
    assert torch.equal(got, want)


def test_bad_pages_and_lengths_are_masked_and_reported():
    lens = [100, 40]
    kc, vc, table = make_cache(lens, 16, 1, 64, seed=4)
    q = torch.randn(2, 2, 64, device="cuda").to(BF)
    good, _ = run_paged(q, kc, vc, table, lens)
    for bad in (-1, kc.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[0, 2] = bad  # rows 32..47 of sequence 0 count as masked
        o, _ = run_paged(q, kc, vc, t, lens, nabla.ERR_PARAM)
        keep = torch.ones(1, 100, dtype=torch.bool, device="cuda")
        keep[:, 32:48] = False
        k, v = rows_of(kc, table, 0, 100).double(), rows_of(vc, table, 0, 100).double()
        for h in range(2):
            x = seq_util.attention(q[0, h:h + 1].double(), k[:, 0], v[:, 0], 0.125, keep)
            seq_util.check(o[0, h:h + 1], x["o"], x["o_tol"], "o")
        assert torch.equal(o[1], good[1])
    o, lse = run_paged(q, kc, vc, table, [-3, 40], nabla.ERR_PARAM)
    assert bool((o[0] == 0).all()) and torch.equal(o[1], good[1]) and bool((lse[0] == -math.inf).all())
    o, _ = run_paged(q, kc, vc, table, [16 * table.shape[1] + 1, 40], nabla.ERR_PARAM)
    assert bool((o[0] == 0).all()) and torch.equal(o[1], good[1])


def append_reference(kc, vc, k, v, table, starts, cu):
    kc, vc = kc.clone(), vc.clone()
    page = kc.shape[1]
    for s, (a, b) in enumerate(zip(cu, cu[1:])):
        p = starts[s] + torch.arange(b - a, device="cuda")
        at = table[s, p // page].long(), p % page
        kc[at], vc[at] = k[a:b], v[a:b]
    return kc, vc


@pytest.mark.parametrize("heads_kv,D,page", [(1, 64, 16), (2, 128, 24), (8, 128, 64), (3, 8, 1), (1, 72, 128)])
@pytest.mark.parametrize("starts,lens", [([0], [1]), ([5, 0, 15], [1, 1, 1]), ([3, 0, 130, 7], [40, 0, 300, 1]),
                                         ([0] * 40, [(i * 7) % 90 for i in range(40)]), ([17], [6000])])
def test_append(heads_kv, D, page, starts, lens):
    total = [a + n for a, n in zip(starts, lens)]
    for heads_first in (False, True):
        kc, vc, table = make_cache(total, page, heads_kv, D, seed=6, heads_first=heads_first)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        kv = torch.randn(cu[-1] + 4, 2 * heads_kv, D, device="cuda").to(BF)  # 4 rows of no sequence
        k, v = kv[:, :heads_kv], kv[:, heads_kv:]
        wk, wv = append_reference(kc, vc, k, v, table, starts, cu)
        dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        ws = nabla.cache_workspace("cuda")
        nabla.cache_append(k, v, kc, vc, table, dev(starts), cu=dev(cu), ws=ws)
        assert nabla.status(ws) == nabla.OK
        assert torch.equal(kc, wk) and torch.equal(vc, wv)


def test_append_one_row_each_and_bad_places():
    starts = [0, 31, 16, 40]
    kc, vc, table = make_cache([n + 1 for n in starts], 16, 2, 64, seed=7, extra_cols=0)
    k, v = (torch.randn(4, 2, 64, device="cuda").to(BF) for _ in range(2))
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    wk, wv = append_reference(kc, vc, k, v, table, starts, [0, 1, 2, 3, 4])
    ck, cv = kc.clone(), vc.clone()
    nabla.cache_append(k, v, ck, cv, table, dev(starts))
    assert torch.equal(ck, wk) and torch.equal(cv, wv)
    ws = nabla.cache_workspace("cuda")
    for s, col, value in ((1, 1, kc.shape[0]), (2, 1, -1)):
        t = table.clone()
        t[s, col] = value
        ck, cv = kc.clone(), vc.clone()
        nabla.cache_append(k, v, ck, cv, t, dev(starts), ws=ws)
        assert nabla.status(ws) == nabla.ERR_PARAM
        page, off = int(table[s, col]), starts[s] % 16
        wk2, wv2 = wk.clone(), wv.clone()  # that row alone is missing
        wk2[page, off], wv2[page, off] = kc[page, off], vc[page, off]
        assert torch.equal(ck, wk2) and torch.equal(cv, wv2)
    ck, cv = kc.clone(), vc.clone()
    nabla.cache_append(k, v, ck, cv, table, dev([0, 31, -1, 16 * table.shape[1]]), ws=ws)
    assert nabla.status(ws) == nabla.ERR_PARAM
    nabla.cache_append(k, v, ck, cv, table, dev(starts), ws=ws)
    assert nabla.status(ws) == nabla.OK and torch.equal(ck, wk)


def test_paged_graph_follows_growing_lengths():
    """A captured decoding step: the lengths live on the device and grow."""
    kc, vc, table = make_cache([400, 300], 16, 2, 128, seed=8)
    q = torch.randn(2, 6, 128, device="cuda").to(BF)
    k, v = (torch.randn(2, 2, 128, device="cuda").to(BF) for _ in range(2))
    lens = torch.tensor([350, 0], dtype=torch.int32, device="cuda")
    ws = nabla.paged_workspace(q, kc)
    o = torch.empty_like(q)

    def step():
        nabla.cache_append(k, v, kc, vc, table, lens)
        lens.add_(1)
        nabla.attn_paged(q, kc, vc, table, lens, o=o, ws=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for n in range(20):
        g.replay()
    torch.cuda.synchronize()
    assert lens.tolist() == [371, 21] and nabla.status(ws) == nabla.OK
    ro, tol, _ = reference(q, kc, vc, table, [371, 21])
    seq_util.check(o, ro, tol, "o")
    assert torch.equal(rows_of(kc, table, 1, 21), k[1].expand(21, 2, 128))
