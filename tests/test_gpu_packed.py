"""Packed-sequence attention against float64 (bounds derived in seq_util.py)."""
import math

import pytest
import torch

from adaptive_block_sparse_fractal_b200 import nabla

import seq_util

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def borders(lens, first=0):
    out = [first]
    for n in lens:
        out.append(out[-1] + n)
    return out


def make(lens_q, lens_k, heads, heads_kv, D, seed=0, behind=0, std=1.0):
    """Packed inputs with `behind` NaN rows behind the last sequence."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    cq, ck = borders(lens_q), borders(lens_k)

    def t(n, h):
        x = (torch.randn(n + behind, h, D, generator=g, device="cuda") * std).to(BF)
        x[n:] = math.nan
        return x
    q, k, v, dout = t(cq[-1], heads), t(ck[-1], heads_kv), t(ck[-1], heads_kv), t(cq[-1], heads)
    dev = lambda c: torch.tensor(c, dtype=torch.int32, device="cuda")
    return q, k, v, dout, cq, ck, dev(cq), dev(ck)


def run_fwd(q, k, v, cu_q, cu_k, causal, **kw):
    ws = nabla.packed_workspace(q, k, cu_q.numel() - 1)
    o = torch.full(q.shape, 7.0, dtype=BF, device="cuda")
    lse = torch.full((q.shape[1], q.shape[0]), 7.0, device="cuda")
    nabla.attn_packed_fwd(q, k, v, cu_q, cu_k, causal=causal, o=o, lse=lse, ws=ws, **kw)
    assert nabla.status(ws) == nabla.OK
    return o, lse


CASES = [
    # lens_q, lens_k, heads, heads_kv
    ([1], [1], 1, 1),
    ([1, 1, 1], [1, 2, 129], 2, 1),
    ([128], [128], 1, 1),
    ([129, 127], [127, 130], 2, 2),
    ([257, 0, 3], [257, 5, 0], 3, 1),
    ([77, 1, 200, 33], [77, 1, 200, 33], 6, 2),
    ([600, 511], [600, 1000], 5, 1),
    ([5, 300], [1500, 40], 4, 4),   # row tiles against many and few keys
    ([100], [30], 8, 2),            # causal: 70 rows keep nothing
    ([64, 64, 64, 64, 64], [0, 64, 1, 128, 63], 7, 1),
    ([1000], [1000], 10, 2),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D", [128, 64])
def test_forward(case, causal, D):
    lens_q, lens_k, hq, hk = CASES[case]
    q, k, v, _, cq, ck, dq_, dk_ = make(lens_q, lens_k, hq, hk, D, seed=case, behind=70)
    o, lse = run_fwd(q, k, v, dq_, dk_, causal)
    r = seq_util.packed(q, k, v, cq, ck, causal)
    n = cq[-1]
    assert bool((o[n:] == 7).all()) and bool((lse[:, n:] == 7).all())  # rows of no sequence
    seq_util.check(o[:n], r["o"][:n], r["o_tol"][:n], "o")
    seq_util.check_lse(lse[:, :n], r["lse"][:, :n])


@pytest.mark.parametrize("D", [128, 64])
def test_forward_split_over_keys(D):
    """Few rows, many keys: the key range is split and joined."""
    for lens_q, lens_k, hq, hk, causal in (([1], [9000], 2, 1, True), ([3, 1], [4100, 6001], 4, 2, True),
                                           ([40], [8192], 6, 2, False), ([2, 0, 5], [5000, 4000, 0], 2, 2, True)):
        q, k, v, _, cq, ck, dq_, dk_ = make(lens_q, lens_k, hq, hk, D, seed=5, behind=3)
        o, lse = run_fwd(q, k, v, dq_, dk_, causal)
        r = seq_util.packed(q, k, v, cq, ck, causal)
        n = cq[-1]
        assert bool((o[n:] == 7).all()) and bool((lse[:, n:] == 7).all())
        seq_util.check(o[:n], r["o"][:n], r["o_tol"][:n], "o")
        seq_util.check_lse(lse[:, :n], r["lse"][:, :n])


def test_forward_rising_scores_and_scale():
    """Maxima that grow by far more than the rescaling headroom along the keys."""
    L, D = 700, 128
    q, k, v, _, cq, ck, cu, _ = make([L], [L], 2, 2, D, seed=3)
    k *= torch.linspace(0.01, 6, L, device="cuda")[:, None, None]
    k = k.to(BF)
    for causal in (False, True):
        o, lse = run_fwd(q, k, v, cu, cu, causal, scale=0.25)
        r = seq_util.packed(q, k, v, cq, ck, causal, scale=0.25)
        # scores reach a few hundred here: their float32 error enters the exponent
        x = float(r["lse"].abs().max())
        seq_util.check(o, r["o"], r["o_tol"] + x * 2.0 ** -20 * r["o_tol"] / seq_util.H, "o")
        seq_util.check(lse, r["lse"], 2.0 ** -20 * (1 + r["lse"].abs()) + 2.0 ** -18, "lse")


def test_neighbouring_sequences_do_not_leak():
    """NaN and infinities in the sequences around one, in the padding behind the
    last and in the gap in front of the first leave its rows alone."""
    D, hq, hk = 128, 4, 2
    q, k, v, _, _, _, _, _ = make([400], [400], hq, hk, D, seed=9)
    cu = torch.tensor([10, 100, 230, 390], dtype=torch.int32, device="cuda")
    for t in (q, k, v):
        t[:10], t[390:] = math.nan, math.nan
        t[10:100], t[230:390] = math.inf, math.nan
    for causal in (False, True):
        o, lse = run_fwd(q, k, v, cu, cu, causal)
        r = seq_util.packed(q, k, v, [100, 230], [100, 230], causal)
        seq_util.check(o, r["o"], r["o_tol"], "o")
        seq_util.check_lse(lse, r["lse"])
        assert bool((o[:10] == 7).all()) and bool((o[390:] == 7).all())


def test_strides_and_layouts():
    """Slices of one fused projection, heads in front, padded rows."""
    L, hq, hk, D = 150, 4, 2, 64
    qkv = torch.randn(L, hq + 2 * hk, D, device="cuda").to(BF)
    cu = torch.tensor([0, 70, L], dtype=torch.int32, device="cuda")
    a, b, c = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    o, lse = run_fwd(a, b, c, cu, cu, True)
    r = seq_util.packed(a, b, c, [0, 70, L], [0, 70, L], True)
    seq_util.check(o, r["o"], r["o_tol"], "o")
    first = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.randn(L, hk, D + 8, device="cuda").to(BF)
    wide[:, :, :D] = b
    out = torch.full((hq, L + 5, D), 7.0, device="cuda").to(BF)
    view = out[:, :L].transpose(0, 1)
    got, lse2 = nabla.attn_packed_fwd(first(a), wide[:, :, :D], first(c), cu, cu, causal=True, o=view)
    assert torch.equal(got, o) and torch.equal(lse2, lse)
    assert bool((out[:, L:] == 7).all())


@pytest.mark.parametrize("cq,ck", [([0, 50, 40], [0, 10, 20]), ([0, 10, 101], [0, 10, 20]),
                                   ([-1, 10, 20], [0, 10, 20]), ([0, 10, 20], [0, 30, 101])])
def test_bad_borders_are_reported_and_nothing_is_written(cq, ck):
    q, k, v, dout, _, _, _, _ = make([100], [100], 2, 1, 64)
    dev = lambda c: torch.tensor(c, dtype=torch.int32, device="cuda")
    ws = nabla.packed_workspace(q, k, 2)
    o = torch.full(q.shape, 7.0, dtype=BF, device="cuda")
    nabla.attn_packed_fwd(q, k, v, dev(cq), dev(ck), o=o, ws=ws)
    assert nabla.status(ws) == nabla.ERR_PARAM
    assert bool((o == 7).all())
    nabla.attn_packed_fwd(q, k, v, dev([0, 50, 100]), dev([0, 50, 100]), o=o, ws=ws)
    assert nabla.status(ws) == nabla.OK and not bool((o == 7).all())


def test_stream_graph_and_many_sequences():
    lens = [(i * 37) % 50 for i in range(1000)]
    q, k, v, _, cq, ck, cu, _ = make(lens, lens, 2, 1, 64, seed=4)
    want, _ = run_fwd(q, k, v, cu, cu, True)
    some = 100
    r = seq_util.packed(q, k, v, cq[:some], ck[:some], True)
    seq_util.check(want, r["o"], r["o_tol"], "o")
    ws = nabla.packed_workspace(q, k, 1000)
    o = torch.zeros_like(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        nabla.attn_packed_fwd(q, k, v, cu, cu, causal=True, o=o, ws=ws)
    s.synchronize()
    assert torch.equal(o, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nabla.attn_packed_fwd(q, k, v, cu, cu, causal=True, o=o, ws=ws)
    o.zero_()
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and nabla.status(ws) == nabla.OK


# ---------------------------------------------------------------------------
# backward
# ---------------------------------------------------------------------------
def run_both(q, k, v, dout, cu_q, cu_k, causal, **kw):
    ws = nabla.packed_workspace(q, k, cu_q.numel() - 1, back=True)
    o, lse = nabla.attn_packed_fwd(q, k, v, cu_q, cu_k, causal=causal, ws=ws, **kw)
    assert nabla.status(ws) == nabla.OK
    full = lambda t: torch.full(t.shape, 7.0, dtype=BF, device="cuda")
    dq, dk, dv = full(q), full(k), full(v)
    nabla.attn_packed_bwd(q, k, v, o, dout, lse, cu_q, cu_k, causal=causal, dq=dq, dk=dk, dv=dv, ws=ws,
                          **kw)
    assert nabla.status(ws) == nabla.OK
    return dq, dk, dv


def check_grads(got, r, n, m):
    for name, g, rows in zip(("dq", "dk", "dv"), got, (n, m, m)):
        assert bool((g[rows:] == 7).all()), name  # rows of no sequence
        seq_util.check(g[:rows], r[name][:rows], r[name + "_tol"][:rows], name)


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D", [128, 64])
def test_backward(case, causal, D):
    lens_q, lens_k, hq, hk = CASES[case]
    q, k, v, dout, cq, ck, cu_q, cu_k = make(lens_q, lens_k, hq, hk, D, seed=case, behind=70)
    got = run_both(q, k, v, dout, cu_q, cu_k, causal)
    r = seq_util.packed(q, k, v, cq, ck, causal, dout=dout)
    check_grads(got, r, cq[-1], ck[-1])


def test_backward_neighbours_strides_and_repeatability():
    """NaN in the sequences around one; slices of a fused projection, gradients
    into slices of another; the same bits every time."""
    L, hq, hk, D = 400, 6, 2, 128
    g = torch.Generator(device="cuda").manual_seed(2)
    qkv = torch.randn(L, hq + 2 * hk, D, generator=g, device="cuda").to(BF)
    dout = torch.randn(L, hq, D, generator=g, device="cuda").to(BF)
    for t in (qkv, dout):
        t[:10], t[10:100], t[230:] = math.nan, math.inf, math.nan
    cu = torch.tensor([10, 100, 230, 390], dtype=torch.int32, device="cuda")
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    for causal in (False, True):
        ws = nabla.packed_workspace(q, k, 3, back=True)
        o, lse = nabla.attn_packed_fwd(q, k, v, cu, cu, causal=causal, ws=ws)
        out = []
        for _ in range(2):
            d = torch.full(qkv.shape, 7.0, dtype=BF, device="cuda")
            dq, dk, dv = d[:, :hq], d[:, hq:hq + hk], d[:, hq + hk:]
            nabla.attn_packed_bwd(q, k, v, o, dout, lse, cu, cu, causal=causal, dq=dq, dk=dk, dv=dv, ws=ws)
            out.append(d)
        r = seq_util.packed(q, k, v, [100, 230], [100, 230], causal, dout=dout)
        for n, t in (("dq", dq), ("dk", dk), ("dv", dv)):
            seq_util.check(t[100:230], r[n][100:230], r[n + "_tol"][100:230], n)
        assert torch.equal(out[0][100:230], out[1][100:230])
        assert bool((d[:10] == 7).all()) and bool((d[390:] == 7).all())


def test_gradients_against_differences():
    """Central differences of the float64 loss sum(o dout) along single
    coordinates: error of the differences ~ eps^2 |f'''| + 2^-52 |f| / eps."""
    lens_q, lens_k, hq, hk, D = [70, 33], [70, 50], 4, 2, 64
    q, k, v, dout, cq, ck, cu_q, cu_k = make(lens_q, lens_k, hq, hk, D, seed=11)
    got = run_both(q, k, v, dout, cu_q, cu_k, True)
    r = seq_util.packed(q, k, v, cq, ck, True, dout=dout)
    base = {"q": q.double(), "k": k.double(), "v": v.double()}

    def loss(p):
        return float((seq_util.packed(p["q"], p["k"], p["v"], cq, ck, True)["o"] * dout.double()).sum())
    eps = 1e-4
    for i, name in enumerate(("q", "k", "v")):
        for at in ((0, 0, 0), (69, 1, 63), (75, 1, 17), (30, 0, 40)):
            p = {n: t.clone() for n, t in base.items()}
            p[name][at] += eps
            up = loss(p)
            p[name][at] -= 2 * eps
            diff = (up - loss(p)) / (2 * eps)
            tol = float(r["d" + name + "_tol"][at]) + 1e-5
            assert abs(float(got[i][at]) - diff) <= tol, (name, at)


def test_backward_in_a_graph_and_zero_rows():
    q, k, v, dout, cq, ck, cu_q, cu_k = make([100, 40], [100, 40], 4, 2, 128, seed=1)
    want = run_both(q, k, v, dout, cu_q, cu_k, True)
    ws = nabla.packed_workspace(q, k, 2, back=True)
    o, lse = torch.empty_like(q), torch.empty(4, 140, device="cuda")
    grads = [torch.empty_like(t) for t in (q, k, v)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nabla.attn_packed_fwd(q, k, v, cu_q, cu_k, causal=True, o=o, lse=lse, ws=ws)
        nabla.attn_packed_bwd(q, k, v, o, dout, lse, cu_q, cu_k, causal=True, dq=grads[0], dk=grads[1],
                              dv=grads[2], ws=ws)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(grads, want))
    # no query at all: dk = dv = 0; no key at all: o = 0, dq = 0
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    e = q[:0]
    o0, lse0 = nabla.attn_packed_fwd(e, k, v, none, cu_k)
    _, dk, dv = nabla.attn_packed_bwd(e, k, v, o0, e, lse0, none, cu_k)
    assert bool((dk == 0).all()) and bool((dv == 0).all())
    o1, lse1 = nabla.attn_packed_fwd(q, k[:0], v[:0], cu_q, none)
    assert bool((o1 == 0).all()) and bool((lse1 == -math.inf).all())
    dq, _, _ = nabla.attn_packed_bwd(q, k[:0], v[:0], o1, dout, lse1, cu_q, none)
    assert bool((dq == 0).all())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("step", [20.0, 80.0, 2000.0])
def test_forward_scores_that_jump_far_above_the_first_tile(D, step):
    """Some rows meet a key whose score lies `step` above all earlier ones, tiles
    after the reference was set; others never do; lengths end inside tiles."""
    lens = [900, 300, 140]
    q, k, v, _, cq, ck, cu, _ = make(lens, lens, 4, 2, D, seed=13, std=0.5)
    for a, b in zip(cq, cq[1:]):
        n = b - a
        for at in (n // 2, n - 3):
            k[a + at, 0] = q[a + n - 1, 1] * (step / float(q[a + n - 1, 1].double().pow(2).sum() * D ** -0.5))
    for causal in (False, True):
        o, lse = run_fwd(q, k, v, cu, cu, causal)
        r = seq_util.packed(q, k, v, cq, ck, causal)
        # a score of s has a float32 error of up to D 2^-24 |s|, which enters P
        e = D * 2.0 ** -24 * (step + 20)
        seq_util.check(o, r["o"], r["o_tol"] * (1 + 4 * e / seq_util.H) + 4 * e * float(v.abs().max()), "o")
        seq_util.check(lse, r["lse"], 2.0 ** -20 * (1 + r["lse"].abs()) + 2.0 ** -18 + e, "lse")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens_q,lens_k,causal", [([2] * 40, [2] * 40, True), ([3, 2, 1, 4] * 8, [3, 2, 1, 4] * 8, True),
                                                  ([70, 9], [2, 3], False), ([20, 31], [20, 31], True),
                                                  ([200, 64], [32, 17], False), ([60, 64, 1], [60, 64, 1], True),
                                                  ([130, 3], [64, 33], False), ([90], [20], True)])
def test_gradients_with_few_keys(lens_q, lens_k, causal, D):
    """Few keys: dP - delta cancels, so delta must not carry the rounding of o.
    The bound without that term: dS is rounded to bf16 once (h |dS|), and P (dP -
    delta) has float32 errors e against its terms (E = 2^-14 covers the scores'
    error, 2^-17 of P in delta and the sums)."""
    q, k, v, dout, cq, ck, cu_q, cu_k = make(lens_q, lens_k, 4, 2, D, seed=21)
    got = run_both(q, k, v, dout, cu_q, cu_k, causal)
    sc, h = D ** -0.5, seq_util.H
    for s in range(len(lens_q)):
        a, b, c, e = cq[s], cq[s + 1], ck[s], ck[s + 1]
        dk, dk_tol = 0, 0
        for hd in range(4):
            Q, K, V, G = q[a:b, hd].double(), k[c:e, hd // 2].double(), v[c:e, hd // 2].double(), dout[a:b, hd].double()
            keep = seq_util.keep_mask(b - a, e - c, causal, "cuda")
            x = seq_util.attention(Q, K, V, sc, keep, G)
            p = ((Q @ K.T) * sc).masked_fill(~keep, -math.inf)
            p = torch.where(keep, torch.softmax(p, 1), torch.zeros_like(p))  # (a row that keeps nothing has p = 0)
            dp = G @ V.T
            ds = p * (dp - (G * x["o"]).sum(1, keepdim=True))
            dds = h * ds.abs() + seq_util.E * p * (G.abs() @ V.abs().T + (G * x["o"]).abs().sum(1, keepdim=True))
            seq_util.check(got[0][a:b, hd], x["dq"], (dds @ K.abs()) * sc + h * x["dq"].abs(), "dq")
            dk, dk_tol = dk + x["dk"], dk_tol + (dds.T @ Q.abs()) * sc
            if hd % 2:
                seq_util.check(got[1][c:e, hd // 2], dk, dk_tol + h * dk.abs(), "dk")
                dk, dk_tol = 0, 0
