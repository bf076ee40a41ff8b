"""Packed attention where single keys stand out: scores far above all earlier
ones, NaN and infinities in keys that a row keeps.  Every column of a key tile is
tried, each with a query row of its own, because columns differ in how their
exponential is taken and a row that is taken again hides what another one missed.
Bounds are derived in seq_util.py."""
import math

import pytest
import torch

from adaptive_block_sparse_fractal_b200 import nabla

import seq_util

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
TILE = 128


def spikes(value, D, keys=512, first=TILE, heads=1):
    """A sequence for each column of a tile: one query row, `keys` keys that score 0
    but one, at `first` + column, that scores `value` (at scale 1)."""
    g = torch.Generator(device="cuda").manual_seed(int(D))
    q = torch.zeros(TILE, heads, D, dtype=BF, device="cuda")
    q[:, :, 0] = 1.0
    k = torch.zeros(TILE * keys, 1, D, dtype=BF, device="cuda")
    at = torch.arange(TILE, device="cuda")
    k[at * keys + first + at, 0, 0] = value
    v, dout = (torch.randn(n, h, D, generator=g, device="cuda").to(BF)
               for n, h in ((TILE * keys, 1), (TILE, heads)))
    cu = lambda n: torch.arange(TILE + 1, dtype=torch.int32, device="cuda") * n
    return q, k, v, dout, cu(1), cu(keys)


def run(q, k, v, cu_q, cu_k, causal, back=False):
    ws = nabla.packed_workspace(q, k, cu_q.numel() - 1, back=back)
    o, lse = nabla.attn_packed_fwd(q, k, v, cu_q, cu_k, causal=causal, scale=1.0, ws=ws)
    assert nabla.status(ws) == nabla.OK
    return o, lse, ws


# (exact in bf16, as is the score)
@pytest.mark.parametrize("step", [20.0, 60.0, 87.0, 88.0, 91.0, 95.0, 120.0, 200.0, 260.0, 384.0, 600.0, 1000.0])
@pytest.mark.parametrize("D", [64, 128])
def test_one_key_far_above_the_others(D, step):
    q, k, v, _, cu_q, cu_k = spikes(step, D)
    r = seq_util.packed(q, k, v, cu_q.tolist(), cu_k.tolist(), False, scale=1.0)
    for causal in (False, True):  # (one row: it keeps every key either way)
        o, lse, _ = run(q, k, v, cu_q, cu_k, causal)
        seq_util.check(o, r["o"], r["o_tol"], "o")
        seq_util.check_lse(lse, r["lse"])


@pytest.mark.parametrize("step", [95.0, 260.0, 600.0])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_alike(D, step):
    """Two row tiles of equal rows, the key at the last columns of a tile."""
    L, keys = 300, 700
    q = torch.zeros(L, 1, D, dtype=BF, device="cuda")
    q[:, :, 0] = 1.0
    v = torch.randn(keys, 1, D, device="cuda").to(BF)
    cu = lambda n: torch.tensor([0, n], dtype=torch.int32, device="cuda")
    for at in (134, 135, 142, 143, 255, 390):
        k = torch.zeros(keys, 1, D, dtype=BF, device="cuda")
        k[at, 0, 0] = step
        for causal in (False, True):
            o, lse, _ = run(q, k, v, cu(L), cu(keys), causal)
            r = seq_util.packed(q, k, v, [0, L], [0, keys], causal, scale=1.0)
            seq_util.check(o, r["o"], r["o_tol"], "o")
            seq_util.check_lse(lse, r["lse"])


@pytest.mark.parametrize("value", [95.0, 260.0, 1000.0, math.nan])
@pytest.mark.parametrize("D", [64, 128])
def test_key_range_split(D, value):
    """One row on many keys: each part of the key range has its own reference."""
    keys = 9000
    q = torch.zeros(1, 1, D, dtype=BF, device="cuda")
    q[:, :, 0] = 1.0
    v = torch.randn(keys, 1, D, device="cuda").to(BF)
    cu = lambda n: torch.tensor([0, n], dtype=torch.int32, device="cuda")
    # parts begin at multiples of a tile, so some begin with these tiles and some do not
    for tile in (1, 2, 3, 40, 41, 42, 43):
        for col in (6, 7, 14, 15, 62, 63, 64, 78, 127):
            k = torch.zeros(keys, 1, D, dtype=BF, device="cuda")
            k[tile * TILE + col, 0, 0] = value
            o, lse, ws = run(q, k, v, cu(1), cu(keys), True)
            assert ws.numel() > 256  # the key range is split
            if math.isnan(value):
                assert bool(torch.isnan(o).all()) and bool(torch.isnan(lse).all())
                continue
            r = seq_util.packed(q, k, v, [0, 1], [0, keys], True, scale=1.0)
            seq_util.check(o, r["o"], r["o_tol"], "o")
            seq_util.check_lse(lse, r["lse"])


@pytest.mark.parametrize("first", [0, TILE, 2 * TILE])
@pytest.mark.parametrize("D", [64, 128])
def test_nan_and_infinite_keys(D, first):
    """A key that is NaN, or scores +inf, makes the rows that keep it NaN; one that
    scores -inf has no weight."""
    for value in (math.nan, math.inf):
        q, k, v, _, cu_q, cu_k = spikes(value, D, first=first)
        for causal in (False, True):
            o, lse, _ = run(q, k, v, cu_q, cu_k, causal)
            assert bool(torch.isnan(o).all()) and bool(torch.isnan(lse).all())
    q, k, v, _, cu_q, cu_k = spikes(-math.inf, D, first=first)
    r = seq_util.packed(q, k, v, cu_q.tolist(), cu_k.tolist(), False, scale=1.0)
    o, lse, _ = run(q, k, v, cu_q, cu_k, False)
    seq_util.check(o, r["o"], r["o_tol"], "o")
    seq_util.check_lse(lse, r["lse"])


@pytest.mark.parametrize("step", [20.0, 95.0, 260.0, 600.0])
@pytest.mark.parametrize("D", [64, 128])
def test_gradients_behind_it(D, step):
    q, k, v, dout, cu_q, cu_k = spikes(step, D, heads=2)
    o, lse, ws = run(q, k, v, cu_q, cu_k, True, back=True)
    got = nabla.attn_packed_bwd(q, k, v, o, dout, lse, cu_q, cu_k, causal=True, scale=1.0, ws=ws)
    assert nabla.status(ws) == nabla.OK
    r = seq_util.packed(q, k, v, cu_q.tolist(), cu_k.tolist(), True, scale=1.0, dout=dout)
    # exp2(score log2e - lse log2e): at most six roundings of 2^-24 of step log2e in the exponent
    # enter P relatively, where seq_util allows E
    more = 1 + 6 * 2.0 ** -24 * step * 1.4427 / seq_util.E
    for n, t in zip(("dq", "dk", "dv"), got):
        seq_util.check(t, r[n], r[n + "_tol"] * more, n)
