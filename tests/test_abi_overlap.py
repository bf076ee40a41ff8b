"""Refusals of outputs that overlap an input, a workspace or another output (CPU:
each call fails this check before anything is enqueued)."""
import ctypes

import pytest

from adaptive_block_sparse_fractal_b200 import build, nabla

FAR = 1 << 32
at = lambda i: (1 << 40) + i * FAR


@pytest.fixture(scope="module")
def L():
    build.build()
    return nabla.lib()


def view(addr, token):
    return nabla.View(addr, 0, 128, token)


SHAPE = dict(seqs=3, heads=8, heads_kv=2, D=128, total_q=1000, total_k=700, causal=1, scale=0.1)
TOTALS = {"q": 1000, "o": 1000, "dout": 1000, "dq": 1000, "k": 700, "v": 700, "dk": 700, "dv": 700}
HEADS = {n: 8 if n in ("q", "o", "dout", "dq") else 2 for n in TOTALS}
TAIL = {n: 2 * ((t - 1) * HEADS[n] * 128 + HEADS[n] * 128) - 16 for n, t in TOTALS.items()}  # the last 16 bytes


def packed(L, names, outs, back, **moved):
    """One call with every buffer far from the others but those in `moved`."""
    s = nabla.Packed(*(SHAPE[k] for k in ("seqs", "heads", "heads_kv", "D", "total_q", "total_k", "causal", "scale")))
    every = list(names) + ["lse", "cu_q", "cu_k", "ws"]
    p = {n: at(i + 1) for i, n in enumerate(every)}
    p.update(moved)
    v = {n: ctypes.byref(view(p[n], HEADS[n] * 128)) for n in names}
    need = L.nabla_packed_workspace_size(ctypes.byref(s), nabla.PACKED_BWD if back else nabla.PACKED_FWD)
    if back:
        return L.nabla_attn_packed_bwd(ctypes.byref(s), *(v[n] for n in names[:5]), p["lse"], p["cu_q"], p["cu_k"],
                                       *(v[n] for n in names[5:]), p["ws"], need, None)
    return L.nabla_attn_packed_fwd(ctypes.byref(s), v["q"], v["k"], v["v"], p["cu_q"], p["cu_k"], v["o"],
                                   p["lse"], p["ws"], need, None)


def test_packed_forward(L):
    names = ("q", "k", "v", "o")
    where = {n: at(i + 1) for i, n in enumerate(names)}
    for n in names:
        assert packed(L, names, ("o",), False, lse=where[n] + TAIL[n]) == nabla.ERR_PARAM
        assert packed(L, names, ("o",), False, ws=where[n] + 256) == nabla.ERR_PARAM
        if n != "o":
            assert packed(L, names, ("o",), False, o=where[n] + TAIL[n]) == nabla.ERR_PARAM
    assert packed(L, names, ("o",), False, lse=at(20), ws=at(20) + 256) == nabla.ERR_PARAM
    for n in ("cu_q", "cu_k"):
        assert packed(L, names, ("o",), False, **{n: where["o"] + 4}) == nabla.ERR_PARAM
        assert packed(L, names, ("o",), False, lse=at(20), **{n: at(20) + 4 * 8 * 1000 - 4}) == nabla.ERR_PARAM


def test_packed_backward(L):
    names = ("q", "k", "v", "o", "dout", "dq", "dk", "dv")
    where = {n: at(i + 1) for i, n in enumerate(names)}
    for out in names[5:]:
        for n in names:
            if n != out:
                assert packed(L, names, names[5:], True, **{out: where[n] + TAIL[n]}) == nabla.ERR_PARAM
        assert packed(L, names, names[5:], True, lse=where[out] + TAIL[out]) == nabla.ERR_PARAM
        assert packed(L, names, names[5:], True, cu_k=where[out]) == nabla.ERR_PARAM
    for n in names:
        assert packed(L, names, names[5:], True, ws=where[n] + 512) == nabla.ERR_PARAM
    assert packed(L, names, names[5:], True, lse=at(20), ws=at(20) + 256) == nabla.ERR_PARAM


def cache(**kw):
    d = dict(k=at(1), v=at(2), table=at(3), pages=100, page_size=16, heads_kv=2, D=128, seqs=3, width=8)
    d.update(kw)
    vw = lambda a: nabla.View(a, 4096, 128, 256)
    return nabla.Cache(vw(d["k"]), vw(d["v"]), d["table"], d["pages"], d["page_size"], d["heads_kv"], d["D"],
                       d["seqs"], d["width"])


POOL = 2 * 100 * 16 * 2 * 128  # bytes


def test_append(L):
    def call(c=None, k=at(4), v=at(5), starts=at(6), cu=at(7), ws=at(8)):
        return L.nabla_cache_append(ctypes.byref(cache() if c is None else c), ctypes.byref(view(k, 256)),
                                    ctypes.byref(view(v, 256)), 30, starts, cu, ws, 256, None)
    for pool in (at(1), at(2)):
        assert call(k=pool + POOL - 16) == nabla.ERR_PARAM and call(v=pool) == nabla.ERR_PARAM
        assert call(starts=pool + 8) == nabla.ERR_PARAM and call(cu=pool + POOL - 4) == nabla.ERR_PARAM
        assert call(ws=pool + 256) == nabla.ERR_PARAM
        assert call(cache(table=pool + 4)) == nabla.ERR_PARAM
    assert call(cu=at(8) + 4) == nabla.ERR_PARAM and call(k=at(8)) == nabla.ERR_PARAM
    assert call(cache(v=at(1) + POOL - 16)) == nabla.ERR_PARAM


def test_paged(L):
    def call(c=None, q=at(4), lens=at(5), o=at(6), lse=at(7), ws=at(8)):
        c = cache() if c is None else c
        return L.nabla_attn_paged(ctypes.byref(c), 4, 0.1, ctypes.byref(view(q, 512)), lens,
                                  ctypes.byref(view(o, 512)), lse, ws,
                                  L.nabla_paged_workspace_size(ctypes.byref(c), 4), None)
    for where in (at(1), at(2), at(4)):
        assert call(o=where + 16) == nabla.ERR_PARAM
        assert call(lse=where + 4) == nabla.ERR_PARAM and call(ws=where + 256) == nabla.ERR_PARAM
    assert call(lse=at(6) + 4) == nabla.ERR_PARAM and call(ws=at(6)) == nabla.ERR_PARAM
    assert call(lse=at(8) + 1024) == nabla.ERR_PARAM
    assert call(lens=at(6)) == nabla.ERR_PARAM and call(lens=at(8) + 4) == nabla.ERR_PARAM
    assert call(cache(table=at(7) + 8)) == nabla.ERR_PARAM


def test_rope_positions(L):
    p = nabla.rope_params_of((22, 21, 21))
    p.D, p.dtype = 128, 0
    n, h = 64, (ctypes.c_int * 2)(2, 0)
    vi, vo = (nabla.View * 2)(nabla.View(at(1), 0, n * 128, 128)), (nabla.View * 2)(nabla.View(at(2), 0, n * 128, 128))
    for pos in (at(2), at(2) + 2 * 2 * n * 128 - 4):
        assert L.nabla_rope(ctypes.byref(p), 1, n, 1, 1, 8, 1, h, vi, vo, pos, 0, 3, None) == nabla.ERR_PARAM
