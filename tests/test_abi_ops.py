"""Host-side refusals of the rotary, packed and cache calls, without a GPU:
every call below fails its checks (or is an empty no-op) before anything is
enqueued, so the made-up pointers are never touched."""
import ctypes

import pytest

from adaptive_block_sparse_fractal_b200 import build, nabla

BASE = 0x10000000


@pytest.fixture(scope="module")
def L():
    build.build()
    return nabla.lib()


def view(addr, token, head=128, batch=0):
    return nabla.View(addr, batch, head, token)


def rope(L, prm=None, B=1, T=4, H=16, W=16, P=8, heads=(2, 2), ins=None, outs=None, pos=None,
         pos_batch=0, axes=0, count=2, D=128, dtype=0, flags=None):
    p = nabla.rope_params_of((22, 21, 21)) if prm is None else prm
    p.D, p.dtype = D, dtype
    if flags is not None:
        p.flags = flags
    n = T * H * W
    size = n * D * 2 * 4
    default = lambda i: nabla.View(BASE + i * size, 0, n * D, D)
    ins = [default(0), default(1)] if ins is None else ins
    outs = [default(2), default(3)] if outs is None else outs
    vi, vo = (nabla.View * 2)(*ins), (nabla.View * 2)(*outs)
    h = (ctypes.c_int * 2)(*heads)
    return L.nabla_rope(ctypes.byref(p), B, T, H, W, P, count, h, vi, vo, pos, pos_batch, axes, None)


def test_rope_rejects_on_host(L):
    P_ = nabla.rope_params_of
    assert rope(L, D=127) == nabla.ERR_SHAPE
    assert rope(L, D=258) == nabla.ERR_SHAPE
    assert rope(L, H=12, flags=nabla.ROPE_FLAT_OUT) == nabla.ERR_SHAPE
    assert rope(L, count=3) == nabla.ERR_SHAPE
    assert rope(L, B=-1) == nabla.ERR_SHAPE
    assert rope(L, dtype=3) == nabla.ERR_PARAM
    assert rope(L, flags=64) == nabla.ERR_PARAM
    assert rope(L, P_((40, 20, 20))) == nabla.ERR_PARAM          # 160 features of 128
    assert rope(L, P_((0, 0, 0))) == nabla.ERR_PARAM
    assert rope(L, P_((-1, 8, 8))) == nabla.ERR_PARAM
    for theta in (0.0, -1.0, float("nan"), float("inf")):
        assert rope(L, P_((8, 8, 8), theta=theta)) == nabla.ERR_PARAM
    assert rope(L, P_((8, 8, 8), offset=float("nan"))) == nabla.ERR_PARAM
    pos = ctypes.c_void_p(BASE)
    assert rope(L, pos=pos, axes=0) == nabla.ERR_PARAM
    assert rope(L, pos=pos, axes=2) == nabla.ERR_PARAM           # three axes are turned
    assert rope(L, pos=pos, axes=3, pos_batch=-1) == nabla.ERR_PARAM
    assert rope(L, pos=ctypes.c_void_p(BASE + 2), axes=3) == nabla.ERR_ALIGN
    n, D = 4 * 16 * 16, 128
    v = lambda addr, token=D, head=n * D: nabla.View(addr, 0, head, token)
    far = 1 << 30
    assert rope(L, ins=[v(None), v(BASE)]) == nabla.ERR_NULL
    assert rope(L, outs=[v(BASE + far), v(BASE + 2 * far + 1)]) == nabla.ERR_ALIGN
    assert rope(L, outs=[v(BASE + far, token=-D), v(BASE + 2 * far)]) == nabla.ERR_PARAM
    assert rope(L, outs=[v(BASE + far, token=0), v(BASE + 2 * far)]) == nabla.ERR_PARAM  # rows coincide
    assert rope(L, outs=[v(BASE + far, token=64), v(BASE + 2 * far)]) == nabla.ERR_PARAM
    assert rope(L, outs=[v(BASE + far), v(BASE + far)]) == nabla.ERR_PARAM               # q_out = k_out
    a, b = v(BASE), v(BASE + far)
    assert rope(L, ins=[a, b], outs=[b, a]) == nabla.ERR_PARAM                           # swapped
    assert rope(L, ins=[a, b], outs=[a, b], flags=nabla.ROPE_FLAT_OUT) == nabla.ERR_PARAM  # in place, reordered
    assert rope(L, ins=[a, b], outs=[v(BASE + 64), b]) == nabla.ERR_PARAM                # shifted
    assert L.nabla_rope(None, 1, 1, 1, 1, 1, 1, None, None, None, None, 0, 0, None) == nabla.ERR_NULL
    assert rope(L, T=0, ins=[v(None), v(None)], outs=[v(None), v(None)]) == nabla.OK     # empty
    assert rope(L, heads=(0, 0), ins=[v(None), v(None)], outs=[v(None), v(None)]) == nabla.OK


def packed(**kw):
    d = dict(seqs=3, heads=8, heads_kv=2, D=128, total_q=1000, total_k=1000, causal=1, scale=0.1)
    d.update(kw)
    return nabla.Packed(*(d[k] for k in ("seqs", "heads", "heads_kv", "D", "total_q", "total_k",
                                         "causal", "scale")))


def fwd(L, s=None, ws=BASE, ws_bytes=1 << 40, cu=BASE, **v):
    s = packed() if s is None else s
    far = 1 << 30
    d = {n: view(BASE + (i + 1) * far, token=1024) for i, n in enumerate("qkvo")}
    d.update(v)
    r = lambda n: None if d[n] is None else ctypes.byref(d[n])
    return L.nabla_attn_packed_fwd(ctypes.byref(s), r("q"), r("k"), r("v"), cu, cu, r("o"), None, ws,
                                   ws_bytes, None)


def test_packed_forward_rejects_on_host(L):
    for bad in (dict(D=96), dict(heads=7), dict(seqs=0), dict(heads_kv=0), dict(total_q=-1),
                dict(total_k=1 << 31), dict(total_q=1 << 29)):
        assert fwd(L, packed(**bad)) == nabla.ERR_SHAPE
        assert L.nabla_packed_workspace_size(ctypes.byref(packed(**bad)), 0) == 0
    for bad in (dict(scale=0.0), dict(scale=float("nan")), dict(causal=2)):
        assert fwd(L, packed(**bad)) == nabla.ERR_PARAM
    assert fwd(L, q=None) == nabla.ERR_NULL
    assert fwd(L, v=view(None, 1024)) == nabla.ERR_NULL
    assert fwd(L, cu=None) == nabla.ERR_NULL
    assert fwd(L, cu=BASE + 2) == nabla.ERR_ALIGN
    assert fwd(L, k=view(BASE + 8, 1024)) == nabla.ERR_ALIGN
    assert fwd(L, k=view(BASE, 1028)) == nabla.ERR_ALIGN
    assert fwd(L, o=view(BASE, 1024, head=64)) == nabla.ERR_PARAM       # heads of o overlap
    assert fwd(L, q=view(BASE, 0)) == nabla.ERR_PARAM
    far = 1 << 30
    assert fwd(L, o=view(BASE + far, 1024)) == nabla.ERR_PARAM          # o is q
    assert fwd(L, o=view(BASE + 2 * far + 16, 1024)) == nabla.ERR_PARAM
    assert fwd(L, ws=None) == nabla.ERR_WORKSPACE
    assert fwd(L, ws_bytes=255) == nabla.ERR_WORKSPACE
    assert fwd(L, ws=BASE + 128) == nabla.ERR_ALIGN
    assert L.nabla_packed_workspace_size(ctypes.byref(packed()), 7) == 0
    # few rows against many keys take room for the parts of the key range
    small, few = packed(seqs=1), packed(seqs=1, total_q=1, total_k=100000)
    size = lambda s: L.nabla_packed_workspace_size(ctypes.byref(s), nabla.PACKED_FWD)
    assert size(packed()) == 256 and size(few) > size(small)


def cache(**kw):
    d = dict(pages=100, page_size=16, heads_kv=2, D=128, seqs=3, width=8, k=BASE, v=BASE + (1 << 30),
             table=BASE, token=256, page=4096)
    d.update(kw)
    vw = lambda a: nabla.View(a, d["page"], 128, d["token"])
    return nabla.Cache(vw(d["k"]), vw(d["v"]), d["table"], d["pages"], d["page_size"], d["heads_kv"],
                       d["D"], d["seqs"], d["width"])


def test_append_rejects_on_host(L):
    far = 1 << 32
    src = view(far, 256)

    def call(c=None, k=src, v=src, total=3, starts=BASE, cu=None, ws=None, n=0):
        return L.nabla_cache_append(ctypes.byref(cache() if c is None else c), ctypes.byref(k),
                                    ctypes.byref(v), total, starts, cu, ws, n, None)
    for bad in (dict(D=20), dict(pages=0), dict(page_size=0), dict(heads_kv=0), dict(width=0), dict(seqs=-1)):
        assert call(cache(**bad)) == nabla.ERR_SHAPE
    assert call(total=4) == nabla.ERR_SHAPE                       # one row a sequence without borders
    assert call(cache(k=None)) == nabla.ERR_NULL
    assert call(cache(table=None)) == nabla.ERR_NULL
    assert call(starts=None) == nabla.ERR_NULL
    assert call(cache(k=BASE + 8)) == nabla.ERR_ALIGN
    assert call(cache(token=250)) == nabla.ERR_ALIGN
    assert call(cache(token=128)) == nabla.ERR_PARAM              # rows of the pool overlap
    assert call(cache(v=BASE)) == nabla.ERR_PARAM                 # K and V in one place
    assert call(k=view(BASE + 512, 256)) == nabla.ERR_PARAM       # source inside the pool
    assert call(starts=BASE + 2) == nabla.ERR_ALIGN
    assert call(ws=BASE, n=16) == nabla.ERR_WORKSPACE
    assert call(ws=BASE + 64, n=256) == nabla.ERR_ALIGN
    assert call(cache(seqs=0), total=0, starts=None) == nabla.OK  # empty


def test_paged_rejects_on_host(L):
    far = 1 << 32

    def call(c=None, heads=4, scale=0.1, q=view(far, 512), lens=BASE, o=view(2 * far, 512), ws=BASE, n=1 << 40):
        return L.nabla_attn_paged(ctypes.byref(cache() if c is None else c), heads, scale,
                                  ctypes.byref(q), lens, ctypes.byref(o), None, ws, n, None)
    for bad in (dict(D=72), dict(D=256), dict(pages=0)):
        assert call(cache(**bad)) == nabla.ERR_SHAPE
        assert L.nabla_paged_workspace_size(ctypes.byref(cache(**bad)), 4) == 0
    assert call(heads=3) == nabla.ERR_SHAPE and call(heads=0) == nabla.ERR_SHAPE
    assert call(scale=-1.0) == nabla.ERR_PARAM and call(scale=float("inf")) == nabla.ERR_PARAM
    assert call(cache(v=None)) == nabla.ERR_NULL
    assert call(lens=None) == nabla.ERR_NULL
    assert call(q=view(far + 2, 512)) == nabla.ERR_ALIGN
    assert call(lens=BASE + 1) == nabla.ERR_ALIGN
    assert call(o=view(far, 512)) == nabla.ERR_PARAM              # o is q
    assert call(o=view(BASE, 512)) == nabla.ERR_PARAM             # o inside the pool
    assert call(ws=None) == nabla.ERR_WORKSPACE and call(n=1000) == nabla.ERR_WORKSPACE


def test_binding_refuses_what_it_is_not_given():
    import torch
    x = torch.zeros(2, 8, 64, dtype=torch.bfloat16)  # not on a GPU
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        nabla.rope(nabla.rope_params_of((8, 8, 8)), x, grid=(8, 1, 1))
    with pytest.raises(ValueError):
        nabla.rope(nabla.rope_params_of((8, 8, 8)), x)            # neither grid nor positions
    with pytest.raises(ValueError):
        nabla.rope_params_of((8, 8, 8, 8))
    with pytest.raises(ValueError):
        nabla.attn_packed_fwd(x, x, x, cu, cu)
    with pytest.raises(ValueError):
        nabla.attn_paged(x, x[None], x[None], cu[None], cu)


def test_packed_backward_rejects_on_host(L):
    far = 1 << 30
    names = ("q", "k", "v", "o", "dout", "dq", "dk", "dv")

    def call(s=None, lse=BASE, ws=BASE, ws_bytes=1 << 40, **v):
        s = packed() if s is None else s
        d = {n: view(BASE + (i + 1) * far, token=1024) for i, n in enumerate(names)}
        d.update(v)
        r = lambda n: None if d[n] is None else ctypes.byref(d[n])
        return L.nabla_attn_packed_bwd(ctypes.byref(s), *(r(n) for n in names[:5]), lse, BASE, BASE,
                                       *(r(n) for n in names[5:]), ws, ws_bytes, None)
    assert call(packed(D=32)) == nabla.ERR_SHAPE
    assert call(packed(scale=-1.0)) == nabla.ERR_PARAM
    for n in names:
        assert call(**{n: None}) == nabla.ERR_NULL
        assert call(**{n: view(BASE + 20 * far + 4, 1024)}) == nabla.ERR_ALIGN
    assert call(lse=None) == nabla.ERR_NULL
    assert call(lse=BASE + 2) == nabla.ERR_ALIGN
    assert call(ws_bytes=256) == nabla.ERR_WORKSPACE
    assert call(dq=view(BASE + far, 1024)) == nabla.ERR_PARAM         # dq is q
    assert call(dk=view(BASE + 8 * far, 1024)) == nabla.ERR_PARAM     # dk is dv
    assert call(dv=view(BASE + 20 * far, 64)) == nabla.ERR_PARAM      # rows of dv overlap
    size = lambda op: L.nabla_packed_workspace_size(ctypes.byref(packed()), op)
    assert size(nabla.PACKED_BWD) == 256 + 2 * ((4 * (1000 // 64 + 3) * 64 * 8 + 255) // 256 * 256)
