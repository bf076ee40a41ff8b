"""Softmax scales that leave float32 once they are in units of log2 (CPU)."""
import ctypes

import pytest

from adaptive_block_sparse_fractal_b200 import build, nabla

at = lambda i: (1 << 40) + (i << 32)


@pytest.mark.parametrize("scale", [2.4e38, 3.4e38, float("inf"), float("nan"), 0.0, -1.0])
def test_scale_is_refused(scale):
    build.build()
    L = nabla.lib()
    v = lambda i, token: ctypes.byref(nabla.View(at(i), 0, 128, token))
    s = nabla.Packed(1, 2, 2, 128, 10, 10, 0, scale)
    assert L.nabla_attn_packed_fwd(ctypes.byref(s), v(1, 256), v(2, 256), v(3, 256), at(4), at(5), v(6, 256), None,
                                   at(7), 1 << 30, None) == nabla.ERR_PARAM
    vw = lambda i: nabla.View(at(i), 4096, 128, 256)
    c = nabla.Cache(vw(1), vw(2), at(3), 100, 16, 2, 128, 3, 8)
    assert L.nabla_attn_paged(ctypes.byref(c), 4, scale, v(4, 512), at(5), v(6, 512), None, at(7), 1 << 30,
                              None) == nabla.ERR_PARAM
