"""Rotary angles at the ends of their range."""
import ctypes

import pytest
import torch

from adaptive_block_sparse_fractal_b200 import build, nabla

BASE = 0x10000000


@pytest.mark.parametrize("pos", [None, BASE])
@pytest.mark.parametrize("kw", [dict(scale=1e300), dict(scale=-1e300), dict(scale=1e20), dict(theta=1e-300),
                                dict(theta=1e-30), dict(offset=1e17), dict(offset=-1e300), dict(scale=1e200, theta=1e-200),
                                dict(offset=(0.0, 0.0, 1e17)), dict(scale=1e308, offset=1e308)])
def test_angles_out_of_range_are_refused(pos, kw):
    build.build()
    p = nabla.rope_params_of((22, 21, 21), **kw)
    p.D, p.dtype = 128, 0
    n = 64
    h = (ctypes.c_int * 2)(2, 0)
    vi = (nabla.View * 2)(nabla.View(BASE + (1 << 30), 0, n * 128, 128))
    vo = (nabla.View * 2)(nabla.View(BASE + (2 << 30), 0, n * 128, 128))
    assert nabla.lib().nabla_rope(ctypes.byref(p), 1, n, 1, 1, 8, 1, h, vi, vo, pos, 0, 3, None) == nabla.ERR_PARAM


@pytest.mark.gpu
@pytest.mark.parametrize("sign", [1, -1])
def test_far_angles_still_rotate(sign):
    """Just inside the range a float64 angle is known to a sixteenth of a turn only, but
    the result is a rotation: the length of a pair stays, within 2^-20 of it (sine and
    cosine are each off by at most 2^-22, four roundings of 2^-24 follow)."""
    N, D = 500, 64
    x = torch.randn(2, N, D, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (N, 1), generator=g, device="cuda").to(torch.int32)
    prm = nabla.rope_params_of((32,), theta=1.0, scale=sign * 0.9 * 2.0 ** 49 * 6.2831853 / 2.0 ** 31)
    y = nabla.rope(prm, x, pos=pos).double().view(2, N, 32, 2)
    a, b = y.norm(dim=-1), x.double().view(2, N, 32, 2).norm(dim=-1)
    assert float(((a - b).abs() / b).max()) <= 2.0 ** -20
    with pytest.raises(nabla.NablaError):
        nabla.rope(nabla.rope_params_of((32,), theta=1.0, scale=1.1 * 2.0 ** 49 * 6.2831853 / 2.0 ** 31), x, pos=pos)
