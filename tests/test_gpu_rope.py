"""Rotary positions against float64, over types, layouts, token orders,
strides and far positions.

Tolerance.  An output is a c - b s rounded once to its type.  With |c|, |s| <= 1
and a, b the inputs, the float32 steps add at most 4 roundings of 2^-24 of
(|a| + |b|), and the float32 sine and cosine of an exactly reduced angle are off
by at most 2^-22 (the series leave out less than 2^-25, their argument, below
pi/4, is rounded at 2^-25, and a few roundings of 2^-25 follow).  So: half a step
of the type relative to the value, plus 2^-21 (|a| + |b|)."""
import pytest
import torch

from adaptive_block_sparse_fractal_b200 import nabla

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def flat_places(T, H, W, P=8):
    v = torch.arange(T * H * W).view(T, H // P, P, W // P, P)
    return v.permute(0, 1, 3, 2, 4).reshape(-1)  # grid token at each flattened place


def reference(x, pairs, pos, theta, scale, offset, layout, inverse):
    """x [..., N, D] float64 (CPU), pos [N, 3] or [B, N, 3]; grid order."""
    ang = []
    for a, n in enumerate(pairs):
        f = torch.tensor([theta[a] ** (-i / n) for i in range(n)], dtype=torch.float64)
        ang.append(((pos[..., a].double() + offset[a]) * scale[a])[..., None] * f)
    ang = torch.cat(ang, -1)
    c, s = ang.cos(), ang.sin() * (-1 if inverse else 1)
    if pos.dim() == 3:
        c, s = c[:, None], s[:, None]
    R = sum(pairs)
    y = x.clone()
    if layout == nabla.ROPE_ADJACENT:
        i, j = torch.arange(0, 2 * R, 2), torch.arange(1, 2 * R, 2)
    else:
        i, j = torch.arange(R), torch.arange(R, 2 * R)
    a, b = x[..., i], x[..., j]
    y[..., i], y[..., j] = a * c - b * s, b * c + a * s
    mag = torch.zeros_like(x)
    mag[..., i] = mag[..., j] = a.abs() + b.abs()
    return y, mag


def close(got, want, mag, dtype):
    got = got.double().cpu()
    tol = want.abs() * (torch.finfo(dtype).eps / 2 * 1.01) + mag * 2.0 ** -21
    if dtype == HF:
        tol = tol + 2.0 ** -25  # subnormal outputs
    assert bool(((got - want).abs() <= tol).all()), float(((got - want).abs() - tol).max())


def grid_pos(T, H, W):
    return torch.stack(torch.meshgrid(torch.arange(T), torch.arange(H), torch.arange(W),
                                      indexing="ij"), -1).reshape(-1, 3)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("layout", [nabla.ROPE_ADJACENT, nabla.ROPE_HALVES])
@pytest.mark.parametrize("flat", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("D,pairs", [(64, (16, 8, 8)), (128, (22, 21, 21)), (128, (8, 16, 8)),
                                     (6, (1, 1, 1)), (80, (0, 7, 6))])
def test_grid(dtype, layout, flat, D, pairs):
    T, H, W, hq, hk = 3, 8, 16, 3, 2
    N = T * H * W
    g = torch.Generator().manual_seed(D + 7 * layout)
    q = torch.randn(hq, N, D, generator=g).to(dtype)
    k = torch.randn(hk, N, D, generator=g).to(dtype)
    for inverse in (False, True):
        prm = nabla.rope_params_of(pairs, theta=(10000.0, 500.0, 77.0), scale=(1.0, 0.5, 2.0),
                                   offset=(3.0, 0.0, -1.5), layout=layout, inverse=inverse)
        qo, ko = nabla.rope(prm, q.cuda(), k.cuda(), grid=(T, H, W), flat_in=flat[0],
                            flat_out=flat[1])
        place = flat_places(T, H, W)
        for x, y in ((q, qo), (k, ko)):
            z = x.double()
            if flat[0]:
                grid = torch.empty_like(z)
                grid[:, place] = z
                z = grid
            want, mag = reference(z, pairs, grid_pos(T, H, W), (10000.0, 500.0, 77.0),
                                  (1.0, 0.5, 2.0), (3.0, 0.0, -1.5), layout, inverse)
            if flat[1]:
                want, mag = want[:, place], mag[:, place]
            close(y, want, mag, dtype)


@pytest.mark.parametrize("N", [1, 2, 77, 333])
@pytest.mark.parametrize("layout,pairs,D", [(nabla.ROPE_ADJACENT, (5, 3), 24),
                                            (nabla.ROPE_HALVES, (8, 8), 64),
                                            (nabla.ROPE_HALVES, (5,), 33 * 2),
                                            (nabla.ROPE_ADJACENT, (64, 64), 256)])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_given_positions_far_and_negative(N, layout, pairs, D, dtype):
    g = torch.Generator().manual_seed(N)
    B, hq, hk = 2, 5, 1
    q = torch.randn(B, N, hq + hk, D, generator=g).to(dtype)
    pos = torch.randint(-50, 2 ** 24, (B, N, len(pairs)), generator=g, dtype=torch.int32)
    prm = nabla.rope_params_of(pairs, theta=1e6, layout=layout)
    qk = q.cuda()
    views = qk[:, :, :hq].transpose(1, 2), qk[:, :, hq:].transpose(1, 2)  # of one projection
    qo, ko = nabla.rope(prm, *views, pos=pos.cuda())
    for x, y in zip(views, (qo, ko)):
        z = x.double().cpu()
        want, mag = reference(z, pairs, pos, (1e6,) * 3, (1.0,) * 3, (0.0,) * 3, layout, False)
        close(y, want, mag, dtype)
    # positions shared by the batch
    qo = nabla.rope(prm, views[0], pos=pos[0].contiguous().cuda())
    want, mag = reference(views[0].double().cpu(), pairs, pos[0], (1e6,) * 3, (1.0,) * 3,
                          (0.0,) * 3, layout, False)
    close(qo, want, mag, dtype)


@pytest.mark.parametrize("layout", [nabla.ROPE_ADJACENT, nabla.ROPE_HALVES])
def test_in_place_on_a_fused_projection_leaves_the_rest(layout):
    N, D = 100, 64
    x = torch.randn(N, 9, D, device="cuda").to(BF)  # 4 q heads, 2 k heads, 3 others
    prm = nabla.rope_params_of((8, 4, 4), layout=layout)
    pos = torch.randint(0, 500, (N, 3), device="cuda", dtype=torch.int32)
    q, k = x[:, :4].transpose(0, 1), x[:, 4:6].transpose(0, 1)
    want = nabla.rope(prm, q.clone(), k.clone(), pos=pos)
    rest = x[:, 6:].clone()
    got = nabla.rope(prm, q, k, pos=pos, q_out=q, k_out=k)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(x[:, 6:], rest)


def test_plain_features_are_copied_whatever_they_hold():
    N, D = 9, 64
    x = torch.randn(2, N, D, device="cuda").to(BF)
    x[:, :, 40:] = float("nan")
    x[:, 3, 50] = float("inf")
    prm = nabla.rope_params_of((10, 6, 4))
    y = nabla.rope(prm, x, grid=(N, 1, 1))
    assert bool(torch.isfinite(y[:, :, :40]).all())
    assert torch.equal(y[:, :, 40:].view(torch.int16), x[:, :, 40:].view(torch.int16))


def test_gradient_of_the_flattening_call():
    """<dy, rope(x)> = <rope^T(dy), x> and the formula's differences."""
    T, H, W, D = 2, 16, 8, 32
    N = T * H * W
    pairs = (6, 5, 5)
    x = torch.randn(3, N, D, device="cuda")
    dy = torch.randn(3, N, D, device="cuda")
    fwd = nabla.rope_params_of(pairs)
    back = nabla.rope_params_of(pairs, inverse=True)
    y = nabla.rope(fwd, x, grid=(T, H, W), flat_out=True)
    dx = nabla.rope(back, dy, grid=(T, H, W), flat_in=True)
    a, b = (dy.double() * y.double()).sum(), (dx.double() * x.double()).sum()
    assert abs(a - b) <= 2.0 ** -20 * (dy.double().abs() * y.double().abs()).sum()
    e = torch.zeros_like(x)
    e[1, 37, 9] = 1.0  # the map is linear: a difference is exact up to rounding
    d = (nabla.rope(fwd, x + e, grid=(T, H, W), flat_out=True).double() - y.double())
    assert abs((d * dy.double()).sum() - dx[1, 37, 9].double()) <= 2.0 ** -17


def test_stream_and_graph():
    x = torch.randn(4, 64, 64, device="cuda").to(BF)
    prm = nabla.rope_params_of((16, 16))
    want = nabla.rope(prm, x, grid=(4, 16, 1))
    out = torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        nabla.rope(prm, x, grid=(4, 16, 1), q_out=out)
    s.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nabla.rope(prm, x, grid=(4, 16, 1), q_out=out)
    x.copy_(torch.randn_like(x, dtype=torch.float32).to(BF))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, nabla.rope(prm, x, grid=(4, 16, 1)))
