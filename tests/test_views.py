"""The host's arithmetic of strided views (csrc/views.h) against sets of bytes (CPU)."""
import ctypes
import os
import random
import subprocess
import tempfile

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def L():
    out = os.path.join(tempfile.mkdtemp(), "libview_check.so")
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-o", out,
                           os.path.join(HERE, "view_check.cpp")])
    return ctypes.CDLL(out)


def pack(addr, n, stride, D, size):
    return (ctypes.c_int64 * 9)(addr, *n, *stride, D, size)


def rows(addr, n, stride, D, size):
    """The bytes of each row."""
    s = [a if k > 1 else 0 for a, k in zip(stride, n)]
    for i in range(n[0]):
        for j in range(n[1]):
            for k in range(n[2]):
                at = addr + (i * s[0] + j * s[1] + k * s[2]) * size
                yield range(at, at + D * size)


def cover(*v):
    return set(x for r in rows(*v) for x in r)


def any_view(rng):
    n = [rng.choice([1, 1, 2, 3, 4]) for _ in range(3)]
    D, size = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4])
    if rng.random() < 0.6:  # dimensions that lie inside one another, with gaps, in any order
        order = [0, 1, 2]
        rng.shuffle(order)
        stride, inner = [0] * 3, D + rng.choice([0, 0, 1, D])
        for i in order:
            stride[i] = inner
            inner = inner * n[i] + rng.choice([0, 0, 1, inner])
    else:
        stride = [rng.randrange(0, 40) for _ in range(3)]
    return 4096 + rng.randrange(0, 200), n, stride, D, size


def test_disjoint_is_exact(L):
    rng = random.Random(1)
    seen = [0, 0]
    for _ in range(6000):
        a, b = any_view(rng), any_view(rng)
        if rng.random() < 0.5:  # slices of one buffer
            b = (a[0] + rng.randrange(0, 64),) + a[1:]
        want = not (cover(*a) & cover(*b))
        assert L.view_disjoint(pack(*a), pack(*b)) == want, (a, b)
        assert L.view_disjoint(pack(*b), pack(*a)) == want, (a, b)
        seen[want] += 1
    assert min(seen) > 500


def test_self_disjoint_is_exact(L):
    rng = random.Random(2)
    seen = [0, 0]
    for _ in range(4000):
        a = any_view(rng)
        all_rows = list(rows(*a))
        want = len(cover(*a)) == sum(len(r) for r in all_rows)
        assert L.view_self_disjoint(pack(*a)) == want, a
        seen[want] += 1
    assert min(seen) > 500


def test_views_of_real_size(L):
    D, H, N, B = 128, 40, 76800, 3
    at = 1 << 40
    w = 3 * H  # q, k and v heads of one projection

    def part(i, n, stride, heads=H, first=None):
        return pack(at + 2 * (i * H * D if first is None else first), [n[0], heads, n[1]], stride, D, 2)
    fused = [N * w * D, D, w * D]
    for n in ((B, N), (1, N), (B, 1), (1, 1)):  # tokens in front; a single token a batch entry too
        q, k, v = (part(i, n, [n[1] * w * D, D, w * D]) for i in range(3))
        assert L.view_disjoint(q, k) == L.view_disjoint(q, v) == L.view_disjoint(k, v) == 1
        assert L.view_disjoint(q, q) == 0 and L.view_self_disjoint(q) == 1
    # heads in front of the tokens, q and k of a head beside one another
    q, k = (part(0, (1, N), [0, 2 * N * D, D], first=i * N * D) for i in range(2))
    assert L.view_disjoint(q, k) == 1
    # one feature too many on either side
    assert L.view_disjoint(part(0, (B, N), fused), part(0, (B, N), fused, first=H * D - 1)) == 0
    assert L.view_disjoint(part(0, (B, N), fused), part(0, (B, N), fused, first=w * D - 1)) == 0
    assert L.view_disjoint(part(0, (1, N), fused), part(0, (1, N), fused, first=N * w * D)) == 1
    # K and V rows of one pool, inside the page, inside the row, and one page apart
    pages, page, heads = 100000, 64, 8
    for k_at, v_at, s in ((0, page * heads * D, [2 * page * heads * D, D, heads * D]),
                          (0, heads * D, [2 * page * heads * D, D, 2 * heads * D]),
                          (0, D, [2 * page * heads * D, 2 * D, 2 * heads * D])):
        k, v = (pack(at + 2 * x, [pages, heads, page], s, D, 2) for x in (k_at, v_at))
        assert L.view_disjoint(k, v) == 1
        shifted = pack(at + 2 * (v_at + 8), [pages, heads, page], s, D, 2)
        assert L.view_disjoint(k, shifted) == 0
    # distances that are not nested: an answer within the bound on the search, never a wrong yes
    odd = pack(at, [1, 1 << 20, 1 << 20], [0, 1031, 1033], D, 2)
    assert L.view_self_disjoint(odd) == 0
    assert L.view_disjoint(pack(at, [0, 4, 4], [1, 1, 1], D, 2), part(0, (B, N), fused)) == 1  # no elements
    assert L.view_disjoint(pack(at, [1, 4, 4], [1, -1, 1], D, 2), part(0, (B, N), fused)) == -1
    assert L.view_disjoint(pack(at, [1, 4, 4], [1, 1 << 46, 1], D, 2), part(0, (B, N), fused)) == -1
