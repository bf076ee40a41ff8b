"""Appending with borders that are no borders: nothing is written, and it is said."""
import pytest
import torch

from adaptive_block_sparse_fractal_b200 import nabla

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(seqs, total, page=16, heads_kv=2, D=64, width=60):
    g = torch.Generator(device="cuda").manual_seed(total)
    shape = (seqs * width, page, heads_kv, D)
    kc, vc = (torch.randn(shape, generator=g, device="cuda").to(BF) for _ in range(2))
    k, v = (torch.randn(total, heads_kv, D, generator=g, device="cuda").to(BF) for _ in range(2))
    table = torch.randperm(seqs * width, generator=g, device="cuda").to(torch.int32).view(seqs, width)
    return k, v, kc, vc, table


# of 40 rows and of 700 (several CTAs; their status word is set by a memset and the kernel)
@pytest.mark.parametrize("total,cu", [(40, [0, 30, 20, 40]), (40, [0, 41, 41, 41]), (40, [-1, 10, 20, 40]),
                                      (40, [0, 10, 20, 41]), (40, [30, 20, 10, 0]), (40, [0, 2 ** 31 - 1, -2 ** 31, 40]),
                                      (700, [0, 500, 499, 700]), (700, [0, 10, 20, 701]), (700, [-5, 10, 20, 700])])
def test_bad_borders_write_nothing(total, cu):
    k, v, kc, vc, table = make(3, total)
    before = kc.clone(), vc.clone()
    ws = nabla.cache_workspace("cuda")
    starts = dev([0, 17, 5])
    nabla.cache_append(k, v, kc, vc, table, starts, cu=dev(cu), ws=ws)
    assert nabla.status(ws) == nabla.ERR_PARAM
    assert torch.equal(kc, before[0]) and torch.equal(vc, before[1])
    nabla.cache_append(k, v, kc, vc, table, starts, cu=dev(cu))  # unreported, unwritten
    torch.cuda.synchronize()
    assert torch.equal(kc, before[0]) and torch.equal(vc, before[1])
    good = [0, 10, 10, total]
    nabla.cache_append(k, v, kc, vc, table, starts, cu=dev(good), ws=ws)
    assert nabla.status(ws) == nabla.OK
    want = before[0].clone(), before[1].clone()
    for s in range(3):
        p = int(starts[s]) + torch.arange(good[s + 1] - good[s], device="cuda")
        at = table[s, p // 16].long(), p % 16
        want[0][at], want[1][at] = k[good[s]:good[s + 1]], v[good[s]:good[s + 1]]
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])


@pytest.mark.parametrize("seqs", [1, 255, 256, 257, 900])
def test_many_sequences_one_bad_border(seqs):
    total = 2 * seqs
    k, v, kc, vc, table = make(seqs, total, width=2)
    before = kc.clone()
    cu = torch.arange(seqs + 1, dtype=torch.int32) * 2
    ws = nabla.cache_workspace("cuda")
    starts = dev([3] * seqs)
    nabla.cache_append(k, v, kc, vc, table, starts, cu=cu.cuda(), ws=ws)
    assert nabla.status(ws) == nabla.OK and not torch.equal(kc, before)
    kc.copy_(before)
    cu[seqs] += 1  # one row more than there are
    nabla.cache_append(k, v, kc, vc, table, starts, cu=cu.cuda(), ws=ws)
    assert nabla.status(ws) == nabla.ERR_PARAM and torch.equal(kc, before)


@pytest.mark.parametrize("seqs,longest", [(1024, 40), (1025, 40), (3000, 12), (20000, 3)])
def test_many_sequences(seqs, longest):
    """Groups of rows that follow one another in a CTA, empty sequences among them."""
    g = torch.Generator().manual_seed(seqs)
    lens = torch.randint(0, longest + 1, (seqs,), generator=g)
    lens[-1] = longest
    starts = torch.randint(0, 9, (seqs,), generator=g)
    cu = torch.cat([torch.zeros(1, dtype=torch.long), lens.cumsum(0)])
    total, width = int(cu[-1]), -(-(longest + 9) // 16)
    k, v, kc, vc, table = make(seqs, total + 3, width=width, heads_kv=1)
    want = kc.clone(), vc.clone()
    seq = torch.repeat_interleave(torch.arange(seqs), lens)
    p = (starts[seq] + torch.arange(total) - cu[seq]).cuda()
    at = table[seq.cuda(), p // 16].long(), p % 16
    want[0][at], want[1][at] = k[:total], v[:total]
    ws = nabla.cache_workspace("cuda")
    nabla.cache_append(k, v, kc, vc, table, starts.to("cuda", torch.int32), cu=cu.to("cuda", torch.int32), ws=ws)
    assert nabla.status(ws) == nabla.OK
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])
    # a bad page under a late group of rows
    table[int(seq[-2]), :] = -1
    nabla.cache_append(k, v, kc, vc, table, starts.to("cuda", torch.int32), cu=cu.to("cuda", torch.int32), ws=ws)
    assert nabla.status(ws) == nabla.ERR_PARAM
