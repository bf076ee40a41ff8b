"""Outputs that lie between the rows of an input, or of another output, without
sharing any: slices of one buffer in every order of its dimensions."""
import pytest
import torch

from adaptive_block_sparse_fractal_b200 import nabla

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def test_rope_of_one_token_a_batch_entry_in_place():
    """A decoding step: q and k of a fused projection of B sequences, one token each."""
    B, hq, hk, D = 5, 6, 2, 64
    x = torch.randn(B, 1, hq + 2 * hk, D, device="cuda").to(BF)
    pos = torch.randint(0, 4000, (B, 1, 3), device="cuda", dtype=torch.int32)
    prm = nabla.rope_params_of((16, 8, 8))
    q, k = x[:, :, :hq].transpose(1, 2), x[:, :, hq:hq + hk].transpose(1, 2)
    want = nabla.rope(prm, q.clone(), k.clone(), pos=pos)
    rest = x[:, :, hq + hk:].clone()
    nabla.rope(prm, q, k, pos=pos, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(x[:, :, hq + hk:], rest)


@pytest.mark.parametrize("batch", [1, 3])
def test_rope_of_heads_that_stand_in_turn(batch):
    """[B, heads, 4, N, D]: q, k and their results of a head beside one another."""
    heads, N, D = 3, 40, 32
    x = torch.randn(batch, heads, 4, N, D, device="cuda").to(BF)
    q, k, qo, ko = (x[:, :, i] for i in range(4))
    prm = nabla.rope_params_of((16,))
    keep = q.clone(), k.clone()
    want = nabla.rope(prm, *keep, grid=(N, 1, 1))
    nabla.rope(prm, q, k, grid=(N, 1, 1), q_out=qo, k_out=ko)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    assert torch.equal(q, keep[0]) and torch.equal(k, keep[1])


def test_packed_calls_between_the_heads_of_their_inputs():
    """Heads in front: [heads, 2, total, D], q beside o and dout beside dq."""
    heads, total, D = 4, 150, 64
    cu = torch.tensor([0, 70, total], dtype=torch.int32, device="cuda")
    first = lambda t: t.transpose(0, 1)  # [total, heads, D]
    new = lambda *s: torch.randn(*s, device="cuda").to(BF)
    qo, kv, dd, out = new(heads, 2, total, D), new(2, heads, total, D), new(heads, 2, total, D), new(heads, 2, total, D)
    q, k, v, dout = first(qo[:, 0]), first(kv[0]), first(kv[1]), first(dd[:, 0])
    o, lse = nabla.attn_packed_fwd(q.contiguous(), k, v, cu, cu, causal=True)
    want = nabla.attn_packed_bwd(q.contiguous(), k, v, o, dout.contiguous(), lse, cu, cu, causal=True)
    got, _ = nabla.attn_packed_fwd(q, k, v, cu, cu, causal=True, o=first(qo[:, 1]))
    assert torch.equal(got, o)
    got = nabla.attn_packed_bwd(q, k, v, o, dout, lse, cu, cu, causal=True, dq=first(dd[:, 1]),
                                dk=first(out[:, 0]), dv=first(out[:, 1]))
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_views_that_share_rows_are_still_refused():
    x = torch.randn(3, 1, 8, 64, device="cuda").to(BF)
    prm = nabla.rope_params_of((32,))
    q = x[:, :, :4].transpose(1, 2)
    pos = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    with pytest.raises(nabla.NablaError) as e:
        nabla.rope(prm, q, pos=pos, q_out=x[:, :, 2:6].transpose(1, 2))
    assert e.value.status == nabla.ERR_PARAM
    k = x[:, :, 4:].transpose(1, 2)
    with pytest.raises(nabla.NablaError) as e:
        nabla.rope(prm, q, k, pos=pos, q_out=k, k_out=q)
    assert e.value.status == nabla.ERR_PARAM
