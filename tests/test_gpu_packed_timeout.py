"""The packed calls when a device-side wait expires: the test flag withholds the
loads that the kernels wait for, each wait gives up after 1 ms, the status says
so, and the next call on the same workspace is right."""
import ctypes

import pytest
import torch

from adaptive_block_sparse_fractal_b200 import nabla

import seq_util

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
TIMEOUT = nabla.DEBUG_TIMEOUT

# lens_q, lens_k: few keys (their barriers in dK, dV), masked rows, many units,
# few rows on many keys (split forward)
CASES = [([200, 64], [32, 17]), ([300, 1, 140], [300, 1, 140]), ([700] * 20, [700] * 20), ([3], [9000]),
         ([64], [64])]


def view(t):
    return nabla.View(t.data_ptr(), 0, t.stride(1), t.stride(0))


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("D", [64, 128])
def test_an_expired_wait_is_reported_and_the_next_call_is_right(case, causal, D):
    lens_q, lens_k = CASES[case]
    hq, hk = 4, 2
    g = torch.Generator(device="cuda").manual_seed(case)
    borders = lambda lens: [sum(lens[:i]) for i in range(len(lens) + 1)]
    cq, ck = borders(lens_q), borders(lens_k)
    new = lambda n, h: torch.randn(n, h, D, generator=g, device="cuda").to(BF)
    q, k, v, dout = new(cq[-1], hq), new(ck[-1], hk), new(ck[-1], hk), new(cq[-1], hq)
    cu_q, cu_k = (torch.tensor(c, dtype=torch.int32, device="cuda") for c in (cq, ck))
    ws = nabla.packed_workspace(q, k, len(lens_q), back=True)
    o, lse = nabla.attn_packed_fwd(q, k, v, cu_q, cu_k, causal=causal, ws=ws)
    grads = nabla.attn_packed_bwd(q, k, v, o, dout, lse, cu_q, cu_k, causal=causal, ws=ws)
    assert nabla.status(ws) == nabla.OK

    shape = nabla.Packed(len(lens_q), hq, hk, D, cq[-1], ck[-1], causal | TIMEOUT, D ** -0.5)
    ref = lambda t: ctypes.byref(view(t))
    stream = torch.cuda.current_stream().cuda_stream
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    L = nabla.lib()
    assert L.nabla_attn_packed_fwd(ctypes.byref(shape), ref(q), ref(k), ref(v), cu_q.data_ptr(),
                                   cu_k.data_ptr(), ref(o2), lse2.data_ptr(), ws.data_ptr(), ws.numel(),
                                   stream) == nabla.OK
    assert nabla.status(ws) == nabla.ERR_TIMEOUT
    out = [torch.empty_like(t) for t in grads]
    assert L.nabla_attn_packed_bwd(ctypes.byref(shape), ref(q), ref(k), ref(v), ref(o), ref(dout),
                                   lse.data_ptr(), cu_q.data_ptr(), cu_k.data_ptr(), *(ref(t) for t in out),
                                   ws.data_ptr(), ws.numel(), stream) == nabla.OK
    assert nabla.status(ws) == nabla.ERR_TIMEOUT

    nabla.attn_packed_fwd(q, k, v, cu_q, cu_k, causal=causal, o=o2, lse=lse2, ws=ws)
    nabla.attn_packed_bwd(q, k, v, o2, dout, lse2, cu_q, cu_k, causal=causal, dq=out[0], dk=out[1],
                          dv=out[2], ws=ws)
    assert nabla.status(ws) == nabla.OK
    assert torch.equal(o2, o) and torch.equal(lse2, lse)
    for a, b in zip(out, grads):
        assert torch.equal(a, b)
    if case == 1:
        r = seq_util.packed(q, k, v, cq, ck, bool(causal), dout=dout)
        seq_util.check(o2, r["o"], r["o_tol"], "o")
        for n, t in zip(("dq", "dk", "dv"), out):
            seq_util.check(t, r[n], r[n + "_tol"], n)
