"""Two copies of the library in one process share no state."""
import ctypes
import os
import shutil
import subprocess
import tempfile

import pytest
import torch

from adaptive_block_sparse_fractal_b200 import build, nabla


def test_no_symbol_is_one_for_the_process():
    build.build()
    out = subprocess.run(["nm", "-C", nabla.LIB_PATH], check=True, capture_output=True, text=True).stdout
    unique = [line for line in out.splitlines() if " u " in line and "nabla" in line]
    assert unique == []


@pytest.mark.gpu
def test_both_launch():
    BF = torch.bfloat16
    q, k, v = (torch.randn(100, h, 128, device="cuda").to(BF) for h in (4, 2, 2))
    dout = torch.randn_like(q)
    cu = torch.tensor([0, 30, 100], dtype=torch.int32, device="cuda")
    kc, vc = (torch.randn(8, 16, 2, 128, device="cuda").to(BF) for _ in range(2))
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4).contiguous()
    lens = torch.tensor([50, 7], dtype=torch.int32, device="cuda")

    def run():
        o, lse = nabla.attn_packed_fwd(q, k, v, cu, cu, causal=True)
        return (o,) + nabla.attn_packed_bwd(q, k, v, o, dout, lse, cu, cu, causal=True) + nabla.attn_paged(
            q[:2].contiguous(), kc, vc, table, lens)
    want = run()
    first, path = nabla.lib(), nabla.LIB_PATH
    copy = os.path.join(tempfile.mkdtemp(), "libnabla_copy.so")
    shutil.copy(path, copy)
    try:
        nabla._lib, nabla.LIB_PATH = None, copy
        got = run()
        assert isinstance(nabla.lib(), ctypes.CDLL) and nabla.lib() is not first
    finally:
        nabla._lib, nabla.LIB_PATH = first, path
    for a, b in zip(got, want):
        assert torch.equal(a, b)
