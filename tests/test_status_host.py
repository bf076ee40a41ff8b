"""status() of something that is no workspace on a GPU (CPU)."""
import pytest
import torch

from adaptive_block_sparse_fractal_b200 import nabla


def test_status_of_host_memory_is_refused():
    with pytest.raises(ValueError):
        nabla.status(torch.zeros(256, dtype=torch.uint8))
