"""Attention of few new tokens where the tables reach more positions than the kernel of single tokens counts."""
import numpy as np
import pytest
import torch

from tests.test_gpu_prefill import F16, HND, _both

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("width", [1, 511, 512])
def test_tables_of_the_largest_batch(gpu_lib, width):
    """16,384 requests of up to `width` pages of 2^20 positions; three of them have any."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    new, lens = np.zeros(16384, int), np.zeros(16384, int)
    for b, n, length in ((0, 3, 700), (9000, 1, 1), (16383, 4, 33)):
        new[b], lens[b] = n, length
    _both(gpu_lib, width, new.tolist(), lens.tolist(), 1, 2, 16, 2 ** 20, HND, F16, width=width)
