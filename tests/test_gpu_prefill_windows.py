"""Attention of prompts with one query head to a KV head, where the window of a segment's first 128 rows begins with a
tile that the window of its other 128 rows has left, but for the first tokens."""
import pytest
import torch

from tests.test_gpu_prefill import BF16, F16, HND, NHD, _both

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(gpu_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sink", [1, 4, 129, 300])
@pytest.mark.parametrize("window", [0, 128, 256, 1024])
def test_windows_that_begin_with_a_tile(gpu_lib, window, sink, D, causal):
    """Whole prompts, and prompts after 384 positions that the cache holds already."""
    new, lens = ([1500], [1884]) if window == 1024 else ([600, 700], [600, 1084])
    _both(gpu_lib, window + sink, new, lens, 1, 1, D, 16, HND, BF16, window_left=window, num_sink_tokens=sink, causal=causal)


@pytest.mark.parametrize("D", [96, 80])
def test_other_heads(gpu_lib, D):
    _both(gpu_lib, D, [700], [700], 2, 1, D, 7, NHD, F16, window_left=256, num_sink_tokens=4)
    _both(gpu_lib, D, [1400], [1400], 1, 1, D, 16, NHD, BF16, window_left=1024, num_sink_tokens=130, logits_soft_cap=20.0)


def test_many_prompts(gpu_lib):
    """Several segments to a CTA, most of them not cut."""
    new = [600 + 5 * (i % 3) for i in range(64)]
    lens = [n + 128 * (i % 4) for i, n in enumerate(new)]
    _both(gpu_lib, 3, new, lens, 1, 1, 64, 16, HND, BF16, window_left=256, num_sink_tokens=4)
