"""What the decode-step calls keep between calls: nothing of a selection."""
import numpy as np
import pytest
import torch

from tests.test_gpu_decode_attention import DEV
from tests.test_gpu_select_pages import _select_case, _t

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(gpu_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield


def test_a_selection_keeps_nothing(gpu_lib):
    nv = gpu_lib
    lens, tables, bounds, q = _select_case(1, [400, 30], 2, 4, 64, 4, torch.float16)
    wide = np.full((2, 300_000), -1, np.int32)
    wide[:, :tables.shape[1]] = tables
    args = (q.to(DEV), _t(bounds), _t(tables), _t(lens), 4, 8)
    want = nv.nvfp4_select_pages(*args)
    wide_args = (*args[:2], _t(wide), *args[3:])
    held = torch.cuda.memory_allocated()
    got = nv.nvfp4_select_pages(*wide_args)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    del got
    assert torch.cuda.memory_allocated() == held
