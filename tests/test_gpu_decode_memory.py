"""A decode-step call that torch's allocator refuses raises what torch raises, and the next call works."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(gpu_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield


def test_out_of_memory(gpu_lib):
    """Outputs of 2^45 bytes are refused before any memory is taken."""
    dev = dict(device="cuda")
    B, H = 64, 64
    q = torch.zeros((B, H, 64), dtype=torch.float16, **dev)
    bounds = torch.zeros((4, H, 2, 64), dtype=torch.float16, **dev)
    tables, lens = torch.zeros((B, 2), dtype=torch.int32, **dev), torch.full((B,), 20, dtype=torch.int32, **dev)
    call = lambda k: gpu_lib.nvfp4_select_pages(q, bounds, tables, lens, 16, k)
    held = torch.cuda.memory_allocated()
    with pytest.raises(torch.OutOfMemoryError):
        call(2 ** 31 - 1)
    assert torch.cuda.memory_allocated() == held
    selected, count = call(2)
    assert (count == 2).all() and (selected == torch.tensor([0, 1], dtype=torch.int32, **dev)).all()
