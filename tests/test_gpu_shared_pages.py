"""Requests whose tables share a prompt's full pages: their bounds and their attention."""
import numpy as np
import pytest
import torch

from tests import decode_reference as R
from tests.test_gpu_decode_attention import _query, _ref, _run
from tests.test_gpu_select_pages import _bounds

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(gpu_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield


@pytest.mark.parametrize("layout", [R.NHD, R.HND])
@pytest.mark.parametrize("ps,D", [(16, 128), (12, 96), (32, 64)])
def test_a_common_prompt(gpu_lib, layout, ps, D):
    common = 5
    lens = [common * ps, common * ps + 1, 9 * ps - 1, 7 * ps, common * ps + 3, common * ps]
    c = R.make_paged(3, lens, 2, D, ps, layout)
    c.tables[1:, :common] = c.tables[0, :common]
    want = np.full((c.k.shape[0], 2, 2, D), 9.0)
    for p, (lo, hi) in R.key_bounds(c).items():
        want[p, :, 0], want[p, :, 1] = lo, hi
    for _ in range(3):
        assert np.array_equal(_bounds(gpu_lib, c), want)
    q = _query(3, len(lens), 8, D, torch.float16)
    out, lse, status = _run(gpu_lib, c, q)
    R.check_attention(out, lse, _ref(c, q), q.dtype)
    assert status == 0
