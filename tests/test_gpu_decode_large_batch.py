"""The largest batch that the decode-step calls accept, for every width of the attention kernel."""
import numpy as np
import pytest
import torch

from tests import decode_reference as R
from tests.test_gpu_decode_attention import DEV, _dev, _query, _ref, _run

pytestmark = pytest.mark.gpu
MOST = 16384


@pytest.fixture(scope="module", autouse=True)
def _cuda(gpu_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("long", [False, True])
def test_attention_of_the_largest_batch(gpu_lib, D, long):
    """Requests of no or one token, a few longer ones among them; dense, and every page selected."""
    lens = np.arange(MOST) % 2
    lens[[5, 4000, 4001, 11111, MOST - 1]] = [70, 31, 500, 2000, 900] if long else 1
    c = R.make_paged(D, lens, 1, D, 16, R.HND, table_dtype=np.int32)
    q = _query(D, MOST, 2, D, torch.float16)
    ref = _ref(c, q)
    out, lse, status = _run(gpu_lib, c, q)
    R.check_attention(out, lse, ref, q.dtype)
    S = c.tables.shape[1]
    sel = np.broadcast_to(np.arange(S, dtype=np.int32), (MOST, 1, S)).copy()
    num = (-(-lens // 16)).astype(np.int32)[:, None]
    out, lse, sparse_status = _run(gpu_lib, c, q, selected=sel, num_selected=num)
    R.check_attention(out, lse, ref, q.dtype)
    assert status == 0 and sparse_status == 0


def test_bounds_of_the_largest_batch_in_the_largest_pages(gpu_lib):
    """Pages of 80,640 bytes: two of them and the scan of 16,384 requests fill a CTA's shared memory."""
    lens = np.zeros(MOST, np.int32)
    lens[[0, 77, MOST - 1]] = [75, 1, 140]
    c = R.make_paged(1, lens, 16, 128, 70, R.HND)
    got = torch.full((c.k.shape[0], 16, 2, 128), 9.0, dtype=torch.float16, device=DEV)
    t = lambda a: torch.as_tensor(a).to(DEV)
    gpu_lib.nvfp4_page_key_bounds(t(c.k), t(c.ks), t(c.tables), t(c.lens), got, None, "HND")
    want = np.full(got.shape, 9.0)
    for p, (lo, hi) in R.key_bounds(c).items():
        want[p, :, 0], want[p, :, 1] = lo, hi
    assert np.array_equal(got.double().cpu().numpy(), want)
