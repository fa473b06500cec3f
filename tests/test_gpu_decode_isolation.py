"""A query head's result does not depend on the other heads' queries, nor on those of other requests."""
import pytest
import torch

from tests import decode_reference as R
from tests.test_gpu_decode_attention import DEV, _dev, _query, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(gpu_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield


@pytest.mark.parametrize("lens,H,G,D", [([300, 1, 31], 2, 4, 64), ([3000 - 61 * i for i in range(32)], 8, 4, 64),
                                        ([5000, 700], 1, 16, 128), ([1000, 2100], 2, 12, 256)])
@pytest.mark.parametrize("factor", [30.0, 0.0, -1.0])
def test_one_head_changed(gpu_lib, lens, H, G, D, factor):
    c = R.make_paged(17, lens, H, D, 16, R.HND)
    q = _query(17, c.B, H * G, D, torch.float16).to(DEV)
    dev = _dev(c)
    want = _run(gpu_lib, c, q, dev)
    hit = torch.zeros(q.shape[:2], dtype=torch.bool, device=DEV)
    for b in range(0, c.B, 2):
        hit[b, 3 * b % q.shape[1]] = True
    q[hit] *= factor
    out, lse, _ = _run(gpu_lib, c, q, dev)
    assert torch.equal(out[~hit], want[0][~hit]) and torch.equal(lse[~hit], want[1][~hit])
    assert not torch.equal(out[hit], want[0][hit])
