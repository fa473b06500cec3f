"""Page bounds over NaN: the minimum and maximum of values with a NaN among them are NaN."""
import numpy as np
import pytest
import torch

from tests import decode_reference as R
from tests.test_gpu_select_pages import BOUNDS, RING, _bounds

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(gpu_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield


@pytest.mark.parametrize("lens,H,D,ps,layout,tdt", BOUNDS + RING)
def test_nan_scales_of_live_slots(gpu_lib, lens, H, D, ps, layout, tdt):
    c = R.make_paged(5, lens, H, D, ps, layout, table_dtype=tdt)
    rng = np.random.Generator(np.random.PCG64(5))
    for b in range(c.B):
        for t in {0, int(rng.integers(0, c.lens[b])), c.lens[b] - 1} if c.lens[b] else ():
            h, j = int(rng.integers(0, H)), int(rng.integers(0, D // 16))
            at = (t % ps, h, j) if layout == R.NHD else (h, t % ps, j)
            c.ks[(c.tables[b, t // ps], *at)] = rng.choice([0x7F, 0xFF])
    got = _bounds(gpu_lib, c)
    want = np.full(got.shape, 9.0)
    for p, (lo, hi) in R.key_bounds(c).items():
        want[p, :, 0], want[p, :, 1] = lo, hi
    assert np.isnan(want).any() and np.array_equal(got, want, equal_nan=True)
