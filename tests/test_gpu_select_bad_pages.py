"""Pages outside the pool come last in a selection, the first and last pages of a request among them."""
import pytest
import torch

from tests.test_gpu_select_pages import DEV, _select_case, _t

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(gpu_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield


@pytest.mark.parametrize("G", [4, 8, 20])
@pytest.mark.parametrize("bad", [[0], [99], [0, 1, 98, 99], list(range(0, 100, 2))])
def test_forced_pages_outside_the_pool(gpu_lib, G, bad):
    nv = gpu_lib
    lens, tables, bounds, q = _select_case(83, [400], 1, G, 64, 4, torch.float16)
    tables[0, bad] = [10 ** 8 if j % 3 else -1 for j in bad]
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    good = [j for j in range(100) if j not in bad]
    k = len(good)  # all that there are; one more takes the first page outside
    call = lambda k: nv.nvfp4_select_pages(q.to(DEV), _t(bounds), _t(tables), _t(lens), 4, k, num_sink_pages=2,
                                           num_recent_pages=3, dev_status=st)
    sel, num = call(k)
    assert sel[0, 0].tolist() == good and num.item() == k
    assert int(st.item()) == nv.DEV_BAD_PAGE
    if len(bad) > 1:
        sel, num = call(k + 1)
        assert sel[0, 0].tolist() == sorted(good + bad[:1]) and num.item() == k + 1
    sel, _ = call(6)  # the forced pages that are in the pool are still among the first
    assert {j for j in (0, 1, 97, 98, 99) if j not in bad} <= set(sel[0, 0].tolist()) <= set(good)
