"""Attention with NaN and infinities in what is read: they show where the formula has them, however the
request's list is cut and joined, and nowhere else."""
import numpy as np
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


# a list is 32 tokens a unit; up to 384 tokens are never cut
SHAPES = {
    "whole": ([300, 1, 384, 31, 64, 200], 2, 64),
    "few parts": ([3000 - 61 * i for i in range(32)], 8, 64),         # two or three runs to a list
    "few parts, 128": ([2600 - 47 * i for i in range(24)], 8, 128),
    "mixed": ([1, 2900, 300, 700, 40, 2000, 384, 385] * 6, 8, 64),    # cut and whole ones in one run
    "many parts": ([3000, 20000, 9000], 1, 64),                       # runs of four units
    "odd head size": ([2500 - 77 * i for i in range(20)], 6, 96),
}
G = 4


def _case(name):
    lens, H, D = SHAPES[name]
    c = R.make_paged(len(name), lens, H, D, 16, R.HND)
    return c, _query(len(name), c.B, H * G, D, torch.float16).to(DEV)


@pytest.mark.parametrize("name", SHAPES)
@pytest.mark.parametrize("step", [2, 3])
def test_nan_in_queries_stays_in_its_request(gpu_lib, name, step):
    c, q = _case(name)
    dev = _dev(c)
    want = _run(gpu_lib, c, q, dev)
    bad = torch.arange(c.B, device=DEV) % step == step - 1
    q2 = q.clone()
    q2[bad] = float("nan")
    for _ in range(5):  # which run joins a list is a matter of timing
        out, lse, _ = _run(gpu_lib, c, q2, dev)
        assert torch.equal(out[~bad], want[0][~bad]) and torch.equal(lse[~bad], want[1][~bad])


@pytest.mark.parametrize("D", [64, 128])
def test_nan_in_the_last_list_of_a_run_that_joins_another(gpu_lib, D):
    """Runs of 60 units and three runs to a multiprocessor: a list of 85 units is cut into 40 and 45, and the
    second part, which comes last, is of a run that goes on to six units of a list with NaN queries."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    units = [50] + [12, 85, 56] * sms
    c = R.make_paged(1, [32 * n for n in units[:-1]], 1, D, 16, R.HND)
    q = _query(1, c.B, G, D, torch.bfloat16).to(DEV)
    dev = _dev(c)
    want = _run(gpu_lib, c, q, dev)
    bad = torch.as_tensor(np.array(units[:-1]) == 56).to(DEV)
    q[bad] = float("nan")
    for _ in range(5):
        out, lse, _ = _run(gpu_lib, c, q, dev)
        assert torch.equal(out[~bad], want[0][~bad]) and torch.equal(lse[~bad], want[1][~bad])
