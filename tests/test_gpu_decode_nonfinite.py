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


@pytest.mark.parametrize("name", SHAPES)
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_nan_and_infinite_queries_show(gpu_lib, name, value):
    """One query head of every second request: NaN, or an infinity (its scores are infinite or NaN, and
    the largest less itself is NaN), at every length."""
    c, q = _case(name)
    dev = _dev(c)
    want = _run(gpu_lib, c, q, dev)
    q2 = q.clone()
    hit = torch.zeros(q.shape[:2], dtype=torch.bool, device=DEV)
    for b in range(0, c.B, 2):
        if value == value and c.lens[b] < 32:
            continue  # (few keys: all of an infinite query's scores may be -inf)
        q2[b, b % q.shape[1], 5] = value
        hit[b, b % q.shape[1]] = True
    out, lse, _ = _run(gpu_lib, c, q2, dev)
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(out[~hit], want[0][~hit]) and torch.equal(lse[~hit], want[1][~hit])


def test_nan_queries_at_every_length(gpu_lib):
    for n in (1, 31, 300, 385, 3000, 100000):
        c = R.make_paged(n, [n], 1, 64, 16, R.NHD)
        q = _query(n, 1, G, 64, torch.bfloat16).to(DEV)
        q[0, 1] = float("nan")
        out, lse, _ = _run(gpu_lib, c, q)
        nan = torch.tensor([False, True, False, False], device=DEV)
        assert torch.equal(torch.isnan(lse[0]), nan), n
        assert torch.equal(torch.isnan(out[0]).all(-1), nan) and torch.equal(torch.isnan(out[0]).any(-1), nan), n


@pytest.mark.parametrize("name", SHAPES)
@pytest.mark.parametrize("which", ["k", "v"])
def test_nan_scales_show_where_they_are(gpu_lib, name, which):
    """A NaN block scale of a live key: every query head of its KV head. Of a live value: the block's 16
    elements of those heads' outputs, and no log-sum-exp."""
    c, q = _case(name)
    want = _run(gpu_lib, c, q)
    out_nan = torch.zeros((c.B, c.H * G, c.D), dtype=torch.bool, device=DEV)
    lse_nan = torch.zeros((c.B, c.H * G), dtype=torch.bool, device=DEV)
    rng = np.random.Generator(np.random.PCG64(1))
    for b in range(0, c.B, 2):
        h, t, j = (int(rng.integers(0, n)) for n in (c.H, c.lens[b], c.D // 16))
        (c.ks if which == "k" else c.vs)[c.tables[b, t // c.ps], h, t % c.ps, j] = 0x7F
        heads = slice(h * G, (h + 1) * G)
        if which == "k":
            out_nan[b, heads], lse_nan[b, heads] = True, True
        else:
            out_nan[b, heads, 16 * j: 16 * j + 16] = True
    out, lse, _ = _run(gpu_lib, c, q)
    assert torch.equal(torch.isnan(out), out_nan) and torch.equal(torch.isnan(lse), lse_nan)
    assert torch.equal(out[~out_nan], want[0][~out_nan]) and torch.equal(lse[~lse_nan], want[1][~lse_nan])
