"""Attention of one new token over a sliding window and the first tokens, which stay visible, against the
64-bit reference; the slots that no position owns hold NaN scales."""
import numpy as np
import pytest
import torch

from tests import decode_reference as R
from tests import prompt_reference as PR
from tests.test_gpu_decode_attention import DEV, _dev, _query, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(gpu_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield


def _ref(c, q, **kw):
    return PR.attention(PR.with_f32_scales(c), q.double().numpy(), np.arange(c.B + 1), q.shape[-1] ** -0.5, **kw)


CASES = [
    # lens, H, G, D, ps, layout, dtype, window, sink
    ([1, 2, 0, 5], 1, 2, 64, 16, R.HND, torch.float16, 0, 1),
    ([300, 31, 77, 200], 2, 4, 128, 16, R.NHD, torch.bfloat16, 20, 4),
    ([300, 301, 330, 64], 2, 1, 128, 16, R.HND, torch.float16, 33, 32),
    ([300, 96, 97], 1, 7, 64, 12, R.NHD, torch.bfloat16, 31, 33),      # sinks that end in the window's unit
    ([500, 100], 2, 3, 96, 7, R.HND, torch.float16, 100, 399),         # and at the window's first token
    ([500, 100], 2, 3, 96, 7, R.HND, torch.float16, 100, 400),
    ([129, 700], 1, 16, 128, 64, R.NHD, torch.float16, 64, 1000000),   # more of them than tokens
    ([3000, 1], 2, 9, 256, 16, R.HND, torch.bfloat16, 700, 100),
    ([5000, 5001, 800], 1, 4, 128, 16, R.HND, torch.float16, 2047, 16),
    ([6000], 4, 2, 64, 32, R.NHD, torch.bfloat16, 1, 2),
    ([4000] * 40, 3, 2, 64, 16, R.HND, torch.float16, 500, 65),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_matches_reference(gpu_lib, i):
    lens, H, G, D, ps, layout, dtype, window, sink = CASES[i]
    c = R.make_paged(i, lens, H, D, ps, layout)
    q = _query(i, c.B, H * G, D, dtype)
    out, lse, status = _run(gpu_lib, c, q, window_left=window, num_sink_tokens=sink)
    PR.check(out, lse, _ref(c, q, window=window, sink=sink), dtype)
    assert status == 0


def test_without_effect(gpu_lib):
    """No window: every position is live already. No first tokens: the window alone, to the last bit."""
    c = R.make_paged(3, [700, 64, 0], 2, 128, 16, R.HND)
    q = _query(3, c.B, 8, 128, torch.bfloat16)
    dev = _dev(c)
    for kw in (dict(), dict(window_left=100)):
        want = _run(gpu_lib, c, q, dev, **kw)
        got = _run(gpu_lib, c, q, dev, num_sink_tokens=0 if kw else 50, **kw)
        assert all(torch.equal(x, y) for x, y in zip(want[:2], got[:2]))


def test_nan_between_the_first_tokens_and_the_window(gpu_lib):
    """What is not live does not show, not even a NaN; a first token's does."""
    c = R.make_paged(5, [400, 400], 1, 64, 16, R.HND)
    for p in range(2, 6):  # positions 32 .. 96 of both requests, NaN
        for s in (c.ks, c.vs):
            s[c.tables[:, p]] = 0x7F
    c.vs[c.tables[1, 0], 0, 3] = 0x7F
    q = _query(5, 2, 4, 64, torch.float16)
    kw = dict(window_left=300, num_sink_tokens=17)
    out, lse, _ = _run(gpu_lib, c, q, **kw)
    PR.check(out, lse, _ref(c, q, window=300, sink=17), q.dtype)
    assert not torch.isnan(out[0]).any() and torch.isnan(out[1]).all() and not torch.isnan(lse).any()


def test_pages_outside_the_pool(gpu_lib):
    c = R.make_paged(6, [400], 1, 64, 16, R.NHD)
    for j, bad in ((0, 10 ** 6), (1, -5), (6, 99999)):  # of the first tokens, and (6) of none that is live
        c.tables[0, j] = bad
    q = _query(6, 1, 4, 64, torch.float16)
    kw = dict(window_left=200, num_sink_tokens=40)
    out, lse, status = _run(gpu_lib, c, q, **kw)
    PR.check(out, lse, _ref(c, q, window=200, sink=40), q.dtype)
    assert status == gpu_lib.DEV_BAD_PAGE


def test_captured_and_replayed(gpu_lib):
    c = R.make_paged(7, [1500, 900], 2, 128, 16, R.HND)
    q = _query(7, 2, 8, 128, torch.bfloat16).to(DEV)
    caches, sf = _dev(c)
    lens = torch.as_tensor(c.lens).to(DEV)
    table = torch.as_tensor(c.tables).to(DEV)
    gk, gv = (torch.tensor([x], device=DEV) for x in (c.gk, c.gv))
    kw = dict(window_left=300, num_sink_tokens=10)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = gpu_lib.nvfp4_paged_attention_decode(q, caches, sf, table, lens, gk, gv, "HND", **kw)
    for now in ([1500, 900], [1, 305], [311, 0]):
        lens.copy_(torch.tensor(now))
        graph.replay()
        torch.cuda.synchronize()
        short = R.Paged(**{**c.__dict__, "lens": np.array(now, np.int32)})
        PR.check(out, lse, _ref(short, q.cpu(), window=300, sink=10), q.dtype)
