"""The decode-step operators together: the example's captured steps, the dense call against
dequantize plus 64-bit attention, and a stalled copy ring of the page bounds."""
import os
import sys

import numpy as np
import pytest
import torch

from tests import decode_reference as R

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _cuda(gpu_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import sparse_decode
        yield sparse_decode
    finally:
        sys.path.remove(os.path.join(ROOT, "examples"))


def test_example_runs_and_covers_what_it_selects(example):
    near, mass, status = example.main(["--batch", "3", "--prompt", "1000", "--steps", "5", "--pages", "24"])
    assert status == 0 and 0.0 < mass <= 1.0 + 1e-3 and near > 0.3
    # selecting every page is dense attention
    near, mass, status = example.main(["--batch", "2", "--prompt", "300", "--steps", "3", "--pages", "40"])
    assert status == 0 and abs(mass - 1.0) < 1e-3 and near > 0.9999


def test_steps_build_the_cache_that_one_call_builds(example):
    """Rows appended token by token and rows appended as a prompt give the same cache and bounds."""
    a, b = example.Layer(2, 64, seed=5), example.Layer(2, 64, seed=5)
    qkv = a.project(2 * 50)
    req = torch.arange(2, device="cuda", dtype=torch.int32)
    pos = torch.arange(50, device="cuda", dtype=torch.int32)
    qa = a.append(qkv, req.repeat_interleave(50), pos.repeat(2))
    a.lens.fill_(50)
    a.renew_bounds(None)
    for t in range(50):
        q = b.append(qkv[t::50].contiguous(), req, pos[t:t + 1].repeat(2))
        b.lens.fill_(t + 1)
        b.renew_bounds(pos[t:t + 1].repeat(2))
        assert torch.equal(q, qa[t::50])
    for x, y in zip(a.codes + a.scales + [a.bounds], b.codes + b.scales + [b.bounds]):
        assert torch.equal(x, y)
    assert int(a.status) == int(b.status) == 0


def test_attention_of_what_dequantize_gives(gpu_lib):
    """Dense attention against attention over nvfp4_dequantize_paged's output, in 64 bits."""
    nv = gpu_lib
    c = R.make_paged(70, [300, 47, 1], 2, 128, 16, R.HND)
    t = lambda x: torch.as_tensor(x).cuda()
    caches, sf = (t(c.k), t(c.v)), (t(c.ks), t(c.vs))
    g = [torch.tensor([x], dtype=torch.float32, device="cuda") for x in (c.gk, c.gv)]
    out = [torch.zeros((3, 300, 2, 128), dtype=torch.float16, device="cuda") for _ in range(2)]
    nv.nvfp4_dequantize_paged(caches, sf, t(c.tables), t(c.lens), *g, *out, "HND")
    q = torch.randn((3, 8, 128), generator=torch.Generator().manual_seed(70)).half()
    got, lse = nv.nvfp4_paged_attention_decode(q.cuda(), caches, sf, t(c.tables), t(c.lens), *g, "HND", sm_scale=0.1)
    k, v = (o.double().cpu() for o in out)
    for b, n in enumerate(c.lens):
        for h in range(2):
            x = q[b, 4 * h:4 * h + 4].double() @ k[b, :n, h].T * 0.1
            want = torch.softmax(x, -1) @ v[b, :n, h]
            # the dequantized rows are rounded to binary16: 2^-11 of each key and value
            slack = 2.0 ** -11 * 0.1 * (q[b, 4 * h:4 * h + 4].double().abs() @ k[b, :n, h].abs().T).max() * 2
            size = torch.softmax(x, -1) @ v[b, :n, h].abs()
            tol = (slack + 3 * 2.0 ** -11) * size + 2.0 ** -24
            assert ((got[b, 4 * h:4 * h + 4].double().cpu() - want).abs() <= tol).all()


def test_stalled_bounds_ring_reports_timeout_and_recovers(gpu_lib):
    nv = gpu_lib
    c = R.make_paged(71, [500, 40], 8, 128, 16, R.HND)
    t = lambda x: torch.as_tensor(x).cuda()
    args = (t(c.k), t(c.ks), t(c.tables), t(c.lens))
    out = torch.zeros((c.k.shape[0], 8, 2, 128), dtype=torch.float16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    os.environ["NVFP4KV_TEST_STALL_PIPELINE"] = "1"
    try:
        nv.nvfp4_page_key_bounds(*args, out, None, "HND", dev_status=st)
        torch.cuda.synchronize()
    finally:
        os.environ.pop("NVFP4KV_TEST_STALL_PIPELINE", None)
    assert int(st.item()) == nv.DEV_TIMEOUT
    st.zero_()
    nv.nvfp4_page_key_bounds(*args, out, None, "HND", dev_status=st)
    got = out.double().cpu().numpy()
    assert int(st.item()) == 0
    for p, (lo, hi) in R.key_bounds(c).items():
        assert np.array_equal(got[p, :, 0], lo) and np.array_equal(got[p, :, 1], hi)
