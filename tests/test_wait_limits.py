"""How long the waits of the prompt attention's warps for one another may last: a second or so, by the constants (CPU),
and in proportion where a test withholds the tiles (GPU)."""
import os
import re
import time

import pytest
import torch

import nvfp4_paged_kv_02_gb300 as nv

CSRC = os.path.join(os.path.dirname(nv.__file__), "csrc")
STALLED_NAPS = 1 << 12  # the limit under NVFP4KV_TEST_STALL_PIPELINE


def _limits():
    with open(os.path.join(CSRC, "tcgen05.cuh")) as f:
        text = f.read()
    nap = int(re.search(r"kNap = (\d+);", text)[1])
    return nap * 1e-9, 1 << int(re.search(r"kNapLimit = 1u << (\d+);", text)[1])


def test_a_wait_lasts_a_second_or_so():
    nap, limit = _limits()
    assert nap * limit < 1.5 and limit > STALLED_NAPS
    with open(os.path.join(CSRC, "prefill.cu")) as f:
        text = f.read()
    assert "kWaitLimit" not in text and "mbar_wait(" not in text and "mbar_try_wait(" not in text
    assert re.search(r"wait_limit = std::min\(a\.pipe\.wait_limit, kNapLimit\)", text)


@pytest.mark.gpu
def test_a_stalled_call_comes_back_in_time(gpu_lib):
    from tests import decode_reference as R
    from tests.test_gpu_prefill import BF16, HND, _indptr, _query, _run
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    nap, _ = _limits()
    c = R.make_paged(1, [300, 700], 2, 128, 16, HND)
    q = _query(1, 320, 4, 128, BF16)
    _run(gpu_lib, c, q, _indptr([300, 20]))
    os.environ["NVFP4KV_TEST_STALL_PIPELINE"] = "1"
    try:
        t0 = time.perf_counter()
        _, _, status = _run(gpu_lib, c, q, _indptr([300, 20]))
        took = time.perf_counter() - t0
    finally:
        os.environ.pop("NVFP4KV_TEST_STALL_PIPELINE")
    assert status == gpu_lib.DEV_TIMEOUT
    # one wait runs out, and the others' last naps; the rest is the host's copies
    assert took < 2 * nap * STALLED_NAPS + 0.5, took
    print(f"stalled call: {took * 1e3:.1f} ms")
