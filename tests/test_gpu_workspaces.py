"""What the decode-step calls keep between calls: a bounded number of attention workspaces, by stream and
not by a stream's handle, and nothing of a selection."""
import threading

import numpy as np
import pytest
import torch

from tests import decode_reference as R
from tests.test_gpu_decode_attention import DEV, _dev, _query, _run
from tests.test_gpu_select_pages import _select_case, _t

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(gpu_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield


@pytest.fixture()
def call(gpu_lib):
    """A call whose list is cut and joined through the workspace, and its result."""
    c = R.make_paged(3, [3000, 700], 1, 64, 16, R.HND)
    q, dev = _query(3, 2, 4, 64, torch.float16).to(DEV), _dev(c)
    want = _run(gpu_lib, c, q, dev)

    def run():
        out, lse, _ = _run(gpu_lib, c, q, dev)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    return run


class Stream:
    def __init__(self):
        handle = torch.zeros(1, dtype=torch.int64)
        assert int(torch.cuda.cudart().cudaStreamCreate(handle.data_ptr())) == 0
        self.handle = int(handle)

    def run(self, call):
        with torch.cuda.stream(torch.cuda.ExternalStream(self.handle)):
            call()  # (ends with a synchronize)

    def destroy(self):
        torch.cuda.synchronize()
        assert int(torch.cuda.cudart().cudaStreamDestroy(self.handle)) == 0


def _kept(nv):
    return nv._calls().workspaces()


def test_streams_that_come_and_go(gpu_lib, call):
    call()
    for _ in range(150):
        s = Stream()
        s.run(call)
        s.destroy()
        assert len(_kept(gpu_lib)) <= 64
    call()


def test_a_stream_is_not_its_handle(gpu_lib, call):
    """A new stream under the handle of one that is gone does not get that one's workspace."""
    call()
    ids, again = {}, 0
    for _ in range(40):
        s = Stream()
        s.run(call)
        mine = _kept(gpu_lib)[0][1]
        assert mine not in ids.values()
        again += s.handle in ids
        ids[s.handle] = mine
        s.destroy()
    if not again:
        pytest.skip("no handle was given twice")


def test_the_per_thread_stream(gpu_lib, call):
    """cudaStreamPerThread is one handle, and another stream in each thread."""
    got = []

    def thread():
        with torch.cuda.stream(torch.cuda.ExternalStream(2)):
            call()
        got.append(_kept(gpu_lib)[0])
    for _ in range(2):
        t = threading.Thread(target=thread)
        t.start()
        t.join()
    assert len(got) == 2 and got[0][1:3] != got[1][1:3] and got[0][2] != 0


def test_many_streams_at_once(gpu_lib, call):
    """More streams than workspaces are kept, with calls in flight on all of them."""
    nv = gpu_lib
    c = R.make_paged(3, [3000, 700], 1, 64, 16, R.HND)
    q, (caches, sf) = _query(3, 2, 4, 64, torch.float16).to(DEV), _dev(c)
    gk, gv = (torch.tensor([x], dtype=torch.float32, device=DEV) for x in (c.gk, c.gv))
    tables, lens = _t(c.tables), _t(c.lens)
    run = lambda: nv.nvfp4_paged_attention_decode(q, caches, sf, tables, lens, gk, gv, "HND")
    want = run()
    streams = [Stream() for _ in range(100)]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for s in streams:
            with torch.cuda.stream(torch.cuda.ExternalStream(s.handle)):
                got.append(run())
        torch.cuda.synchronize()
        for out, lse in got:
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert len(_kept(nv)) == 64
    for s in streams:
        s.destroy()


def test_a_selection_keeps_nothing(gpu_lib):
    nv = gpu_lib
    lens, tables, bounds, q = _select_case(1, [400, 30], 2, 4, 64, 4, torch.float16)
    wide = np.full((2, 300_000), -1, np.int32)
    wide[:, :tables.shape[1]] = tables
    args = (q.to(DEV), _t(bounds), _t(tables), _t(lens), 4, 8)
    want = nv.nvfp4_select_pages(*args)
    wide_args = (*args[:2], _t(wide), *args[3:])
    before, held = _kept(nv), torch.cuda.memory_allocated()
    got = nv.nvfp4_select_pages(*wide_args)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    del got
    assert _kept(nv) == before and torch.cuda.memory_allocated() == held
