"""The workspaces that are kept between calls are bounded by their bytes too: those of prompts are four to eight times the
decode calls'."""
import pytest
import torch

from tests import decode_reference as R
from tests.test_gpu_prefill import BF16, HND, _args, _indptr, _query
from tests.test_gpu_workspaces import Stream, _kept

pytestmark = pytest.mark.gpu
MOST = 656 << 20


def test_prompts_on_many_streams(gpu_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    nv = gpu_lib
    c = R.make_paged(1, [3000, 700], 1, 128, 16, HND)   # few rows over a long cache: its list is cut and joined
    q = _query(1, 12, 4, 128, BF16)
    args = _args(c, q, _indptr([8, 4]))
    want = nv.nvfp4_paged_attention_prefill(*args)
    one = _kept(nv)[0][3]
    streams = [Stream() for _ in range(40)]
    torch.cuda.synchronize()
    for _ in range(2):
        got = []
        for s in streams:
            with torch.cuda.stream(torch.cuda.ExternalStream(s.handle)):
                got.append(nv.nvfp4_paged_attention_prefill(*args))
            assert sum(k[3] for k in _kept(nv)) <= MOST and _kept(nv)[0][3] == one
        torch.cuda.synchronize()
        for out, lse in got:
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert len(_kept(nv)) == MOST // one == 16
    # the decode calls' are small: 64 of them as before
    a = (*args[:3], *args[4:])
    q2 = args[0][:2].contiguous()
    want = nv.nvfp4_paged_attention_decode(q2, *a[1:])
    for s in streams:
        with torch.cuda.stream(torch.cuda.ExternalStream(s.handle)):
            out, lse = nv.nvfp4_paged_attention_decode(q2, *a[1:])
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert sum(k[3] for k in _kept(nv)) <= MOST
    more = [Stream() for _ in range(70)]
    for s in more:
        with torch.cuda.stream(torch.cuda.ExternalStream(s.handle)):
            nv.nvfp4_paged_attention_decode(q2, *a[1:])
    torch.cuda.synchronize()
    assert len(_kept(nv)) == 64
    for s in streams + more:
        s.destroy()
