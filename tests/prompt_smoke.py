"""One small call of each operator of prompts, windows and axes against the references (used by the smoke run)."""
import numpy as np
import torch

from tests import decode_reference as R
from tests import prompt_reference as PR
from tests.test_gpu_decode_attention import _query
from tests.test_gpu_decode_attention import _run as decode
from tests.test_gpu_norm_rope import _same
from tests.test_gpu_prefill import _indptr, _ref, _run
from tests.test_gpu_rotary_axes import AxesCase


def run(nv) -> None:
    # positions of three axes: query rows and cache bytes equal
    case = AxesCase(2, 24, 8, 2, 64, 16, R.HND, torch.bfloat16, 64, axes=3)
    _same(case, *case.call(nv), case.expect())
    c = R.make_paged(1, [37, 300, 0, 1500], 2, 64, 16, R.HND)
    kw = dict(window_left=100, num_sink_tokens=4)
    # prompts and chunks (rows of 128), and drafts (few rows)
    for new in ([37, 130, 0, 60], [2, 4, 0, 1]):
        q = _query(1, sum(new), 4, 64, torch.bfloat16)
        out, lse, status = _run(nv, c, q, _indptr(new), **kw)
        PR.check(out, lse, _ref(c, q, _indptr(new), **kw), q.dtype)
        if status:
            raise AssertionError(f"smoke: status {status}")
    # one token over a window and the first tokens
    q = _query(2, c.B, 4, 64, torch.bfloat16)
    out, lse, _ = decode(nv, c, q, **kw)
    PR.check(out, lse, _ref(c, q, np.arange(c.B + 1), **kw), q.dtype)
