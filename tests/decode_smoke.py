"""One small call of each decode-step operator against the references (used by the smoke run)."""
import numpy as np
import torch

from tests import decode_reference as R
from tests.test_gpu_decode_attention import _dev, _query, _ref, _run
from tests.test_gpu_norm_rope import Case, _same
from tests.test_gpu_select_pages import _bounds, _check_select


def run(nv) -> None:
    # norm, rotation and append: query rows and cache bytes equal
    case = Case(2, 24, 8, 2, 64, 16, R.HND, torch.bfloat16, 64)
    _same(case, *case.call(nv), case.expect())
    # bounds and selection equal
    c = R.make_paged(1, [37, 100, 0, 1500], 2, 64, 16, R.HND)
    bounds = _bounds(nv, c)
    want = np.full(bounds.shape, 9.0)
    for p, (lo, hi) in R.key_bounds(c).items():
        want[p, :, 0], want[p, :, 1] = lo, hi
    if not np.array_equal(bounds, want):
        raise AssertionError("smoke: page bounds differ from the reference")
    q = _query(1, c.B, 8, 64, torch.bfloat16)
    small = bounds.astype(np.float16)
    small[want[:, 0, 0, 0] == 9.0] = 0  # (pages of no request)
    _check_select(nv, (c.lens, c.tables, small, q), 16, 8, 1, 1)
    # attention over all pages and over every second one
    R.check_attention(*_run(nv, c, q)[:2], _ref(c, q), q.dtype)
    pages = -(-c.lens // 16)
    sel, num = np.full((c.B, 2, 64), -1, np.int32), np.repeat((pages + 1) // 2, 2).astype(np.int32).reshape(-1, 2)
    for b, n in enumerate(pages):
        sel[b, :, :(n + 1) // 2] = np.arange(0, n, 2)
    out, lse, status = _run(nv, c, q, selected=sel, num_selected=num)
    R.check_attention(out, lse, _ref(c, q, selected=sel, num_selected=num), q.dtype)
    if status:
        raise AssertionError(f"smoke: status {status}")
