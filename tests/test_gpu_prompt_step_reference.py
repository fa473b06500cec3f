"""A layer's prompts in chunks, in one call, and its captured steps and drafts, each against the 64-bit reference over the
cache as it is, with the bounds of the roundings (tests/prompt_reference.py)."""
import os
import sys

import numpy as np
import pytest
import torch

from tests import decode_reference as R
from tests import prompt_reference as PR

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(gpu_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import windowed_prompts
        yield windowed_prompts
    finally:
        sys.path.remove(os.path.join(ROOT, "examples"))


def _check(layer, q, indptr, out, lse):
    c = R.Paged(layer.B, layer.H, layer.D, layer.ps, R.HND, layer.lens.cpu().numpy(), layer.tables.cpu().numpy(),
                *(x.cpu().numpy() for pair in zip(layer.codes, layer.scales) for x in pair), layer.gk.item(), layer.gv.item())
    ref = PR.attention(c, q.double().cpu().numpy(), indptr, layer.D ** -0.5, window=layer.seen["window_left"],
                       sink=layer.seen["num_sink_tokens"])
    PR.check(out, lse, ref, torch.bfloat16)


@pytest.mark.parametrize("window,sink,group", [(99, 5, 4), (128, 4, 1), (-1, 0, 2)])
def test_chunks_steps_and_drafts(example, window, sink, group):
    B, n, steps = 2, 390, 4
    layer = example.Layer(B, n + steps, window, sink, heads=2, group=group, seed=9)
    req = torch.arange(B, device="cuda", dtype=torch.int32)

    def part(lo, hi):
        k = hi - lo
        q = layer.append(layer.project(B * k), req.repeat_interleave(k), torch.arange(lo, hi, device="cuda", dtype=torch.int32).repeat(B),
                         example.axis_positions(lo, k, 60).repeat(1, B).contiguous())
        layer.lens.fill_(hi)
        return q

    rows = []
    for lo, hi in ((0, 1), (1, 79), (79, n)):
        q = part(lo, hi)
        rows.append(q.view(B, hi - lo, *q.shape[1:]))
        ptr = np.arange(B + 1, dtype=np.int32) * (hi - lo)
        _check(layer, q, ptr, *layer.prompt(q, torch.as_tensor(ptr).cuda()))
    q = torch.cat(rows, 1).flatten(0, 1)  # the whole prompt once more, in one call
    ptr = np.arange(B + 1, dtype=np.int32) * n
    _check(layer, q, ptr, *layer.prompt(q, torch.as_tensor(ptr).cuda()))
    drafts = []
    one = np.arange(B + 1, dtype=np.int32)
    for i in range(steps):
        q = part(n + i, n + i + 1)
        drafts.append(q)
        _check(layer, q, one, *layer.step(q))
    q = torch.stack(drafts, 1).flatten(0, 1)
    _check(layer, q, one * steps, *layer.prompt(q, torch.as_tensor(one * steps).cuda()))
    assert int(layer.status) == 0
