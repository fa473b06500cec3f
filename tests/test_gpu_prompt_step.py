"""The operators of prompts, windows and axes together: the example's chunks, captured steps and drafts; chunks
against one call; attention against what dequantize gives."""
import os
import sys

import numpy as np
import pytest
import torch

from tests import prompt_smoke

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
        import windowed_prompts
        yield windowed_prompts
    finally:
        sys.path.remove(os.path.join(ROOT, "examples"))


@pytest.mark.parametrize("args", [["--batch", "3", "--prompt", "700", "--chunk", "300", "--steps", "5", "--window", "255"],
                                  ["--batch", "1", "--prompt", "2100", "--chunk", "2100", "--steps", "3", "--sink", "0"]])
def test_example_verifies_its_steps(example, args):
    """Two ways to the same attention: weights rounded to binary16 (2^-11 of the magnitudes, which outputs bound
    from below), outputs to bf16 (half a step of 2^-8 each)."""
    apart, lse_apart, size, status = example.main(args)
    assert status == 0
    assert apart <= size * 2 * 2.0 ** -8 + 0.02 * size and lse_apart <= 1e-4


def test_chunks_give_what_one_call_gives(example):
    """Rows of a prompt in chunks of 1, 77 and the rest, and in one call: the same cache, the same attention."""
    one, many = example.Layer(2, 400, 99, 5, seed=5), example.Layer(2, 400, 99, 5, seed=5)
    n = 333
    qkv = one.project(2 * n).view(2, n, -1, one.D)
    req = torch.arange(2, device="cuda", dtype=torch.int32)

    def part(layer, lo, hi):
        k = hi - lo
        q = layer.append(qkv[:, lo:hi].flatten(0, 1).contiguous(), req.repeat_interleave(k),
                         torch.arange(lo, hi, device="cuda", dtype=torch.int32).repeat(2),
                         example.axis_positions(lo, k, 60).repeat(1, 2).contiguous())
        layer.lens.fill_(hi)
        out, lse = layer.prompt(q, (torch.arange(3, device="cuda") * k).int())
        return [t.view(2, k, *t.shape[1:]) for t in (q, out, lse)]

    whole = part(one, 0, n)
    parts = [torch.cat(t, 1) for t in zip(*(part(many, lo, hi) for lo, hi in ((0, 1), (1, 78), (78, n))))]
    assert torch.equal(whole[0], parts[0])
    for x, y in zip(one.codes + one.scales, many.codes + many.scales):
        assert torch.equal(x, y)
    size = whole[1].float().abs().max().item()
    assert (whole[1].float() - parts[1].float()).abs().max().item() <= size * (2.0 ** -7 + 0.02)
    assert (whole[2] - parts[2]).abs().max().item() <= 1e-4
    assert int(one.status) == int(many.status) == 0


def test_attention_of_what_dequantize_gives(gpu_lib, example):
    """Prefill attention against plain attention over the rows that nvfp4_dequantize_paged writes."""
    layer = example.Layer(2, 300, -1, 0, seed=6)
    n = 200
    req = torch.arange(2, device="cuda", dtype=torch.int32)
    q = layer.append(layer.project(2 * n), req.repeat_interleave(n), torch.arange(n, device="cuda", dtype=torch.int32).repeat(2),
                     example.axis_positions(0, n, 50).repeat(1, 2).contiguous())
    layer.lens.fill_(n)
    out, lse = layer.prompt(q, torch.tensor([0, n, 2 * n], device="cuda", dtype=torch.int32))
    rows = [torch.zeros((2, n, layer.H, layer.D), dtype=torch.float16, device="cuda") for _ in range(2)]
    gpu_lib.nvfp4_dequantize_paged(layer.codes, layer.scales, layer.tables, layer.lens, layer.gk, layer.gv, *rows, "HND")
    k, v = (x.double().repeat_interleave(layer.G, 2).transpose(1, 2) for x in rows)  # [2, Hq, n, D]
    x = q.view(2, n, -1, layer.D).double().transpose(1, 2) @ k.transpose(-1, -2) * layer.D ** -0.5
    x = x.masked_fill(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), -torch.inf)
    want = (x.softmax(-1) @ v).transpose(1, 2).flatten(0, 1)
    mass = (x.softmax(-1) @ v.abs()).transpose(1, 2).flatten(0, 1)
    # the dequantized rows are rounded to binary16: 2^-11 of a value and, through the scores, 2^-11 of sum |q k| twice
    size = (q.view(2, n, -1, layer.D).double().abs().transpose(1, 2) @ k.abs().transpose(-1, -2) * layer.D ** -0.5).amax().item()
    tol = 2.0 ** -8 * want.abs() + (2 * 2.0 ** -11 + 2 * 2.0 ** -11 * size) * mass + 1e-6
    assert ((out.double() - want).abs() <= tol).all()
    assert np.isfinite(lse.cpu().numpy()).all()


def test_smoke_calls(gpu_lib):
    prompt_smoke.run(gpu_lib)
