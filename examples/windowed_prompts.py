"""Prompts of text and image patches through a layer with a sliding window whose first tokens stay visible.

A prompt comes in chunks: each is normalized, rotated by positions with three axes (time, height, width),
quantized and appended to the paged NVFP4 cache, and attends to what the window lets it see. Then every decode
step appends one token per request and attends with the same window and first tokens; the step is captured into
a CUDA graph once and replayed. At the end drafts are verified: the last tokens once more, as one call, which has
to give what their own steps gave.

    python examples/windowed_prompts.py [--batch 4] [--prompt 3000] [--chunk 512] [--steps 8] [--window 1023] [--sink 16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_paged_kv_02_gb300 as nv  # noqa: E402


class Layer:
    """One attention layer's cache, norms and window. The projections are drawn at random."""

    def __init__(self, batch, tokens, window, sink, heads=8, group=4, head_dim=128, page_size=16, seed=0):
        self.H, self.G, self.D, self.ps, self.B = heads, group, head_dim, page_size, batch
        self.seen = dict(window_left=window, num_sink_tokens=sink)
        self.gen = torch.Generator("cuda").manual_seed(seed)
        dev = dict(device="cuda")
        pages = -(-tokens // page_size)
        pool = batch * pages
        self.tables = torch.randperm(pool, generator=self.gen, **dev).int().view(batch, pages).contiguous()
        self.indices, self.indptr = self.tables.flatten(), (torch.arange(batch + 1, **dev) * pages).int()
        self.codes = [torch.zeros((pool, heads, page_size, head_dim // 2), dtype=torch.uint8, **dev) for _ in range(2)]
        self.scales = [torch.zeros((pool, heads, page_size, head_dim // 16), dtype=torch.uint8, **dev) for _ in range(2)]
        self.lens = torch.zeros(batch, dtype=torch.int32, **dev)
        self.weights = [torch.ones(head_dim, dtype=torch.bfloat16, **dev) for _ in range(2)]
        half = head_dim // 2
        self.axes = nv.nvfp4_rotary_axes([half // 4, half * 3 // 8, half - half // 4 - half * 3 // 8])
        angle = torch.arange(tokens, dtype=torch.float64, **dev)[:, None] * 10000.0 ** -(torch.arange(half, dtype=torch.float64, **dev) / half)
        self.table = torch.cat([angle.cos(), angle.sin()], -1).float()
        self.gk, self.gv = (torch.tensor([4.0 / (6 * 448)], **dev) for _ in range(2))
        self.status = torch.zeros(1, dtype=torch.int32, **dev)

    def project(self, rows):
        return torch.randn((rows, (self.G + 2) * self.H, self.D), generator=self.gen, device="cuda").bfloat16()

    def append(self, qkv, requests, positions, axis_positions):
        """Queries of the rows, rotated; the keys and values go into the cache."""
        q, k, v = qkv.split([self.G * self.H, self.H, self.H], 1)
        return nv.nvfp4_qk_norm_rope_append_paged(
            q, k, v, *self.weights, self.table, requests, positions, self.codes, self.scales, self.indices, self.indptr,
            None, self.gk, self.gv, "HND", dev_status=self.status, rotary_positions=axis_positions, rotary_axes=self.axes)

    def prompt(self, q, indptr):
        """Attention of each request's last tokens."""
        return nv.nvfp4_paged_attention_prefill(q, self.codes, self.scales, indptr, self.tables, self.lens, self.gk, self.gv,
                                                "HND", dev_status=self.status, **self.seen)

    def step(self, q):
        """Attention of one new token of each request."""
        return nv.nvfp4_paged_attention_decode(q, self.codes, self.scales, self.tables, self.lens, self.gk, self.gv, "HND",
                                               dev_status=self.status, **self.seen)


def axis_positions(first, n, text):
    """[3, n] positions of the tokens from `first` on: `text` tokens of text, then images of 24 x 31 patches."""
    i = torch.arange(first, first + n, device="cuda")
    j = (i - text).clamp(min=0)
    patch = torch.stack([text + j // 744, text + j // 31 % 24, text + j % 31])
    return torch.where(i < text, i, patch).int()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("batch", 4), ("prompt", 3000), ("chunk", 512), ("steps", 8), ("window", 1023), ("sink", 16)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args(argv)
    layer = Layer(a.batch, a.prompt + a.steps + 1, a.window, a.sink)
    requests = torch.arange(a.batch, device="cuda", dtype=torch.int32)

    # the prompts, in chunks
    for first in range(0, a.prompt, a.chunk):
        n = min(a.chunk, a.prompt - first)
        where = torch.arange(first, first + n, device="cuda", dtype=torch.int32).repeat(a.batch)
        q = layer.append(layer.project(a.batch * n), requests.repeat_interleave(n), where,
                         axis_positions(first, n, a.prompt // 5).repeat(1, a.batch).contiguous())
        layer.lens.fill_(first + n)
        layer.prompt(q, (torch.arange(a.batch + 1, device="cuda") * n).int())

    # a step: its inputs are the projections; positions and lengths move on inside it
    qkv = layer.project(a.batch)
    positions = torch.full((a.batch,), a.prompt, device="cuda", dtype=torch.int32)

    def step():
        q = layer.append(qkv, requests, positions, positions.expand(3, -1).contiguous())
        layer.lens.copy_(positions + 1)
        out, lse = layer.step(q)
        positions.add_(1)
        return q, out, lse

    step()  # once outside a graph: the binding's workspaces
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, out, lse = step()
    steps = []
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(a.steps):
        qkv.copy_(layer.project(a.batch))
        graph.replay()
        steps.append([t.clone() for t in (q, out, lse)])
    end.record()

    # the last tokens as drafts to be verified, in one call
    drafts = min(a.steps, 4)
    q, out, lse = (torch.stack(t, 1).flatten(0, 1) for t in zip(*steps[-drafts:]))
    again, again_lse = layer.prompt(q, (torch.arange(a.batch + 1, device="cuda") * drafts).int())
    torch.cuda.synchronize()
    apart = (again.float() - out.float()).abs().max().item()
    lse_apart = (again_lse - lse).abs().max().item()
    size = out.float().abs().max().item()
    status = int(layer.status.item())
    print(f"{a.steps} steps of {a.batch} requests at {a.prompt}+ tokens, window {a.window} and {a.sink} first tokens: "
          f"{begin.elapsed_time(end) / a.steps * 1e3:.0f} us a step; {drafts} drafts verified: outputs up to {size:.3f}, "
          f"apart by {apart:.5f}, log-sum-exp by {lse_apart:.6f}, status {status}")
    return apart, lse_apart, size, status


if __name__ == "__main__":
    main()
