"""Decode steps over a paged NVFP4 cache with the pages that matter only.

A prompt's projections go into the cache (norm, rotation and quantize-append in one pass), the
bounds of its pages are taken, and then every step appends one token per request, renews the
bounds of the page that it went to, selects pages for each (request, KV head) by their bounds and
attends to them. The step is captured into a CUDA graph once and replayed. The last step is
repeated over all pages, to say how far the selection is from dense attention.

    python examples/sparse_decode.py [--batch 8] [--prompt 4096] [--steps 16] [--pages 64]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_paged_kv_02_gb300 as nv  # noqa: E402


class Layer:
    """One attention layer's cache and norms. The projections are drawn at random, so few positions
    stand out, and the share of the weight that the selection holds is far below a trained model's."""

    def __init__(self, batch, tokens, heads=8, group=4, head_dim=128, page_size=16, seed=0):
        self.H, self.G, self.D, self.ps, self.B = heads, group, head_dim, page_size, batch
        self.gen = torch.Generator("cuda").manual_seed(seed)
        pages = -(-tokens // page_size)
        pool = batch * pages
        dev = dict(device="cuda")
        self.tables = torch.randperm(pool, generator=self.gen, **dev).int().view(batch, pages).contiguous()
        self.indices, self.indptr = self.tables.flatten(), (torch.arange(batch + 1, **dev) * pages).int()
        self.codes = [torch.zeros((pool, heads, page_size, head_dim // 2), dtype=torch.uint8, **dev) for _ in range(2)]
        self.scales = [torch.zeros((pool, heads, page_size, head_dim // 16), dtype=torch.uint8, **dev) for _ in range(2)]
        self.bounds = torch.zeros((pool, heads, 2, head_dim), dtype=torch.float16, **dev)
        self.lens = torch.zeros(batch, dtype=torch.int32, **dev)
        self.weights = [torch.ones(head_dim, dtype=torch.bfloat16, **dev) for _ in range(2)]
        half = torch.arange(head_dim // 2, dtype=torch.float64, **dev) / (head_dim // 2)
        angle = torch.arange(tokens, dtype=torch.float64, **dev)[:, None] * 10000.0 ** -half
        self.table = torch.cat([angle.cos(), angle.sin()], -1).float()
        self.gk, self.gv = (torch.tensor([4.0 / (6 * 448)], **dev) for _ in range(2))
        self.status = torch.zeros(1, dtype=torch.int32, **dev)

    def project(self, rows):
        qkv = torch.randn((rows, (self.G + 2) * self.H, self.D), generator=self.gen, device="cuda")
        return (qkv * (1 + (torch.rand(qkv.shape[:2], generator=self.gen, device="cuda") < 0.02)[..., None] * 3)).bfloat16()

    def append(self, qkv, requests, positions):
        """Queries of the rows, rotated; the keys and values go into the cache."""
        q, k, v = qkv.split([self.G * self.H, self.H, self.H], 1)
        return nv.nvfp4_qk_norm_rope_append_paged(
            q, k, v, *self.weights, self.table, requests, positions, self.codes, self.scales, self.indices,
            self.indptr, None, self.gk, self.gv, "HND", dev_status=self.status)

    def renew_bounds(self, first):
        nv.nvfp4_page_key_bounds(self.codes[0], self.scales[0], self.tables, self.lens, self.bounds, first, "HND",
                                 dev_status=self.status)

    def attend(self, q, pages=None):
        cache = (self.codes, self.scales, self.tables, self.lens)
        if pages is None:
            return nv.nvfp4_paged_attention_decode(q, *cache, self.gk, self.gv, "HND", dev_status=self.status)
        chosen = nv.nvfp4_select_pages(q, self.bounds, self.tables, self.lens, self.ps, pages, num_sink_pages=1,
                                       num_recent_pages=2, dev_status=self.status)
        return nv.nvfp4_sparse_paged_attention_decode(q, *cache, *chosen, self.gk, self.gv, "HND",
                                                      dev_status=self.status)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("batch", 8), ("prompt", 4096), ("steps", 16), ("pages", 64)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args(argv)
    layer = Layer(a.batch, a.prompt + a.steps + 1)
    requests = torch.arange(a.batch, device="cuda", dtype=torch.int32)

    # the prompts
    layer.append(layer.project(a.batch * a.prompt), requests.repeat_interleave(a.prompt),
                 torch.arange(a.prompt, device="cuda", dtype=torch.int32).repeat(a.batch))
    layer.lens.fill_(a.prompt)
    layer.renew_bounds(None)

    # a step: its inputs are the projections; positions and lengths move on inside it
    qkv = layer.project(a.batch)
    positions = torch.full((a.batch,), a.prompt, device="cuda", dtype=torch.int32)

    def step():
        q = layer.append(qkv, requests, positions)
        layer.lens.copy_(positions + 1)
        layer.renew_bounds(positions)
        out, lse = layer.attend(q, a.pages)
        positions.add_(1)
        return q, out, lse

    step()  # once outside a graph: the binding's workspaces
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, out, lse = step()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(a.steps):
        qkv.copy_(layer.project(a.batch))
        graph.replay()
    end.record()
    dense, dense_lse = layer.attend(q)
    torch.cuda.synchronize()
    near = torch.nn.functional.cosine_similarity(out.float().flatten(1), dense.float().flatten(1)).mean().item()
    mass = torch.exp(lse - dense_lse).mean().item()
    status = int(layer.status.item())
    print(f"{a.steps} steps of {a.batch} requests at {a.prompt}+ tokens: {begin.elapsed_time(end) / a.steps * 1e3:.0f} us "
          f"a step; {a.pages} of {-(-int(layer.lens[0]) // layer.ps)} pages hold {mass:.3f} of the weight, cosine to "
          f"dense attention {near:.4f}, status {status}")
    return near, mass, status


if __name__ == "__main__":
    main()
