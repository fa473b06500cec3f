"""Cases, plain forms and 64-bit values of the decode-step operators over an NVFP4 paged cache.

One decode step of a model that keeps its keys and values in NVFP4 pages:

  append   per-head RMS norm and rotation of the query and key rows, then quantize-append of
           the key and value rows (nvfp4_qk_norm_rope_append_paged)
  bounds   element-wise minimum and maximum of each page's keys (nvfp4_page_key_bounds)
  select   the pages whose bounds promise the largest scores (nvfp4_select_pages)
  attend   attention of one new token per request (nvfp4_paged_attention_decode)
  sparse   the same over selected pages (nvfp4_sparse_paged_attention_decode)

Fields of a case: `op`; `dtype` f16 | bf16; `layout` NHD | HND; `ps` slots of a page; `hkv`
key/value heads; `g` query heads of each of them; `d` head_dim; `b` requests, whose lengths are
spread between `lo` and `hi` (evenly in the logarithm; the first `empty` of them are 0).
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
DEVICE = "cuda"


# ---- the cases ---------------------------------------------------------------------------

def listed():
    base = dict(dtype="bf16", layout="HND", ps=16, hkv=8, g=4, d=128, empty=0)
    return [
        # one new token of each of 64 running requests: a decode step, where latency counts
        dict(base, name="append-step", op="append", b=64, new=1, lo=512, hi=4096, rot=128,
             interleaved=False, four_over_six=False),
        # prompts of odd lengths, partial rotation of adjacent pairs, the 4over6 recipe
        dict(base, name="append-prompts", op="append", dtype="f16", layout="NHD", ps=32, b=4,
             new=8191, lo=1, hi=300, rot=64, interleaved=True, four_over_six=True),
        # the page that a decode step has written to, of each request
        dict(base, name="bounds-step", op="bounds", b=64, lo=512, hi=4096, last=1),
        # every page of 16 prompts, in larger pages of token-major rows
        dict(base, name="bounds-prompts", op="bounds", dtype="f16", layout="NHD", ps=32, b=16,
             lo=9001, hi=16384, last=0),
        # 64 requests of ordinary length, 64 pages (1024 tokens) for each head
        dict(base, name="select-batch", op="select", b=64, lo=1024, hi=16384, k=64, sink=1,
             recent=2),
        # few long requests: 8 K pages each, wide query groups
        dict(base, name="select-long", op="select", dtype="f16", g=8, b=4, lo=100000, hi=131072,
             k=256, sink=1, recent=4),
        # a handful of short requests, one empty, an odd head size: the smallest calls
        dict(base, name="attend-small", op="attend", dtype="f16", layout="NHD", ps=12, hkv=2, g=3,
             d=96, b=5, lo=1, hi=77, empty=1),
        # a decode batch
        dict(base, name="attend-batch", op="attend", g=8, b=64, lo=512, hi=4096),
        # one long document
        dict(base, name="attend-long", op="attend", dtype="f16", layout="NHD", ps=64, b=1,
             lo=131071, hi=131071),
        # a large batch of ragged lengths: what bounds a server's step
        dict(base, name="attend-large", op="attend", b=128, lo=128, hi=16384, empty=2),
        # 64 selected pages of each head
        dict(base, name="sparse-batch", op="sparse", b=64, lo=1024, hi=16384, k=64),
        # few long requests, 256 selected pages, head size 64
        dict(base, name="sparse-long", op="sparse", dtype="f16", layout="NHD", g=6, d=64, b=4,
             lo=100000, hi=131072, k=256),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["append", "bounds", "select", "attend", "attend", "sparse"])
    c = dict(op=op, dtype=rng.choice(["f16", "bf16"]), layout=rng.choice(["NHD", "HND"]),
             ps=rng.choice([4, 12, 16, 16, 32, 64, 100]), hkv=rng.choice([1, 2, 3, 4, 8, 8, 16]),
             g=rng.choice([1, 2, 4, 4, 5, 7, 8, 8, 12, 16]),
             d=rng.choice([64, 64, 96, 128, 128, 128, 128, 192, 256]),
             b=spread(1, 96), empty=0)
    # bytes and operations stay below those of the largest listed case
    most = (128 * 3300 * 8 * 128) // (c["hkv"] * c["d"]) // max(1, c["g"] // 4)
    if op == "append":
        c.update(new=rng.choice([1, 1, spread(1, 4096)]), lo=1, hi=spread(2, 4096),
                 rot=rng.choice([c["d"], c["d"], 32, 64]), interleaved=rng.random() < 0.4,
                 four_over_six=rng.random() < 0.4)
        c["new"] = max(1, min(c["new"], 32764 * 48 * 128 // (c["b"] * c["hkv"] * (c["g"] + 2) * c["d"])))
        return c
    hi = spread(1, max(2, min(131072, most // c["b"])))
    c.update(lo=max(1, spread(1, hi) // 2), hi=hi)
    if op == "attend":
        c["empty"] = rng.choice([0, 0, 1])
    if op == "bounds":
        c["last"] = rng.choice([0, 0, 1])
    if op in ("select", "sparse"):
        c["k"] = spread(1, 300)
    if op == "select":
        c.update(sink=rng.choice([0, 1, 2]), recent=rng.choice([1, 2, 4]))
    return c


def lengths(case):
    """The requests' lengths, smallest first."""
    b, lo, hi = case["b"], case["lo"], case["hi"]
    lens = [int(round(lo * (hi / lo) ** ((i + 0.5) / b))) for i in range(b)]
    if b == 1:
        lens = [hi]
    return [0] * min(case.get("empty", 0), b) + lens[case.get("empty", 0):]


def work(case):
    hkv, g, d, ps = case["hkv"], case["g"], case["d"], case["ps"]
    lens = lengths(case)
    pages = [-(-n // ps) for n in lens]
    row = d * 9 // 16  # a key or value row of one head: codes and scales
    q_io = 2 * case["b"] * hkv * g * d * 2
    if case["op"] == "append":
        n = case["b"] * case["new"]
        io = n * ((2 * g + 2) * hkv * d * 2 + 2 * hkv * row + 8) + case["rot"] * 4 * min(n, max(lens) + case["new"])
        return {"bytes": io + 4 * d, "flops": n * hkv * d * (10 * (g + 1) + 4)}
    if case["op"] == "bounds":
        first = [max(0, n - 1) if case["last"] else 0 for n in lens]
        slots = sum(n - f // ps * ps for n, f in zip(lens, first) if n)
        wrote = sum(p - f // ps for p, f, n in zip(pages, first, lens) if n)
        return {"bytes": slots * hkv * row + wrote * (hkv * d * 4 + 4), "flops": 3 * slots * hkv * d}
    if case["op"] == "select":
        kept = sum(min(p, case["k"]) for p in pages)
        return {"bytes": q_io // 2 + sum(pages) * (hkv * d * 4 + 4) + case["b"] * hkv * (case["k"] + 1) * 4,
                "flops": 4 * sum(pages) * hkv * g * d + kept}
    if case["op"] == "sparse":
        tokens = sum(min(n, case["k"] * ps) for n in lens)
        tables = sum(min(p, case["k"]) for p in pages) * hkv * 8
    else:
        tokens, tables = sum(lens), sum(pages) * 4
    return {"bytes": q_io + case["b"] * hkv * g * 4 + tokens * hkv * row * 2 + tables,
            "flops": 4 * tokens * hkv * g * d}


# ---- the codec in elementary operations ---------------------------------------------------

def _pair_table(device):
    """The two values that a byte of codes stands for, [256, 2]."""
    mag = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=device)
    val = torch.cat([mag, -mag])
    byte = torch.arange(256, device=device)
    return torch.stack([val[byte & 15], val[byte >> 4]], dim=-1)


def _decode(codes, scales):
    """codes [..., d/2], scale bytes [..., d/16] -> e2m1 * S in float32 [..., d]."""
    v = _pair_table(codes.device)[codes.int()].flatten(-2)
    s = scales.view(torch.float8_e4m3fn).float()
    return (v.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


def _halving(t):
    """The sum over the last dimension (a power of two) by halves: t[i] + t[i + n/2]."""
    while t.shape[-1] > 1:
        h = t.shape[-1] // 2
        t = t[..., :h] + t[..., h:]
    return t[..., 0]


def _padded(t):
    """The last dimension filled up with zeros to a power of two."""
    n = t.shape[-1]
    return torch.nn.functional.pad(t, (0, (1 << (n - 1).bit_length()) - n))


def _candidate(x, top, gs, cap):
    """One scale candidate: the magnitude codes with their signs, the scale, the decoded values."""
    amax = x.abs().amax(-1, keepdim=True)
    s = torch.clamp(amax / (top * gs), max=cap).to(torch.float8_e4m3fn)
    den = s.float() * gs
    inv = torch.where(den == 0, torch.zeros_like(den), torch.clamp(1.0 / den, max=torch.finfo(torch.float32).max))
    y = x * inv
    m = y.abs()
    code = ((m > 0.25).int() + (m >= 0.75).int() + (m > 1.25).int() + (m >= 1.75).int()
            + (m > 2.5).int() + (m >= 3.5).int() + (m > 5.0).int()) + 8 * torch.signbit(y).int()
    mag = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=x.device)
    return code, s, torch.cat([mag, -mag])[code] * s.float()


def _encode(rows, gs, four_over_six):
    """rows [..., d] -> packed codes [..., d/2], scale bytes [..., d/16]."""
    x = rows.float().unflatten(-1, (-1, 16))
    code, s, w = _candidate(x, 6.0, gs, 256.0 if four_over_six else 448.0)
    if four_over_six:
        code_b, s_b, w_b = _candidate(x, 4.0, gs, 448.0)
        # the element errors are rounded once: formed in 64 bits, which hold the residual
        err, err_b = (_halving((x.double() - v.double() * gs.double()).float().abs()) for v in (w, w_b))
        take = (err_b < err)[..., None]
        code = torch.where(take, code_b, code)
        s = torch.where(take, s_b.float(), s.float()).to(torch.float8_e4m3fn)
    code = code.flatten(-2)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8), s.squeeze(-1).view(torch.uint8)


# ---- inputs ------------------------------------------------------------------------------

def _cache(case, gen, pages, gs):
    """Codes and scales of `pages` pages of N(0, 1) rows."""
    hkv, d, ps = case["hkv"], case["d"], case["ps"]
    inner = (ps, hkv) if case["layout"] == "NHD" else (hkv, ps)
    codes = torch.empty((pages, *inner, d // 2), dtype=torch.uint8, device=DEVICE)
    scales = torch.empty((pages, *inner, d // 16), dtype=torch.uint8, device=DEVICE)
    step = max(1, (1 << 26) // (ps * hkv * d))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        codes[p:p + n], scales[p:p + n] = _encode(
            torch.randn((n, *inner, d), generator=gen, device=DEVICE), gs, False)
    return codes, scales


def _tables(case, lens, gen):
    """Page tables of `lens` tokens a request in a pool with some pages to spare, permuted."""
    ps = case["ps"]
    pages = [-(-n // ps) for n in lens]
    used = sum(pages)
    pool = used + used // 10 + 1
    indices = torch.randperm(pool, generator=gen, device=DEVICE)[:used].int()
    indptr = torch.tensor([0] + pages, device=DEVICE).cumsum(0).int()
    width = max(max(pages), 1)
    col = torch.arange(width, device=DEVICE)
    at = indptr[:-1, None].long() + col
    n = torch.tensor(pages, device=DEVICE)[:, None]
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEVICE)
    if used:
        table = torch.where(col < n, indices[at.clamp(max=used - 1)], table)
    return pool, indices, indptr, table.contiguous()


def prepare(case, seed):
    gen = torch.Generator(DEVICE).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    hkv, g, d, ps, b = case["hkv"], case["g"], case["d"], case["ps"], case["b"]
    lens = lengths(case)
    order = torch.randperm(b, generator=gen, device=DEVICE).tolist()
    lens = [lens[i] for i in order]
    if case["op"] == "append":
        lens = [n + case["new"] for n in lens]
    s = dict(case=case, page_size=ps, layout=case["layout"], sm_scale=1.0 / math.sqrt(d),
             gk=torch.tensor([5.5 / (6 * 448)], device=DEVICE), gv=torch.tensor([5.0 / (6 * 448)], device=DEVICE),
             seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEVICE))
    pool, s["kv_indices"], s["kv_indptr"], s["block_tables"] = _tables(case, lens, gen)
    inner = (ps, hkv) if case["layout"] == "NHD" else (hkv, ps)

    if case["op"] == "append":
        n = b * case["new"]
        qkv = torch.randn((n, (g + 2) * hkv, d), generator=gen, device=DEVICE)
        # a few channels of the projections stand out, as they do in trained models
        qkv = (qkv * (1 + 6 * (torch.rand(((g + 2) * hkv, d), generator=gen, device=DEVICE) < 0.02))).to(dt)
        s["query"], s["key"], s["value"] = qkv[:, :g * hkv], qkv[:, g * hkv:(g + 1) * hkv], qkv[:, (g + 1) * hkv:]
        s["q_weight"], s["k_weight"] = ((1 + 0.2 * torch.randn(d, generator=gen, device=DEVICE)).to(dt) for _ in range(2))
        first = s["seq_lens"] - case["new"]
        new = torch.arange(case["new"], device=DEVICE, dtype=torch.int32)
        s["positions"] = (first[:, None] + new).flatten()
        s["batch_indices"] = torch.arange(b, device=DEVICE, dtype=torch.int32).repeat_interleave(case["new"])
        half = case["rot"] // 2
        freq = 10000.0 ** (-torch.arange(half, device=DEVICE, dtype=torch.float64) / half)
        angle = torch.arange(max(lens), device=DEVICE, dtype=torch.float64)[:, None] * freq
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], -1).float()
        if case["four_over_six"]:
            s["gk"], s["gv"] = s["gk"] * (448 / 256), s["gv"] * (448 / 256)
        for name in ("k", "v"):
            s[name + "_codes"] = torch.zeros((pool, *inner, d // 2), dtype=torch.uint8, device=DEVICE)
            s[name + "_scales"] = torch.zeros((pool, *inner, d // 16), dtype=torch.uint8, device=DEVICE)
        return s

    s["query"] = (1.5 * torch.randn((b, g * hkv, d), generator=gen, device=DEVICE)).to(dt)
    if case["op"] == "select":
        mid = 0.6 * torch.randn((pool, hkv, d), generator=gen, device=DEVICE)
        lo = mid - 1 - torch.rand((pool, hkv, d), generator=gen, device=DEVICE)
        hi = mid + 1 + torch.rand((pool, hkv, d), generator=gen, device=DEVICE)
        s["key_bounds"] = (400 * torch.stack([lo, hi], 2)).half()
        return s
    s["k_codes"], s["k_scales"] = _cache(case, gen, pool, s["gk"])
    # the slots past a request's end hold what was there before, here scales that are NaN
    n = s["seq_lens"].long()
    part = ((n % ps) > 0).nonzero()[:, 0]
    last = s["block_tables"][part, (n[part] - 1) // ps].long()
    past = torch.arange(ps, device=DEVICE) >= (n[part] % ps)[:, None]

    def spoil(scales):
        hole = past[:, :, None, None] if case["layout"] == "NHD" else past[:, None, :, None]
        scales[last] = torch.where(hole, torch.full_like(scales[last], 0x7F), scales[last])

    spoil(s["k_scales"])
    if case["op"] == "bounds":
        s["first_positions"] = (s["seq_lens"] - 1).clamp(min=0) if case["last"] else torch.zeros_like(s["seq_lens"])
        s["key_bounds"] = torch.zeros((pool, hkv, 2, d), dtype=torch.float16, device=DEVICE)
        return s
    s["v_codes"], s["v_scales"] = _cache(case, gen, pool, s["gv"])
    spoil(s["v_scales"])
    if case["op"] == "sparse":
        # k of each request's pages for every head, in ascending order, the last one among them
        width = s["block_tables"].shape[1]
        pages = (n + ps - 1) // ps
        col = torch.arange(width, device=DEVICE)
        key = torch.rand((b, hkv, width), generator=gen, device=DEVICE)
        key = torch.where(col == pages[:, None, None] - 1, torch.full_like(key, -1), key)
        key = torch.where(col < pages[:, None, None], key, torch.full_like(key, 2))
        k = min(case["k"], width)
        pick = key.argsort(-1)[..., :k]
        s["num_selected"] = pages.clamp(max=k).int()[:, None].expand(b, hkv).contiguous()
        pick = torch.where(col[:k] < s["num_selected"][..., None], pick, torch.full_like(pick, 1 << 30)).sort(-1)[0]
        s["selected"] = torch.where(pick < (1 << 30), pick, torch.full_like(pick, -1)).int().contiguous()
    return s


# ---- one pass ----------------------------------------------------------------------------

def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import nvfp4_paged_kv_02_gb300 as nv
        if op == "append":
            recipe = nv.NVFP44Over6Config(256.0, "MAE", False) if s["case"]["four_over_six"] else None
            q = nv.nvfp4_qk_norm_rope_append_paged(
                s["query"], s["key"], s["value"], s["q_weight"], s["k_weight"], s["cos_sin"],
                s["batch_indices"], s["positions"], (s["k_codes"], s["v_codes"]),
                (s["k_scales"], s["v_scales"]), s["kv_indices"], s["kv_indptr"], None, s["gk"],
                s["gv"], s["layout"], eps=1e-6, rotary_interleaved=s["case"]["interleaved"],
                nvfp4_4over6=recipe)
            return _appended(s, q)
        if op == "bounds":
            nv.nvfp4_page_key_bounds(s["k_codes"], s["k_scales"], s["block_tables"], s["seq_lens"],
                                     s["key_bounds"], s["first_positions"], s["layout"])
            return s["key_bounds"]
        if op == "select":
            c = s["case"]
            return nv.nvfp4_select_pages(s["query"], s["key_bounds"], s["block_tables"],
                                         s["seq_lens"], s["page_size"], c["k"],
                                         num_sink_pages=c["sink"], num_recent_pages=c["recent"])
        cache = ((s["k_codes"], s["v_codes"]), (s["k_scales"], s["v_scales"]))
        if op == "sparse":
            return nv.nvfp4_sparse_paged_attention_decode(
                s["query"], *cache, s["block_tables"], s["seq_lens"], s["selected"],
                s["num_selected"], s["gk"], s["gv"], s["layout"], sm_scale=s["sm_scale"])
        return nv.nvfp4_paged_attention_decode(
            s["query"], *cache, s["block_tables"], s["seq_lens"], s["gk"], s["gv"], s["layout"],
            sm_scale=s["sm_scale"])
    return {"append": _append, "bounds": _bounds, "select": _select, "attend": _attend,
            "sparse": _attend_selected}[op](s)


def _appended(s, q):
    # the cache is updated state: its scales are e4m3 values; a byte of codes is a pair of e2m1
    # values in the one form a user has it, and equal bytes are equal values
    return {"query": q, "k_codes": s["k_codes"], "v_codes": s["v_codes"],
            "k_scales": s["k_scales"].view(torch.float8_e4m3fn), "v_scales": s["v_scales"].view(torch.float8_e4m3fn)}


def _norm_rope(x, weight, s):
    """RMS norm and rotation of rows [n, heads, d], the sum of squares in the operator's order."""
    d, rot = x.shape[-1], s["cos_sin"].shape[-1]
    x = x.float()
    # eight squares by halves; the two groups of eight that rotate together; then all by halves
    eight = _halving((x * x).unflatten(-1, (-1, 8)))
    turned = rot // 8
    both = torch.cat([eight[..., :turned // 2] + eight[..., turned // 2:turned],
                      eight[..., turned::2] + eight[..., turned + 1::2]], -1)
    mean = _halving(_padded(both))[..., None] * (1.0 / d)
    y = x * (1.0 / torch.sqrt(mean + 1e-6)) * weight.float()
    c, t = (v[:, None] for v in s["cos_sin"][s["positions"].long()].chunk(2, -1))
    if s["case"]["interleaved"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turn = torch.stack([a * c - b * t, b * c + a * t], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turn = torch.cat([a * c - b * t, b * c + a * t], -1)
    return torch.cat([turn, y[..., rot:]], -1)


def _append(s):
    dt = s["query"].dtype
    q = _norm_rope(s["query"], s["q_weight"], s).to(dt)
    k = _norm_rope(s["key"], s["k_weight"], s).to(dt)
    pos = s["positions"].long()
    at = s["kv_indptr"].long()[s["batch_indices"].long()] + pos // s["page_size"]
    page, slot = s["kv_indices"].long()[at], pos % s["page_size"]
    where = (page, slot) if s["layout"] == "NHD" else (page, slice(None), slot)
    for name, rows, gs in (("k", k, s["gk"]), ("v", s["value"], s["gv"])):
        codes, scales = _encode(rows, gs, s["case"]["four_over_six"])
        s[name + "_codes"][where] = codes
        s[name + "_scales"][where] = scales
    return _appended(s, q)


def _bounds(s):
    b, width = s["block_tables"].shape
    ps = s["page_size"]
    n, col = s["seq_lens"].long()[:, None], torch.arange(width, device=DEVICE)
    b_at, col_at = ((col >= s["first_positions"].long()[:, None] // ps) & (col * ps < n)).nonzero(as_tuple=True)
    page = s["block_tables"][b_at, col_at].long()
    x = _decode(s["k_codes"][page], s["k_scales"][page])
    if s["layout"] == "HND":
        x = x.transpose(1, 2)
    live = (col_at[:, None] * ps + torch.arange(ps, device=DEVICE) < n[b_at])[:, :, None, None]
    s["key_bounds"][page, :, 0] = torch.where(live, x, torch.full_like(x, math.inf)).amin(1).half()
    s["key_bounds"][page, :, 1] = torch.where(live, x, torch.full_like(x, -math.inf)).amax(1).half()
    return s["key_bounds"]


def _select(s):
    c = s["case"]
    b, width = s["block_tables"].shape
    bounds = s["key_bounds"][s["block_tables"].clamp(min=0).long()].float().transpose(1, 2)  # [b, hkv, width, 2, d]
    q = s["query"].float().view(b, c["hkv"], c["g"], 1, c["d"])
    # each product is exact; the sum runs over pairs of chains in groups of eight, then by halves
    term = q.clamp(min=0) * bounds[:, :, None, :, 1] + q.clamp(max=0) * bounds[:, :, None, :, 0]
    term = term.unflatten(-1, (-1, 4, 2))
    chain = term[..., 0, :] + term[..., 1, :] + term[..., 2, :] + term[..., 3, :]
    score = _halving(_padded(chain[..., 0] + chain[..., 1])).amax(2)
    pages = ((s["seq_lens"].long() + s["page_size"] - 1) // s["page_size"])[:, None, None]
    col = torch.arange(width, device=DEVICE)
    kept = (col < c["sink"]) | (col >= pages - c["recent"])
    score = torch.where(kept, torch.full_like(score, math.inf), score)
    score = torch.where(col < pages, score, torch.full_like(score, -math.inf))
    count = pages.clamp(max=c["k"]).expand(b, c["hkv"], 1)
    best = score.sort(dim=-1, descending=True, stable=True)[1][..., :c["k"]]
    best = torch.where(col[:best.shape[-1]] < count, best, torch.full_like(best, 1 << 30)).sort(-1)[0]
    best = torch.nn.functional.pad(best, (0, c["k"] - best.shape[-1]), value=1 << 30)
    return torch.where(best < (1 << 30), best, torch.full_like(best, -1)).int(), count[..., 0].int()


def _softmax_product(s, k, v, live):
    """softmax(q k) v of k, v [b, hkv, t, d] where `live`, in 32 bits."""
    c = s["case"]
    b = s["query"].shape[0]
    q = s["query"].float().view(b, c["hkv"], c["g"], c["d"])
    score = torch.matmul(q, k.transpose(-1, -2)) * (s["gk"] * s["sm_scale"])
    score = torch.where(live[:, :, None], score, torch.full_like(score, -math.inf))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total) * s["gv"]
    lse = (top + torch.log(total))[..., 0]
    return o.view(b, -1, c["d"]).to(s["query"].dtype), lse.view(b, -1)


def _attend(s):
    table = s["block_tables"].clamp(min=0).long()
    t = torch.arange(table.shape[1] * s["page_size"], device=DEVICE)
    live = (t < s["seq_lens"][:, None])[:, None]
    rows = []
    for name in ("k", "v"):
        x = _decode(s[name + "_codes"][table], s[name + "_scales"][table])  # [b, pages, ., ., d]
        x = (x if s["layout"] == "HND" else x.transpose(2, 3)).transpose(1, 2).flatten(2, 3)
        rows.append(torch.where(live[..., None], x, torch.zeros_like(x)))
    return _softmax_product(s, *rows, live)


def _attend_selected(s):
    ps = s["page_size"]
    page = s["block_tables"].clamp(min=0).long().unsqueeze(1).expand(-1, s["case"]["hkv"], -1).gather(
        2, s["selected"].clamp(min=0).long())  # [b, hkv, k]
    t = s["selected"].long()[..., None] * ps + torch.arange(ps, device=DEVICE)
    live = ((s["selected"] >= 0)[..., None] & (t < s["seq_lens"][:, None, None, None])).flatten(2)
    head = torch.arange(s["case"]["hkv"], device=DEVICE)[None, :, None]
    rows = []
    for name in ("k", "v"):
        codes, scales = s[name + "_codes"], s[name + "_scales"]
        if s["layout"] == "NHD":
            codes, scales = codes.transpose(1, 2), scales.transpose(1, 2)
        x = _decode(codes[page, head], scales[page, head]).flatten(2, 3)
        rows.append(torch.where(live[..., None], x, torch.zeros_like(x)))
    return _softmax_product(s, *rows, live)


# ---- the definitions in 64 bits -----------------------------------------------------------

def _real(codes, scales):
    """The real numbers of codes and scales by the formats' bit fields, in 64 bits."""
    def field(c):
        e, m = (c >> 1) & 3, (c & 1).double()
        v = torch.where(e == 0, m / 2, torch.ldexp(1 + m / 2, e - 1))
        return torch.where(c >= 8, -v, v)
    c, b = codes.int(), scales.int()
    v = torch.stack([field(c & 15), field(c >> 4)], -1).reshape(*codes.shape[:-1], -1)
    e, m = (b >> 3) & 15, (b & 7).double()
    sc = torch.where(e == 0, torch.ldexp(m, torch.full_like(e, -9)), torch.ldexp(1 + m / 8, e - 7))
    sc = torch.where((b & 127) == 127, torch.full_like(sc, math.nan), torch.where(b >= 128, -sc, sc))
    return v * sc.repeat_interleave(16, -1)


def _rotated(x, weight, s):
    """Norm and rotation as complex numbers times e^(i angle), in 64 bits."""
    rot = s["cos_sin"].shape[-1]
    x = x.double()
    y = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * weight.double()
    row = s["cos_sin"].double()[s["positions"].long()][:, None]
    turn = torch.complex(row[..., :rot // 2], row[..., rot // 2:])
    if s["case"]["interleaved"]:
        z = torch.view_as_complex(y[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * turn
        head = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * turn
        head = torch.cat([z.real, z.imag], -1)
    return torch.cat([head, y[..., rot:]], -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        # the codes are bytes and the scales of rows that were rounded on the way: no such value
        return {"query": _rotated(s["query"], s["q_weight"], s), "k_codes": None, "v_codes": None,
                "k_scales": None, "v_scales": None}
    if case["op"] == "select":
        return None  # whole numbers only
    ps, g = case["ps"], case["g"]
    if case["op"] == "bounds":
        out = torch.zeros_like(s["key_bounds"], dtype=torch.float64)
        first = s["first_positions"].tolist()
        for i, n in enumerate(s["seq_lens"].tolist()):
            if n == 0:
                continue
            table = s["block_tables"][i, first[i] // ps:-(-n // ps)].long()
            x = _real(s["k_codes"][table], s["k_scales"][table])
            x = x if case["layout"] == "NHD" else x.transpose(1, 2)  # [pages, ps, hkv, d]
            r = n - (first[i] // ps + len(table) - 1) * ps
            out[table[:-1]] = torch.stack([x[:-1].amin(1), x[:-1].amax(1)], 2)
            out[table[-1]] = torch.stack([x[-1, :r].amin(0), x[-1, :r].amax(0)], 1)
        return out
    o = torch.zeros(s["query"].shape, dtype=torch.float64, device=DEVICE)
    lse = torch.full(s["query"].shape[:2], -math.inf, dtype=torch.float64, device=DEVICE)
    for i, n in enumerate(s["seq_lens"].tolist()):
        for h in range(case["hkv"] if n else 0):
            if case["op"] == "sparse":
                pages = s["selected"][i, h, :int(s["num_selected"][i, h])].long()
            else:
                pages = torch.arange(-(-n // ps), device=DEVICE)
            t = (pages[:, None] * ps + torch.arange(ps, device=DEVICE)).flatten()
            at = s["block_tables"][i][pages].long()
            rows = []
            for name in ("k", "v"):
                c, f = s[name + "_codes"], s[name + "_scales"]
                c, f = (c[at, :, h], f[at, :, h]) if case["layout"] == "NHD" else (c[at, h], f[at, h])
                rows.append(_real(c, f).flatten(0, 1)[t < n])
            q = s["query"][i, h * g:(h + 1) * g].double()
            x = q @ rows[0].T * (s["gk"].double() * case["d"] ** -0.5)
            lse[i, h * g:(h + 1) * g] = torch.logsumexp(x, -1)
            o[i, h * g:(h + 1) * g] = torch.softmax(x, -1) @ rows[1] * s["gv"].double()
    return o, lse
