"""Cases, plain forms and 64-bit values of the operators that read several new tokens at once, or a
window of the past with the first tokens kept, and of positions with several axes.

  prompt   attention of the last tokens of each request over its paged NVFP4 cache: prompts, chunks of
           prompts, drafts to be verified (nvfp4_paged_attention_prefill)
  sinks    attention of one new token per request over a sliding window and the first tokens
           (nvfp4_paged_attention_decode with num_sink_tokens)
  axes     norm, rotation by positions with several axes (time, height, width), and the append
           (nvfp4_qk_norm_rope_append_paged with rotary_positions)

Fields of a case: `op`; `dtype` f16 | bf16; `layout` NHD | HND; `ps` slots of a page; `hkv` key/value
heads; `g` query heads of each of them; `d` head_dim; `b` requests, which hold between `lo` and `hi`
tokens before the new ones (spread evenly in the logarithm; the first `empty` of them hold none).
prompt and sinks: `new`, `new_hi` new tokens of a request; `causal`; `window` tokens to the left of a
query that it sees (-1: all) besides the first `sink`; `cap` of the logits (0: none). axes: `new` tokens;
`rot` rotated elements, of adjacent pairs when `interleaved`; `sections`: the pairs of each axis, one after
the other or, with `mixed`, in turn; `four_over_six`.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
DEVICE = "cuda"


# ---- the cases ---------------------------------------------------------------------------

def listed():
    base = dict(dtype="bf16", layout="HND", ps=16, hkv=8, g=4, d=128, empty=0)
    prompt = dict(base, op="prompt", causal=True, window=-1, sink=0, cap=0.0)
    sinks = dict(base, op="sinks", new=1, new_hi=1, causal=True, cap=0.0)
    axes = dict(base, op="axes", rot=128, interleaved=False, mixed=False, four_over_six=False)
    return [
        # a handful of short requests with a few new tokens, odd sizes: the smallest calls
        dict(prompt, name="prompt-small", dtype="f16", layout="NHD", ps=12, hkv=2, g=3, d=96, b=5, lo=1, hi=77,
             empty=1, new=1, new_hi=9, window=50, sink=4),
        # drafts of four tokens to be verified, for a batch of running requests
        dict(prompt, name="prompt-verify", b=64, lo=512, hi=4096, new=4, new_hi=4),
        # chunks of prompts of ragged lengths beside what their requests hold already
        dict(prompt, name="prompt-chunks", b=8, lo=100, hi=8192, new=64, new_hi=2048),
        # one long prompt
        dict(prompt, name="prompt-long", dtype="f16", layout="NHD", ps=64, b=1, lo=1, hi=1, empty=1, new=12345,
             new_hi=12345),
        # prompts of a layer with a sliding window and first tokens that stay visible, wide query groups
        dict(prompt, name="prompt-window", hkv=4, g=8, b=4, lo=1, hi=1, empty=4, new=6001, new_hi=8191, window=1023,
             sink=64),
        # tokens of images that see each other, large heads, capped logits
        dict(prompt, name="prompt-images", dtype="f16", hkv=4, g=2, d=256, b=16, lo=40, hi=512, new=256, new_hi=1024,
             causal=False, cap=50.0),
        # one new token of a few short requests of a layer with a small window
        dict(sinks, name="sinks-small", dtype="f16", layout="NHD", ps=12, hkv=2, g=3, d=96, b=16, lo=1, hi=300,
             empty=1, window=63, sink=4),
        # a decode batch of ragged lengths
        dict(sinks, name="sinks-batch", b=128, lo=128, hi=16384, window=2047, sink=16),
        # few long requests, a wide window
        dict(sinks, name="sinks-long", dtype="f16", layout="NHD", ps=64, g=8, b=4, lo=60000, hi=100000, window=32767,
             sink=128),
        # one new token of each of 64 running requests whose prompts held images
        dict(axes, name="axes-step", b=64, new=1, lo=512, hi=4096, sections="16 24 24"),
        # prompts of text and images, an axis' pairs next to each other
        dict(axes, name="axes-prompts", b=4, new=8191, lo=1, hi=300, sections="16 24 24"),
        # prompts of video, the axes in turn, partial rotation of adjacent pairs, the 4over6 recipe
        dict(axes, name="axes-video", dtype="f16", layout="NHD", ps=32, b=4, new=8191, lo=1, hi=300, rot=64,
             interleaved=True, sections="12 10 10", mixed=True, four_over_six=True),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["prompt", "prompt", "prompt", "sinks", "axes"])
    c = dict(op=op, dtype=rng.choice(["f16", "bf16"]), layout=rng.choice(["NHD", "HND"]),
             ps=rng.choice([4, 12, 16, 16, 32, 64, 100]), hkv=rng.choice([1, 2, 3, 4, 8, 8]),
             g=rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 8, 12]),
             d=rng.choice([64, 64, 80, 96, 128, 128, 128, 128, 192, 256]), empty=0)
    heads = c["hkv"] * c["g"] * c["d"]
    if op == "axes":
        c["b"] = spread(1, 96)
        rot = rng.choice([c["d"], c["d"], 32, 64])
        pairs = rot // 2
        one = rng.randint(1, pairs - 2)
        two = rng.randint(1, pairs - one - 1)
        c.update(new=rng.choice([1, 1, spread(1, 4096)]), lo=1, hi=spread(2, 4096), rot=rot,
                 interleaved=rng.random() < 0.4, mixed=rng.random() < 0.4, four_over_six=rng.random() < 0.4,
                 sections=rng.choice([f"{pairs}", f"{one} {pairs - one}", f"{one} {two} {pairs - one - two}"]))
        c["new"] = max(1, min(c["new"], 32764 * 48 * 128 // (c["b"] * c["hkv"] * (c["g"] + 2) * c["d"])))
        return c
    c["window"] = rng.choice([-1, spread(1, 8192), spread(1, 1024)])
    c["sink"] = rng.choice([0, 1, 4, spread(1, 300)]) if c["window"] >= 0 else 0
    c["cap"] = rng.choice([0.0, 0.0, 30.0])
    if op == "sinks":
        c["window"] = spread(1, 30000)
        c["b"] = spread(1, 96)
        hi = spread(1, max(2, min(131072, 400000 * 8 * 128 // (c["hkv"] * c["d"]) // c["b"])))
        c.update(new=1, new_hi=1, causal=True, lo=max(1, spread(1, hi) // 2), hi=hi, empty=rng.choice([0, 0, 1]))
        return c
    c.update(b=spread(1, 64), causal=rng.random() < 0.8)
    hi = spread(1, max(2, 200000 // c["b"]))
    new_hi = spread(1, 8192)
    # operations stay below those of the largest listed case, its tokens' bytes too
    while (c["b"] * new_hi * (hi + new_hi) * heads > 2.5e11 or c["b"] * new_hi * heads > 4e7) and new_hi > 1:
        new_hi = new_hi * 2 // 3
    c.update(lo=max(1, spread(1, hi) // 2), hi=hi, new=max(1, spread(1, new_hi)), new_hi=new_hi,
             empty=rng.choice([0, 0, 1]))
    return c


def _spaced(b, lo, hi):
    if b == 1:
        return [hi]
    return [int(round(lo * (hi / lo) ** ((i + 0.5) / b))) for i in range(b)]


def lengths(case):
    """The requests' tokens before the new ones, and their new ones."""
    b, empty = case["b"], min(case["empty"], case["b"])
    held = [0] * empty + _spaced(b, case["lo"], case["hi"])[empty:]
    new = _spaced(b, case["new"], case.get("new_hi", case["new"]))
    return held, [new[(5 * i + 2) % b] if b % 5 else new[(i * 7 + 3) % b] for i in range(b)]


def _pairs(case):
    """Pairs of a query token and a position that it sees, and positions that some query token sees."""
    total = seen = 0
    for held, new in zip(*lengths(case)):
        n = held + new
        p = torch.arange(held, n, dtype=torch.int64)
        hi = p + 1 if case["causal"] else torch.full_like(p, n)
        lo = (p - case["window"]).clamp(min=0) if case["window"] >= 0 else torch.zeros_like(p)
        sink = torch.minimum(torch.minimum(lo, hi), torch.full_like(p, case["sink"]))
        total += int((hi - torch.minimum(lo, hi) + sink).sum())
        first = int(lo[0])
        seen += int(hi[-1]) - first + min(case["sink"], first)
    return total, seen


def work(case):
    hkv, g, d = case["hkv"], case["g"], case["d"]
    held, new = lengths(case)
    row = d * 9 // 16  # a key or value row of one head: codes and scales
    rows = sum(new)
    if case["op"] == "axes":
        io = rows * ((2 * g + 2) * hkv * d * 2 + 2 * hkv * row + 8 + 4 * len(case["sections"].split()))
        table = case["rot"] * 4 * min(rows, max(a + b for a, b in zip(held, new)))
        return {"bytes": io + table + 4 * d, "flops": rows * hkv * d * (10 * (g + 1) + 4)}
    pairs, seen = _pairs(case)
    io = rows * hkv * g * (4 * d + 4) + seen * hkv * row * 2 + -(-seen // case["ps"]) * 4
    return {"bytes": io, "flops": 4 * pairs * hkv * g * d}


# ---- the codec in elementary operations ---------------------------------------------------

def _magnitudes(device):
    mag = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=device)
    return torch.cat([mag, -mag])


def _decode(codes, scales):
    """codes [..., d/2], scale bytes [..., d/16] -> e2m1 * S in float32 [..., d]."""
    val, byte = _magnitudes(codes.device), torch.arange(256, device=codes.device)
    v = torch.stack([val[byte & 15], val[byte >> 4]], dim=-1)[codes.int()].flatten(-2)
    s = scales.view(torch.float8_e4m3fn).float()
    return (v.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


def _halving(t):
    """The sum over the last dimension (a power of two) by halves: t[i] + t[i + n/2]."""
    while t.shape[-1] > 1:
        h = t.shape[-1] // 2
        t = t[..., :h] + t[..., h:]
    return t[..., 0]


def _padded(t):
    n = t.shape[-1]
    return torch.nn.functional.pad(t, (0, (1 << (n - 1).bit_length()) - n))


def _candidate(x, top, gs, cap):
    """One scale candidate: the codes, the scale, the decoded values."""
    amax = x.abs().amax(-1, keepdim=True)
    s = torch.clamp(amax / (top * gs), max=cap).to(torch.float8_e4m3fn)
    den = s.float() * gs
    inv = torch.where(den == 0, torch.zeros_like(den), torch.clamp(1.0 / den, max=torch.finfo(torch.float32).max))
    y = x * inv
    m = y.abs()
    code = ((m > 0.25).int() + (m >= 0.75).int() + (m > 1.25).int() + (m >= 1.75).int()
            + (m > 2.5).int() + (m >= 3.5).int() + (m > 5.0).int()) + 8 * torch.signbit(y).int()
    return code, s, _magnitudes(x.device)[code] * s.float()


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


def _axis_of_pair(case):
    """The axis of each pair, from the pairs of each axis."""
    left = [int(n) for n in case["sections"].split()]
    if not case["mixed"]:
        return [a for a, n in enumerate(left) for _ in range(n)]
    order = []
    while any(left):  # in turn, until an axis has had its pairs
        for a in range(len(left)):
            if left[a]:
                order.append(a)
                left[a] -= 1
    return order


def _axis_positions(axes, first, new):
    """[axes, new] positions of tokens from `first` on: some text, then frames of 24 x 31 patches."""
    i = torch.arange(new)
    text = max(1, new // 5)
    j = (i - text).clamp(min=0)
    frame = torch.stack([text + j // 744, text + j // 31 % 24, text + j % 31])
    pos = torch.where(i < text, i, frame)[:axes]
    return (first + torch.minimum(pos, torch.tensor(new - 1))).int()


def prepare(case, seed):
    gen = torch.Generator(DEVICE).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    hkv, g, d, ps, b = case["hkv"], case["g"], case["d"], case["ps"], case["b"]
    order = torch.randperm(b, generator=gen, device=DEVICE).tolist()
    held, new = ([v[i] for i in order] for v in lengths(case))
    lens = [x + y for x, y in zip(held, new)]
    s = dict(case=case, page_size=ps, layout=case["layout"], sm_scale=1.0 / math.sqrt(d),
             gk=torch.tensor([5.5 / (6 * 448)], device=DEVICE), gv=torch.tensor([5.0 / (6 * 448)], device=DEVICE),
             seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEVICE), lens=lens, new=new)
    pool, s["kv_indices"], s["kv_indptr"], s["block_tables"] = _tables(case, lens, gen)
    rows = sum(new)

    if case["op"] == "axes":
        qkv = torch.randn((rows, (g + 2) * hkv, d), generator=gen, device=DEVICE)
        # a few channels of the projections stand out, as they do in trained models
        qkv = (qkv * (1 + 6 * (torch.rand(((g + 2) * hkv, d), generator=gen, device=DEVICE) < 0.02))).to(dt)
        s["query"], s["key"], s["value"] = qkv[:, :g * hkv], qkv[:, g * hkv:(g + 1) * hkv], qkv[:, (g + 1) * hkv:]
        s["q_weight"], s["k_weight"] = ((1 + 0.2 * torch.randn(d, generator=gen, device=DEVICE)).to(dt) for _ in range(2))
        s["positions"] = torch.cat([torch.arange(x, x + y) for x, y in zip(held, new)]).int().to(DEVICE)
        s["batch_indices"] = torch.repeat_interleave(torch.arange(b), torch.tensor(new)).int().to(DEVICE)
        axes = len(case["sections"].split())
        s["rotary_positions"] = torch.cat([_axis_positions(axes, x, y) for x, y in zip(held, new)], 1).to(DEVICE)
        s["rotary_axes"] = torch.tensor(_axis_of_pair(case), dtype=torch.uint8, device=DEVICE)
        half = case["rot"] // 2
        freq = 10000.0 ** (-torch.arange(half, device=DEVICE, dtype=torch.float64) / half)
        angle = torch.arange(max(lens), device=DEVICE, dtype=torch.float64)[:, None] * freq
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], -1).float()
        if case["four_over_six"]:
            s["gk"], s["gv"] = s["gk"] * (448 / 256), s["gv"] * (448 / 256)
        inner = (ps, hkv) if case["layout"] == "NHD" else (hkv, ps)
        for name in ("k", "v"):
            s[name + "_codes"] = torch.zeros((pool, *inner, d // 2), dtype=torch.uint8, device=DEVICE)
            s[name + "_scales"] = torch.zeros((pool, *inner, d // 16), dtype=torch.uint8, device=DEVICE)
        return s

    s["query"] = (1.5 * torch.randn((rows, g * hkv, d), generator=gen, device=DEVICE)).to(dt)
    s["qo_indptr"] = torch.tensor([0] + new, device=DEVICE).cumsum(0).int()
    n = s["seq_lens"].long()
    part = ((n % ps) > 0).nonzero()[:, 0]
    last = s["block_tables"][part, (n[part] - 1) // ps].long()
    past = torch.arange(ps, device=DEVICE) >= (n[part] % ps)[:, None]
    hole = past[:, :, None, None] if case["layout"] == "NHD" else past[:, None, :, None]
    for name, gs in (("k", s["gk"]), ("v", s["gv"])):
        s[name + "_codes"], scales = _cache(case, gen, pool, gs)
        # the slots past a request's end hold what was there before, here scales that are NaN
        scales[last] = torch.where(hole, torch.full_like(scales[last], 0x7F), scales[last])
        s[name + "_scales"] = scales
    return s


# ---- one pass ----------------------------------------------------------------------------

def run(state):
    s, c = state, state["case"]
    if not own:
        return {"prompt": _attend, "sinks": _attend, "axes": _append}[c["op"]](s)
    import nvfp4_paged_kv_02_gb300 as nv
    cache = ((s["k_codes"], s["v_codes"]), (s["k_scales"], s["v_scales"]))
    if c["op"] == "axes":
        recipe = nv.NVFP44Over6Config(256.0, "MAE", False) if c["four_over_six"] else None
        q = nv.nvfp4_qk_norm_rope_append_paged(
            s["query"], s["key"], s["value"], s["q_weight"], s["k_weight"], s["cos_sin"], s["batch_indices"],
            s["positions"], *cache, s["kv_indices"], s["kv_indptr"], None, s["gk"], s["gv"], s["layout"], eps=1e-6,
            rotary_interleaved=c["interleaved"], nvfp4_4over6=recipe, rotary_positions=s["rotary_positions"],
            rotary_axes=s["rotary_axes"])
        return _appended(s, q)
    if c["op"] == "sinks":
        return nv.nvfp4_paged_attention_decode(
            s["query"], *cache, s["block_tables"], s["seq_lens"], s["gk"], s["gv"], s["layout"],
            sm_scale=s["sm_scale"], logits_soft_cap=c["cap"], window_left=c["window"], num_sink_tokens=c["sink"])
    return nv.nvfp4_paged_attention_prefill(
        s["query"], *cache, s["qo_indptr"], s["block_tables"], s["seq_lens"], s["gk"], s["gv"], s["layout"],
        causal=c["causal"], sm_scale=s["sm_scale"], logits_soft_cap=c["cap"], window_left=c["window"],
        num_sink_tokens=c["sink"])


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
    pair = torch.arange(rot // 2, device=DEVICE)
    at = s["rotary_positions"].long()[s["rotary_axes"].long()].T  # [n, pairs]
    c, t = s["cos_sin"][at, pair][:, None], s["cos_sin"][at, rot // 2 + pair][:, None]
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


def _live(c, p, n):
    """Which of positions 0 .. n a query at each of the positions p sees, [queries, n]."""
    t = torch.arange(n, device=DEVICE)
    live = torch.ones((len(p), n), dtype=torch.bool, device=DEVICE)
    if c["window"] >= 0:
        live = (t >= p[:, None] - c["window"]) | (t < c["sink"])
    if c["causal"]:
        live = live & (t <= p[:, None])
    return live


def _attend(s):
    c = s["case"]
    hkv, g, d, ps = c["hkv"], c["g"], c["d"], c["ps"]
    out = torch.empty_like(s["query"])
    lse = torch.empty(s["query"].shape[:2], dtype=torch.float32, device=DEVICE)
    row = 0
    for i, (n, new) in enumerate(zip(s["lens"], s["new"])):
        pages = s["block_tables"][i, :-(-n // ps)].long()
        kv = []
        for name in ("k", "v"):
            x = _decode(s[name + "_codes"][pages], s[name + "_scales"][pages])
            x = (x if c["layout"] == "HND" else x.transpose(1, 2)).transpose(0, 1).flatten(1, 2)[:, :n]
            kv.append(x)  # [hkv, n, d]
        step = max(1, (1 << 28) // (hkv * g * n))
        for q0 in range(0, new, step):
            q1 = min(new, q0 + step)
            live = _live(c, torch.arange(n - new + q0, n - new + q1, device=DEVICE), n)
            q = s["query"][row + q0:row + q1].float().view(-1, hkv, g, d).permute(1, 2, 0, 3).reshape(hkv, -1, d)
            x = torch.matmul(q, kv[0].transpose(1, 2)) * (s["gk"] * s["sm_scale"])
            if c["cap"] > 0:
                x = c["cap"] * torch.tanh(x / c["cap"])
            x = x.view(hkv, g, -1, n).masked_fill_(~live, -math.inf).view(hkv, -1, n)
            top = x.amax(-1, keepdim=True)
            p = torch.exp(x - top)
            total = p.sum(-1, keepdim=True)
            o = torch.matmul(p, kv[1]) / total * s["gv"]
            out[row + q0:row + q1] = o.view(hkv, g, -1, d).permute(2, 0, 1, 3).flatten(1, 2).to(out.dtype)
            lse[row + q0:row + q1] = (top + torch.log(total)).view(hkv, g, -1).permute(2, 0, 1).flatten(1, 2)
        row += new
    return out, lse


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
    table = torch.complex(s["cos_sin"][:, :rot // 2].double(), s["cos_sin"][:, rot // 2:].double())
    turn = torch.empty((x.shape[0], 1, rot // 2), dtype=table.dtype, device=DEVICE)
    for k, axis in enumerate(_axis_of_pair(s["case"])):
        turn[:, 0, k] = table[s["rotary_positions"][axis].long(), k]
    if s["case"]["interleaved"]:
        z = torch.view_as_complex(y[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * turn
        head = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * turn
        head = torch.cat([z.real, z.imag], -1)
    return torch.cat([head, y[..., rot:]], -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "axes":
        # the codes are bytes and the scales of rows that were rounded on the way: no such value
        return {"query": _rotated(s["query"], s["q_weight"], s), "k_codes": None, "v_codes": None,
                "k_scales": None, "v_scales": None}
    ps, g, d = case["ps"], case["g"], case["d"]
    o = torch.empty(s["query"].shape, dtype=torch.float64, device=DEVICE)
    lse = torch.empty(s["query"].shape[:2], dtype=torch.float64, device=DEVICE)
    row = 0
    for i, (n, new) in enumerate(zip(s["lens"], s["new"])):
        at = s["block_tables"][i, :-(-n // ps)].long()
        t = torch.arange(n, device=DEVICE)
        for h in range(case["hkv"]):
            kv = []
            for name in ("k", "v"):
                c, f = s[name + "_codes"], s[name + "_scales"]
                c, f = (c[at, :, h], f[at, :, h]) if case["layout"] == "NHD" else (c[at, h], f[at, h])
                kv.append(_real(c, f).flatten(0, 1)[:n])
            step = max(1, (1 << 27) // (g * n))
            for q0 in range(0, new, step):
                q1 = min(new, q0 + step)
                p = torch.arange(n - new + q0, n - new + q1, device=DEVICE)[:, None]
                dead = torch.zeros((q1 - q0, n), dtype=torch.bool, device=DEVICE)
                if case["causal"]:
                    dead |= t > p
                if case["window"] >= 0:
                    dead |= (p - t > case["window"]) & (t >= case["sink"])
                for k in range(h * g, (h + 1) * g):
                    x = s["query"][row + q0:row + q1, k].double() @ kv[0].T * (s["gk"].double() * case["d"] ** -0.5)
                    if case["cap"] > 0:
                        x = torch.tanh(x / case["cap"]) * case["cap"]
                    x = x.masked_fill(dead, -math.inf)
                    lse[row + q0:row + q1, k] = torch.logsumexp(x, -1)
                    o[row + q0:row + q1, k] = torch.softmax(x, -1) @ kv[1] * s["gv"].double()
        row += new
    return o, lse
