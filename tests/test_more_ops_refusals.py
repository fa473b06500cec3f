"""What the entry points of prompts, of windows with first tokens and of positions with several axes refuse,
on the CPU: every check comes before the first CUDA call, so made-up addresses are never touched."""
import math

import pytest
import torch

import nvfp4_paged_kv_02_gb300 as nv
from tests.test_decode_ops_refusals import ALI, FAKE, INV, P, UNS, cache, err


@pytest.fixture(scope="module")
def lib():
    return nv.load()


def axes(lib, **kw):
    a = dict(q=FAKE, D=128, cs=FAKE, rot=128, inter=0, ap=FAKE, na=3, pa=FAKE, pos=FAKE, nnz=4, kc=cache(), vc=cache(), B=2)
    a.update(kw)
    return lib.nvfp4_qk_norm_rope_axes_append_paged(
        P(a["q"]), P(FAKE), P(FAKE), 1, a["nnz"], 32, 8, a["D"], 4096, 1024, 1024, P(FAKE), P(FAKE), 1e-6, P(a["cs"]),
        100, a["rot"], a["inter"], P(a["ap"]), a["na"], P(a["pa"]), P(FAKE), P(a["pos"]), a["kc"], a["vc"], 16, 1, P(FAKE),
        4, P(FAKE), None, a["B"], 1.0, 1.0, None, None, None, P(FAKE), 4096, None, None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(na=0), INV, "num_rotary_axes"), (dict(na=9), INV, "num_rotary_axes"), (dict(na=-1), INV, "num_rotary_axes"),
    (dict(ap=None), INV, "null"), (dict(pa=None), INV, "null"), (dict(cs=None), INV, "null"), (dict(pos=None), INV, "null"),
    (dict(ap=FAKE + 2), ALI, "rotary_positions"), (dict(pa=FAKE + 1), ALI, "pair_axes"), (dict(rot=24), INV, "rotary_dim"),
    (dict(D=24), INV, "head_dim"), (dict(q=None), INV, "query is null"), (dict(inter=2), INV, "interleaved"),
])
def test_axes_refuse(lib, kw, code, text):
    assert axes(lib, **kw) == code
    assert text in err(lib) and "nvfp4_qk_norm_rope_axes_append_paged" in err(lib)


def test_append_of_nothing_with_axes(lib):
    assert axes(lib, nnz=0, q=None, ap=None, pa=None) == nv.OK and err(lib) == ""


def test_axis_of_pairs():
    assert nv.nvfp4_rotary_axes([2, 3, 1], device="cpu").tolist() == [0, 0, 1, 1, 1, 2]
    assert nv.nvfp4_rotary_axes([2, 3, 1], in_turn=True, device="cpu").tolist() == [0, 1, 2, 0, 1, 1]
    assert nv.nvfp4_rotary_axes([4], device="cpu").tolist() == [0] * 4
    assert nv.nvfp4_rotary_axes([0, 2], device="cpu").dtype == torch.uint8
    for bad in ([], [1] * 9, [3, -1]):
        with pytest.raises(ValueError, match="sections"):
            nv.nvfp4_rotary_axes(bad, device="cpu")


def sinks(lib, **kw):
    a = dict(q=FAKE, window=10, sink=4, sm=0.1, cap=0.0, B=2, lens=FAKE, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return lib.nvfp4_paged_attention_decode_sinks(
        P(a["q"]), 1, 4096, 32, cache(), cache(), 16, 8, 128, 1, P(FAKE), 0, 4, P(a["lens"]), a["B"], P(FAKE), P(FAKE),
        a["sm"], a["cap"], a["window"], a["sink"], P(FAKE), P(FAKE), None, P(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(sink=-1), INV, "num_sink_tokens"), (dict(sink=-2 ** 31), INV, "num_sink_tokens"), (dict(sm=math.inf), INV, "sm_scale"),
    (dict(q=None), INV, "query"), (dict(wsb=100), INV, "workspace"), (dict(ws=FAKE + 8), ALI, "workspace"),
    (dict(B=16385), UNS, "batch_size"),
])
def test_sinks_refuse(lib, kw, code, text):
    assert sinks(lib, **kw) == code
    assert text in err(lib) and "nvfp4_paged_attention_decode_sinks" in err(lib)


def test_sinks_of_nothing(lib):
    assert sinks(lib, B=0) == nv.OK


def prefill(lib, **kw):
    a = dict(q=FAKE, dtype=1, nnz=9, qs=4096, Hq=32, H=8, ptr=FAKE, kc=cache(), vc=cache(), ps=16, D=128, layout=1, bt=FAKE, tdt=0,
             maxp=4, lens=FAKE, B=2, ks=FAKE, vs=FAKE, causal=1, sm=0.1, cap=0.0, window=-1, sink=0, out=FAKE, lse=FAKE, ws=FAKE,
             wsb=1 << 40)
    a.update(kw)
    return lib.nvfp4_paged_attention_prefill(
        P(a["q"]), a["dtype"], a["nnz"], a["qs"], a["Hq"], P(a["ptr"]), a["kc"], a["vc"], a["ps"], a["H"], a["D"], a["layout"],
        P(a["bt"]), a["tdt"], a["maxp"], P(a["lens"]), a["B"], P(a["ks"]), P(a["vs"]), a["causal"], a["sm"], a["cap"], a["window"],
        a["sink"], P(a["out"]), P(a["lse"]), None, P(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(D=24), INV, "head_dim"), (dict(D=272, kc=cache(D=272), vc=cache(D=272)), UNS, "256"), (dict(dtype=2), INV, "dtype"),
    (dict(Hq=0), INV, "num_qo_heads"), (dict(Hq=31), INV, "num_qo_heads"), (dict(H=0), INV, "num_kv_heads"), (dict(ps=0), INV, "page_size"),
    (dict(layout=2), INV, "kv_layout"), (dict(tdt=3), INV, "table_dtype"), (dict(maxp=-1), INV, "negative"), (dict(B=-1), INV, "negative"),
    (dict(nnz=-1), INV, "negative"), (dict(B=16385), UNS, "batch_size"), (dict(causal=2), INV, "causal"), (dict(sm=math.nan), INV, "sm_scale"),
    (dict(cap=-1.0), INV, "soft_cap"), (dict(cap=math.inf), INV, "soft_cap"), (dict(sink=-1), INV, "num_sink_tokens"),
    (dict(q=None), INV, "query is null"), (dict(qs=4000), INV, "row stride"), (dict(qs=4100), ALI, "query"), (dict(q=FAKE + 8), ALI, "query"),
    (dict(out=None), INV, "out is null"), (dict(out=FAKE + 8), ALI, "out"), (dict(lse=FAKE + 2), ALI, "lse"), (dict(ks=FAKE + 1), ALI, "scales"),
    (dict(ptr=None), INV, "null"), (dict(lens=None), INV, "null"), (dict(bt=None), INV, "null"), (dict(vs=None), INV, "null"),
    (dict(kc=cache(data=FAKE + 8)), ALI, "k_cache"), (dict(vc=cache(dstride=10)), INV, "v_cache"), (dict(kc=cache(pages=1 << 31), vc=cache(pages=1 << 31)), UNS, "pages"),
    (dict(nnz=1 << 31), UNS, "query rows"), (dict(nnz=1 << 29), UNS, "query rows"),
    (dict(maxp=(1 << 31) - 1), UNS, "positions"), (dict(maxp=1 << 27), UNS, "positions"), (dict(ws=None), INV, "workspace"), (dict(wsb=1000), INV, "workspace"), (dict(ws=FAKE + 8), ALI, "workspace"),
])
def test_prefill_refuses(lib, kw, code, text):
    assert prefill(lib, **kw) == code
    assert text in err(lib) and "nvfp4_paged_attention_prefill" in err(lib)


def test_prefill_of_nothing(lib):
    assert prefill(lib, nnz=0, q=None, out=None) == nv.OK and prefill(lib, B=0) == nv.OK


def test_prefill_workspace_size(lib):
    import ctypes
    n = ctypes.c_int64()
    f = lib.nvfp4_paged_attention_prefill_workspace_bytes
    assert f(128, ctypes.byref(n)) == nv.OK and n.value >= nv.COUNTER_BYTES
    assert f(72, ctypes.byref(n)) == INV and f(0, ctypes.byref(n)) == INV and f(272, ctypes.byref(n)) == UNS and f(64, None) == INV


def test_prefill_takes_cuda_tensors_only():
    q = torch.zeros((1, 2, 64), dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int32)
    c = torch.zeros((1, 1, 16, 32), dtype=torch.uint8)
    s = torch.zeros((1, 1, 16, 4), dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        nv.nvfp4_paged_attention_prefill(q, (c, c), (s, s), i, i.view(1, 2), i[:1], torch.ones(1), torch.ones(1), "HND")
