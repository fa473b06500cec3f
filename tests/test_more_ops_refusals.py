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
