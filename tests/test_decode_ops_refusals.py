"""What the decode-step entry points refuse, on the CPU: every check comes before the first CUDA call,
so made-up addresses are never touched."""
import ctypes
import math

import pytest
import torch

import nvfp4_paged_kv_02_gb300 as nv

FAKE = 1 << 20
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    return nv.load()


def err(lib):
    return lib.nvfp4_last_error_string().decode()


def cache(ps=16, H=8, D=128, pages=4, data=FAKE, sf=FAKE, dstride=None, sstride=None):
    return nv._Cache(data, sf, ps * H * D // 2 if dstride is None else dstride,
                     ps * H * D // 16 if sstride is None else sstride, pages)


def append(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, dtype=1, nnz=4, Hq=32, H=8, D=128, qs=4096, ks=1024, vs=1024, qw=FAKE, kw=FAKE,
             eps=1e-6, cs=FAKE, npos=100, rot=128, inter=0, bi=FAKE, pos=FAKE, kc=cache(), vc=cache(), ps=16, layout=1,
             idx=FAKE, nidx=4, ptr=FAKE, last=None, B=2, ksc=1.0, vsc=1.0, kd=None, vd=None, recipe=None, out=FAKE,
             outs=4096)
    a.update(kw)
    return lib.nvfp4_qk_norm_rope_append_paged(
        P(a["q"]), P(a["k"]), P(a["v"]), a["dtype"], a["nnz"], a["Hq"], a["H"], a["D"], a["qs"], a["ks"], a["vs"],
        P(a["qw"]), P(a["kw"]), a["eps"], P(a["cs"]), a["npos"], a["rot"], a["inter"], P(a["bi"]), P(a["pos"]),
        a["kc"], a["vc"], a["ps"], a["layout"], P(a["idx"]), a["nidx"], P(a["ptr"]), P(a["last"]), a["B"], a["ksc"],
        a["vsc"], P(a["kd"]), P(a["vd"]), a["recipe"], P(a["out"]), a["outs"], None, None)


INV, UNS, ALI = nv.ERR_INVALID_ARG, nv.ERR_UNSUPPORTED, nv.ERR_ALIGNMENT


@pytest.mark.parametrize("kw,code,text", [
    (dict(D=24), INV, "head_dim"), (dict(D=528, rot=16, kc=cache(D=528), vc=cache(D=528)), UNS, "512"),
    (dict(Hq=0), INV, "num_qo_heads"), (dict(H=0), INV, "num_kv_heads"), (dict(ps=0), INV, "page_size"),
    (dict(layout=3), INV, "kv_layout"), (dict(dtype=2), INV, "dtype"), (dict(nnz=-1), INV, "negative"),
    (dict(eps=-1.0), INV, "eps"), (dict(eps=math.nan), INV, "eps"), (dict(rot=8), INV, "rotary_dim"),
    (dict(rot=144), INV, "rotary_dim"), (dict(rot=-16), INV, "rotary_dim"), (dict(inter=2), INV, "interleaved"),
    (dict(kd=FAKE), INV, "both"), (dict(ksc=0.0), INV, "positive finite"), (dict(vsc=math.inf), INV, "positive finite"),
    (dict(kd=FAKE + 2, vd=FAKE), ALI, "4-byte"), (dict(kc=cache(dstride=10)), INV, "data_page_stride"),
    (dict(vc=cache(data=FAKE + 8)), ALI, "16-byte"), (dict(q=None), INV, "query is null"),
    (dict(qs=4000), INV, "row stride"), (dict(ks=1028), ALI, "key"), (dict(v=FAKE + 2), ALI, "value"),
    (dict(out=FAKE + 4), ALI, "query_out"), (dict(outs=4104), INV, "in place"), (dict(out=None), INV, "query_out"),
    (dict(cs=None), INV, "null"), (dict(ptr=None), INV, "null"), (dict(idx=None), INV, "null"),
    (dict(qw=FAKE + 8), ALI, "weights"), (dict(cs=FAKE + 4), ALI, "cos_sin"), (dict(B=0), INV, "batch_size"),
    (dict(nidx=-1), INV, "num_kv_indices"), (dict(nnz=1 << 60), UNS, "2^40"),
])
def test_append_refuses(lib, kw, code, text):
    assert append(lib, **kw) == code
    assert text in err(lib)


def test_append_of_nothing(lib):
    assert append(lib, nnz=0, q=None, k=None, v=None, out=None) == nv.OK and err(lib) == ""


def bounds(lib, **kw):
    a = dict(kc=cache(), ps=16, H=8, D=128, layout=1, bt=FAKE, tdt=0, maxp=4, lens=FAKE, first=None, B=2, out=FAKE)
    a.update(kw)
    return lib.nvfp4_page_key_bounds(a["kc"], a["ps"], a["H"], a["D"], a["layout"], P(a["bt"]), a["tdt"], a["maxp"],
                                     P(a["lens"]), P(a["first"]), a["B"], P(a["out"]), None, None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(D=8), INV, "head_dim"), (dict(layout=-1), INV, "kv_layout"), (dict(tdt=2), INV, "table_dtype"),
    (dict(maxp=-1), INV, "negative"), (dict(B=16385), UNS, "batch_size"), (dict(bt=None), INV, "null"),
    (dict(lens=None), INV, "null"), (dict(out=None), INV, "null"), (dict(out=FAKE + 2), ALI, "key_bounds"),
    (dict(kc=cache(sstride=1)), INV, "sf_page_stride"),
])
def test_bounds_refuses(lib, kw, code, text):
    assert bounds(lib, **kw) == code
    assert text in err(lib)


def test_bounds_of_nothing(lib):
    assert bounds(lib, B=0) == nv.OK and bounds(lib, maxp=0) == nv.OK


def select(lib, **kw):
    a = dict(q=FAKE, dtype=0, qs=4096, Hq=32, H=8, D=128, kb=FAKE, pages=10, ps=16, bt=FAKE, tdt=0, maxp=4, lens=FAKE,
             B=2, k=8, sink=1, recent=1, sel=FAKE, num=FAKE, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return lib.nvfp4_select_pages(P(a["q"]), a["dtype"], a["qs"], a["Hq"], a["H"], a["D"], P(a["kb"]), a["pages"],
                                  a["ps"], P(a["bt"]), a["tdt"], a["maxp"], P(a["lens"]), a["B"], a["k"], a["sink"],
                                  a["recent"], P(a["sel"]), P(a["num"]), None, P(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(D=272), UNS, "256"), (dict(D=20), INV, "head_dim"), (dict(Hq=30), INV, "multiple"), (dict(dtype=5), INV, "dtype"),
    (dict(ps=0), INV, "page_size"), (dict(k=0), INV, "max_selected"), (dict(sink=-1), INV, "negative"),
    (dict(recent=-1), INV, "negative"), (dict(pages=-1), INV, "negative"), (dict(q=None), INV, "query"),
    (dict(qs=100), INV, "row stride"), (dict(q=FAKE + 8), ALI, "query"), (dict(kb=None), INV, "null"),
    (dict(sel=None), INV, "null"), (dict(kb=FAKE + 8), ALI, "key_bounds"), (dict(wsb=0), INV, "workspace"),
    (dict(ws=None), INV, "workspace"), (dict(ws=FAKE + 8), ALI, "workspace"), (dict(tdt=7), INV, "table_dtype"),
])
def test_select_refuses(lib, kw, code, text):
    assert select(lib, **kw) == code
    assert text in err(lib)


def attend(lib, **kw):
    a = dict(q=FAKE, dtype=0, qs=4096, Hq=32, kc=cache(), vc=cache(), ps=16, H=8, D=128, layout=1, bt=FAKE, tdt=0,
             maxp=4, lens=FAKE, B=2, ks=FAKE, vs=FAKE, sm=0.1, cap=0.0, win=-1, out=FAKE, lse=FAKE, ws=FAKE,
             wsb=1 << 40, sel=None, num=FAKE, S=None)
    a.update(kw)
    head = (P(a["q"]), a["dtype"], a["qs"], a["Hq"], a["kc"], a["vc"], a["ps"], a["H"], a["D"], a["layout"], P(a["bt"]),
            a["tdt"], a["maxp"], P(a["lens"]), a["B"])
    tail = (P(a["out"]), P(a["lse"]), None, P(a["ws"]), a["wsb"], None)
    if a["S"] is None:
        return lib.nvfp4_paged_attention_decode(*head, P(a["ks"]), P(a["vs"]), a["sm"], a["cap"], a["win"], *tail)
    return lib.nvfp4_sparse_paged_attention_decode(*head, P(a["sel"]), P(a["num"]), a["S"], P(a["ks"]), P(a["vs"]),
                                                   a["sm"], a["cap"], *tail)


@pytest.mark.parametrize("kw,code,text", [
    (dict(D=272, kc=cache(D=272), vc=cache(D=272)), UNS, "256"), (dict(D=24), INV, "head_dim"),
    (dict(Hq=36), INV, "multiple"), (dict(Hq=0), INV, "multiple"), (dict(dtype=3), INV, "dtype"),
    (dict(layout=2), INV, "kv_layout"), (dict(tdt=2), INV, "table_dtype"), (dict(maxp=-2), INV, "negative"),
    (dict(B=20000), UNS, "batch_size"), (dict(sm=math.nan), INV, "sm_scale"), (dict(sm=math.inf), INV, "sm_scale"),
    (dict(cap=-1.0), INV, "soft_cap"), (dict(cap=math.inf), INV, "soft_cap"), (dict(q=None), INV, "query"),
    (dict(qs=8), INV, "row stride"), (dict(q=FAKE + 2), ALI, "query"), (dict(out=None), INV, "out"),
    (dict(out=FAKE + 8), ALI, "out"), (dict(bt=None), INV, "null"), (dict(lens=None), INV, "null"),
    (dict(ks=None), INV, "null"), (dict(vs=FAKE + 1), ALI, "4-byte"), (dict(lse=FAKE + 2), ALI, "4-byte"),
    (dict(wsb=0), INV, "workspace"), (dict(ws=None), INV, "workspace"), (dict(ws=FAKE + 4), ALI, "workspace"),
    (dict(kc=cache(dstride=17000 * 16 + 8)), ALI, "16-byte"), (dict(vc=cache(pages=-1)), INV, "num_pages"),
    (dict(S=0, sel=FAKE), INV, "max_selected"), (dict(S=4, sel=None), INV, "null"), (dict(S=4, sel=FAKE, num=None), INV, "null"),
])
def test_attention_refuses(lib, kw, code, text):
    assert attend(lib, **kw) == code
    assert text in err(lib)


def test_attention_of_nothing(lib):
    assert attend(lib, B=0) == nv.OK and attend(lib, B=0, S=4) == nv.OK


def test_workspace_sizes(lib):
    n = ctypes.c_int64()
    assert lib.nvfp4_select_pages_workspace_bytes(2, 3, 100, ctypes.byref(n)) == nv.OK and n.value >= 2 * 3 * 100 * 4
    assert lib.nvfp4_select_pages_workspace_bytes(2, 0, 100, ctypes.byref(n)) == INV
    assert lib.nvfp4_paged_attention_workspace_bytes(32, 8, 128, ctypes.byref(n)) == nv.OK
    assert n.value >= nv.COUNTER_BYTES
    assert lib.nvfp4_paged_attention_workspace_bytes(32, 7, 128, ctypes.byref(n)) == INV
    assert lib.nvfp4_paged_attention_workspace_bytes(32, 8, 300, ctypes.byref(n)) == INV
    assert lib.nvfp4_paged_attention_workspace_bytes(32, 8, 512, ctypes.byref(n)) == UNS


def test_binding_takes_cuda_tensors_only():
    q = torch.zeros((1, 2, 64), dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int32)
    c = torch.zeros((1, 1, 16, 32), dtype=torch.uint8)
    s = torch.zeros((1, 1, 16, 4), dtype=torch.uint8)
    g = torch.ones(1)
    with pytest.raises(ValueError, match="CUDA"):
        nv.nvfp4_paged_attention_decode(q, (c, c), (s, s), i.view(1, 2), i[:1], g, g, "HND")
    with pytest.raises(ValueError, match="CUDA"):
        nv.nvfp4_select_pages(q, torch.zeros((1, 1, 2, 64), dtype=torch.float16), i.view(1, 2), i[:1], 16, 1)
    with pytest.raises(ValueError, match="CUDA"):
        nv.nvfp4_page_key_bounds(c, s, i.view(1, 2), i[:1], torch.zeros((1, 1, 2, 64), dtype=torch.float16))
    with pytest.raises(ValueError, match="CUDA"):
        nv.nvfp4_qk_norm_rope_append_paged(q, q, q, None, None, None, i, i, (c, c), (s, s), i, i, None, 1.0, 1.0)
