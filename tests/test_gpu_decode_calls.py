"""What the decode-step calls refuse by the tensors' properties (nothing is launched), and the forms
that their arguments may take."""
import numpy as np
import pytest
import torch

from tests import decode_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
H, G, D, PS = 2, 3, 64, 16


@pytest.fixture(scope="module", autouse=True)
def _cuda(gpu_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield


@pytest.fixture()
def s():
    """Arguments of every call, on a cache of two requests."""
    c = R.make_paged(3, [40, 17], H, D, PS, R.NHD)
    t = lambda a: torch.as_tensor(np.ascontiguousarray(a)).to(DEV)
    gen = torch.Generator(DEV).manual_seed(1)
    rand = lambda *n: torch.randn(n, generator=gen, device=DEV).half()
    pages = c.k.shape[0]
    return dict(k=t(c.k), v=t(c.v), ks=t(c.ks), vs=t(c.vs), tables=t(c.tables), lens=t(c.lens), q=rand(2, H * G, D),
                key=rand(2, H, D), value=rand(2, H, D), gk=torch.full((1,), 0.01, device=DEV),
                gv=torch.full((1,), 0.02, device=DEV), bounds=torch.zeros((pages, H, 2, D), dtype=torch.float16, device=DEV),
                w=torch.ones(D, dtype=torch.float16, device=DEV), table=torch.ones((64, D), device=DEV),
                req=torch.arange(2, dtype=torch.int32, device=DEV), pos=torch.tensor([39, 16], dtype=torch.int32, device=DEV),
                indices=t(c.tables).flatten().int().clamp(min=0), indptr=torch.tensor(
                    [0, c.tables.shape[1], 2 * c.tables.shape[1]], dtype=torch.int32, device=DEV),
                sel=torch.zeros((2, H, 4), dtype=torch.int32, device=DEV), num=torch.ones((2, H), dtype=torch.int32, device=DEV))


def _append(nv, s, **kw):
    s = dict(s, out=None, status=None, ks_=s["gk"], vs_=s["gv"], layout="NHD", last=None)
    s.update(kw)
    return nv.nvfp4_qk_norm_rope_append_paged(
        s["q"], s["key"], s["value"], s["w"], s.get("w2", s["w"]), s["table"], s["req"], s["pos"], (s["k"], s["v"]),
        (s["ks"], s["vs"]), s["indices"], s["indptr"], s["last"], s["ks_"], s["vs_"], s["layout"], out=s["out"],
        dev_status=s["status"])


def _bounds(nv, s, **kw):
    s = dict(s, first=None, status=None)
    s.update(kw)
    return nv.nvfp4_page_key_bounds(s["k"], s["ks"], s["tables"], s["lens"], s["bounds"], s["first"], "NHD",
                                    dev_status=s["status"])


def _select(nv, s, **kw):
    s = dict(s, out=None, status=None, n=4)
    s.update(kw)
    return nv.nvfp4_select_pages(s["q"], s["bounds"], s["tables"], s["lens"], PS, s["n"], out=s["out"],
                                 dev_status=s["status"])


def _dense(nv, s, **kw):
    s = dict(s, out=None, lse=None, status=None)
    s.update(kw)
    return nv.nvfp4_paged_attention_decode(s["q"], (s["k"], s["v"]), (s["ks"], s["vs"]), s["tables"], s["lens"], s["gk"],
                                           s["gv"], "NHD", out=s["out"], lse=s["lse"], dev_status=s["status"])


def _sparse(nv, s, **kw):
    s = dict(s, out=None, lse=None, status=None)
    s.update(kw)
    return nv.nvfp4_sparse_paged_attention_decode(
        s["q"], (s["k"], s["v"]), (s["ks"], s["vs"]), s["tables"], s["lens"], s["sel"], s["num"], s["gk"], s["gv"], "NHD",
        out=s["out"], lse=s["lse"], dev_status=s["status"])


CHANGES = {
    # argument: what is wrong with it
    "q": [lambda x: x.float(), lambda x: x[0], lambda x: x.cpu(), lambda x: x[..., :48], lambda x: x.transpose(0, 1),
          lambda x: x[..., ::2]],
    "key": [lambda x: x.bfloat16(), lambda x: x[:1], lambda x: x[:, :1], lambda x: x.cpu()],
    "value": [lambda x: x.bfloat16(), lambda x: x[:, :, :48]],
    "w": [lambda x: x.float(), lambda x: x[:48], lambda x: x.cpu()],
    "table": [lambda x: x.half(), lambda x: x.flatten(), lambda x: x[:, ::2]],
    "req": [lambda x: x.long(), lambda x: x[:1]],
    "pos": [lambda x: x.long(), lambda x: x.repeat(2)[::2][:1]],
    "k": [lambda x: x[0], lambda x: x.transpose(1, 2), lambda x: x.int(), lambda x: x.cpu(), lambda x: x[:-1]],
    "v": [lambda x: x[..., :24], lambda x: x.cpu()],
    "ks": [lambda x: x[..., :2], lambda x: x.int(), lambda x: x[:-1], lambda x: x.cpu()],
    "vs": [lambda x: x[:, :-1], lambda x: x.half()],
    "indices": [lambda x: x.long(), lambda x: x[::2]],
    "indptr": [lambda x: x.long(), lambda x: x.cpu()],
    "ks_": [lambda x: x.double(), lambda x: x.cpu()],
    "last": [lambda x: torch.ones(1, dtype=torch.int32, device=DEV), lambda x: torch.ones(2, device=DEV)],
    "tables": [lambda x: x.short(), lambda x: x[:1], lambda x: x.t(), lambda x: x[0], lambda x: x.cpu()],
    "lens": [lambda x: x.long(), lambda x: x[:1], lambda x: x.cpu()],
    "bounds": [lambda x: x.float(), lambda x: x[:, :, 0], lambda x: x[..., :48], lambda x: x.transpose(0, 1), lambda x: x.cpu()],
    "first": [lambda x: torch.zeros(1, dtype=torch.int32, device=DEV), lambda x: torch.zeros(2, device=DEV)],
    "gk": [lambda x: x.double(), lambda x: 0.01],
    "gv": [lambda x: x.cpu(), lambda x: x[:0]],
    "sel": [lambda x: x.long(), lambda x: x[:1], lambda x: x[0], lambda x: x[:, :, ::2]],
    "num": [lambda x: x.long(), lambda x: x[:, :1], lambda x: x[0]],
    "lse": [lambda x: torch.empty((2, H * G), device=DEV).half(), lambda x: torch.empty((1, H * G), device=DEV)],
    "status": [lambda x: torch.zeros(1, device=DEV), lambda x: torch.zeros(1, dtype=torch.int32)],
    "n": [lambda x: 2 ** 40],
}
CALLS = {
    "append": (_append, ["q", "key", "value", "w", "table", "req", "pos", "k", "v", "ks", "vs", "indices", "indptr", "ks_",
                         "last", "status"]),
    "bounds": (_bounds, ["k", "ks", "tables", "lens", "bounds", "first", "status"]),
    "select": (_select, ["q", "bounds", "tables", "lens", "n", "status"]),
    "dense": (_dense, ["q", "k", "v", "ks", "vs", "tables", "lens", "gk", "gv", "lse", "status"]),
    "sparse": (_sparse, ["q", "tables", "lens", "sel", "num", "gk", "gv", "lse", "status"]),
}

@pytest.mark.parametrize("call,name,i", [(c, n, i) for c, (_, names) in CALLS.items() for n in names
                                         for i in range(len(CHANGES[n]))])
def test_refusals(gpu_lib, s, call, name, i):
    before = {k: v.clone() for k, v in s.items()}
    value = s.get(name, s["gk"] if name == "ks_" else None)
    with pytest.raises(ValueError):
        CALLS[call][0](gpu_lib, s, **{name: CHANGES[name][i](value)})
    torch.cuda.synchronize()
    for k, v in s.items():
        assert torch.equal(v, before[k]), k


def test_forms_of_the_arguments(gpu_lib, s):
    nv = gpu_lib
    want, want_lse = _dense(nv, s)
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    got = _dense(nv, s, out=out, lse=lse)
    assert got[0].data_ptr() == out.data_ptr() and got[1].data_ptr() == lse.data_ptr()
    same = [
        got,
        _dense(nv, s, tables=s["tables"].long()),
        _dense(nv, s, ks=s["ks"].view(torch.float8_e4m3fn), vs=s["vs"].view(torch.float8_e4m3fn)),
        nv.nvfp4_paged_attention_decode(s["q"], [s["k"], s["v"]], torch.stack([s["ks"], s["vs"]], 1), s["tables"], s["lens"],
                                        s["gk"], s["gv"], 0, sm_scale=D ** -0.5),
    ]
    for o, l in same:
        assert torch.equal(o, want) and torch.equal(l, want_lse)
    assert _dense(nv, s, q=s["q"][:0], tables=s["tables"][:0], lens=s["lens"][:0])[0].shape == (0, H * G, D)
    # scales by value and in device memory; a Parameter for weights
    a = _append(nv, s)
    k = s["k"].clone(), s["ks"].clone()
    b = _append(nv, s, ks_=float(s["gk"]), vs_=float(s["gv"]), w=torch.nn.Parameter(s["w"]))
    assert torch.equal(a, b) and torch.equal(k[0], s["k"]) and torch.equal(k[1], s["ks"])
    with pytest.raises(nv.NVFP4KVError):  # what the library itself refuses
        _append(nv, s, ks_=-1.0, vs_=1.0)
    with pytest.raises(nv.NVFP4KVError):
        _select(nv, s, n=0)
    with pytest.raises(TypeError):
        _append(nv, s, ks_="1", vs_=1.0)
    with pytest.raises(KeyError):
        _append(nv, s, layout="DHN")
