"""Norm, rotation and append in one pass: query rows and cache bytes are exactly those of the
operator's binary32 order (tests/decode_reference.py) followed by the CPU oracle's append; the
norm and rotation themselves against 64 bits."""
import numpy as np
import pytest
import torch

import oracle as O
import workloads as W
from tests import decode_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
SENT = 0xA5


@pytest.fixture(scope="module", autouse=True)
def _cuda(gpu_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield


def _t(a):
    return torch.as_tensor(np.ascontiguousarray(a)).to(DEV)


class Case:
    def __init__(self, seed, nnz, Hq, H, D, ps, layout, dtype, rot, inter=False, recipe=None, norm=(True, True),
                 fused=True, B=3, gs=(0.004, 0.003)):
        self.__dict__.update({k: v for k, v in locals().items() if k != "self"})
        rng = np.random.Generator(np.random.PCG64(seed))
        g = torch.Generator().manual_seed(seed)
        self.rows = [(torch.randn((nnz, h, D), generator=g) * (1 + 5 * (torch.rand((h, D), generator=g) < 0.05))
                      ).to(dtype) for h in (Hq, H, H)]
        self.w = [(1 + 0.3 * torch.randn(D, generator=g)).to(dtype) if n else None for n in norm]
        self.table = R.cos_sin(200, rot) if rot else None
        # nnz different (request, position) pairs, in any order
        pairs = rng.permutation(B * 200)[:nnz]
        self.bi, self.pos = (pairs // 200).astype(np.int32), (pairs % 200).astype(np.int32)
        per = -(-200 // ps)
        self.P = B * per + 2
        self.indices = rng.permutation(self.P)[: B * per].astype(np.int32)
        self.indptr = (np.arange(B + 1) * per).astype(np.int32)

    def expect(self):
        """(query rows as 16-bit patterns, K and V caches) by the reference and the oracle."""
        bf16 = self.dtype == torch.bfloat16
        out = []
        for x, w in zip(self.rows[:2], self.w):
            y = R.norm_rope(x.float().numpy(), None if w is None else w.float().numpy(), 1e-5, self.table, self.pos,
                            self.inter)
            out.append(torch.from_numpy(np.ascontiguousarray(y)).to(self.dtype))
        dps, sps = self.ps * self.H * self.D // 2, self.ps * self.H * self.D // 16
        kc, vc = (O.PagedCache(np.full(self.P * dps, SENT, np.uint8), np.full(self.P * sps, SENT, np.uint8), dps, sps)
                  for _ in range(2))
        HD = self.H * self.D
        gk, gv = (float(np.float32(g)) for g in self.gs)
        r = None if self.recipe is None else O.Recipe(*self.recipe)
        if self.nnz:
            O.quantize_append_paged(W.bits16(out[1]), W.bits16(self.rows[2]), bf16, self.nnz, self.H, self.D, HD, HD,
                                    self.bi, self.pos, kc, vc, self.ps, self.layout, self.indices, self.indptr, gk,
                                    gv, r, 0)
        return out[0], kc, vc

    def call(self, nv, out=None, status=None, **kw):
        inner = (self.ps, self.H) if self.layout == R.NHD else (self.H, self.ps)
        c = [torch.full((self.P, *inner, self.D // n), SENT, dtype=torch.uint8, device=DEV) for n in (2, 2, 16, 16)]
        if self.fused:
            qkv = torch.cat(self.rows, 1).to(DEV)
            q, k, v = qkv.split([self.Hq, self.H, self.H], 1)
        else:
            q, k, v = (x.to(DEV) for x in self.rows)
        if out == "in place":
            out = q
        r = None if self.recipe is None else nv.NVFP44Over6Config(
            self.recipe[0], "MSE" if self.recipe[1] else "MAE", bool(self.recipe[2]))
        gk, gv = ((_t(np.array([g], np.float32)) for g in self.gs) if self.fused else self.gs)
        got = nv.nvfp4_qk_norm_rope_append_paged(
            q, k, v, *(None if w is None else w.to(DEV) for w in self.w),
            None if self.table is None else _t(self.table), kw.pop("bi", _t(self.bi)), kw.pop("pos", _t(self.pos)),
            (c[0], c[1]), (c[2], c[3]), kw.pop("indices", _t(self.indices)), _t(self.indptr), kw.pop("last", None),
            gk, gv, "NHD" if self.layout == R.NHD else "HND", eps=1e-5, rotary_interleaved=self.inter,
            nvfp4_4over6=r, out=out, dev_status=status)
        torch.cuda.synchronize()
        return got, [x.cpu().numpy().reshape(-1) for x in c]


def _same(case, got, caches, want):
    q, kc, vc = want
    assert np.array_equal(W.bits16(got.cpu()), W.bits16(q)), "query rows"
    for name, a, b in (("K codes", caches[0], kc.data), ("V codes", caches[1], vc.data), ("K scales", caches[2], kc.sf),
                       ("V scales", caches[3], vc.sf)):
        bad = np.flatnonzero(a != b)
        assert bad.size == 0, f"{name}: {bad.size} bytes differ, first at {bad[0]}"


CASES = [
    # seed, nnz, Hq, H, D, ps, layout, dtype, rot, inter, recipe, norm, fused
    (1, 1, 1, 1, 16, 2, R.NHD, torch.float16, 16),
    (2, 64, 32, 8, 128, 16, R.HND, torch.bfloat16, 128),
    (3, 33, 10, 2, 128, 16, R.NHD, torch.float16, 64, True),
    (4, 17, 6, 3, 64, 12, R.HND, torch.bfloat16, 64, True, (256.0, 0, 0)),
    (5, 50, 5, 1, 80, 6, R.NHD, torch.float16, 80, False, (256.0, 1, 0)),
    (6, 9, 4, 4, 96, 16, R.HND, torch.bfloat16, 32, False, (448.0, 0, 1)),
    (7, 21, 7, 1, 192, 64, R.NHD, torch.float16, 192, False, (256.0, 1, 1)),
    (8, 13, 8, 2, 256, 16, R.HND, torch.bfloat16, 256),
    (9, 5, 3, 1, 512, 4, R.NHD, torch.float16, 64, True),
    (10, 40, 4, 2, 128, 16, R.HND, torch.bfloat16, 0),
    (11, 40, 4, 2, 128, 16, R.HND, torch.float16, 128, False, None, (False, False)),
    (12, 40, 4, 2, 64, 16, R.NHD, torch.bfloat16, 48, True, None, (True, False), False),
    (13, 40, 4, 2, 64, 16, R.NHD, torch.bfloat16, 0, False, None, (False, False), False),
    (14, 550, 16, 4, 128, 32, R.NHD, torch.bfloat16, 128, False, (256.0, 0, 1)),
    (15, 0, 4, 2, 64, 16, R.NHD, torch.bfloat16, 64),
    (16, 31, 9, 5, 112, 16, R.HND, torch.float16, 96),
    (17, 31, 3, 3, 32, 16, R.HND, torch.float16, 16),
]


MANY = [  # a warp for all rows of a token; key and value rows in one step, or in steps of their own
    (18, 3500, 6, 3, 64, 16, R.NHD, torch.bfloat16, 64),
    (19, 3300, 3, 1, 128, 16, R.HND, torch.float16, 128, True, (256.0, 0, 0)),
    (20, 3300, 2, 6, 128, 32, R.NHD, torch.bfloat16, 64, False, (256.0, 1, 1)),
    (21, 3300, 4, 4, 128, 16, R.HND, torch.bfloat16, 128),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_same_bytes_as_norm_rotation_then_append(gpu_lib, i):
    case = Case(*CASES[i])
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    got, caches = case.call(gpu_lib, status=st)
    assert int(st.item()) == 0
    _same(case, got, caches, case.expect())


@pytest.mark.parametrize("i", range(len(MANY)))
def test_many_tokens(gpu_lib, i):
    case = Case(*MANY[i], B=20)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    got, caches = case.call(gpu_lib, status=st)
    assert int(st.item()) == 0
    _same(case, got, caches, case.expect())


@pytest.mark.parametrize("i", [1, 4, 8])
def test_in_place_and_given_output(gpu_lib, i):
    case = Case(*CASES[i])
    want = case.expect()
    _same(case, *case.call(gpu_lib, out="in place"), want)
    wide = torch.zeros((case.nnz, case.Hq + 3, case.D), dtype=case.dtype, device=DEV)
    got, caches = case.call(gpu_lib, out=wide[:, 1:case.Hq + 1])
    _same(case, got.contiguous(), caches, want)
    assert (wide[:, 0] == 0).all() and (wide[:, -2:] == 0).all()


@pytest.mark.parametrize("i", [1, 2, 4, 7])
def test_near_the_formula_in_64_bits(gpu_lib, i):
    case = Case(*CASES[i])
    got, _ = case.call(gpu_lib)
    x, w = case.rows[0].double().numpy(), case.w[0].double().numpy()
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5) * w
    rot = case.table.shape[1]
    c, s = (t[:, None].astype(np.float64) for t in np.split(case.table[case.pos], 2, -1))
    ia = np.arange(0, rot, 2) if case.inter else np.arange(rot // 2)
    ib = ia + (1 if case.inter else rot // 2)
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    size = np.abs(y)
    size[..., ia] = size[..., ib] = np.abs(a) + np.abs(b)
    # about D/8 + 12 operations of 2^-24 each, then one rounding
    tol = torch.finfo(case.dtype).eps / 2 * np.abs(y) + (case.D / 8 + 12) * 2.0 ** -24 * size + 2.0 ** -25
    assert (np.abs(got.double().cpu().numpy() - y) <= tol * 1.01).all()


def test_rows_that_have_no_place(gpu_lib):
    """Bad requests, positions past the table or the described space, pages outside the pool: reported,
    and every other row is as it would be without them."""
    nv = gpu_lib
    case = Case(30, 64, 4, 2, 128, 16, R.HND, torch.bfloat16, 128)
    q, kc, vc = case.expect()
    bi, pos, indices = case.bi.copy(), case.pos.copy(), case.indices.copy()
    bi[3], bi[4] = -1, 7                       # no such request: the query row is still written
    pos[10], pos[11] = -2, 1 << 20             # outside the rotation table: nothing is written
    last = np.array([200 - 16 * 12] * 3, np.int32)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    sent = torch.full((64, 4, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    got, caches = case.call(nv, out=sent, status=st, bi=_t(bi), pos=_t(pos), last=_t(last))
    assert int(st.item()) == nv.DEV_BAD_BATCH | nv.DEV_BAD_POSITION
    keep = np.ones(64, bool)
    keep[[10, 11]] = False
    assert torch.equal(got.cpu()[keep], q[keep]) and (got[[10, 11]] == 3.0).all()
    per = len(indices) // 3
    for i in (3, 4, 10, 11):
        page, slot = indices[case.bi[i] * per + case.pos[i] // 16], case.pos[i] % 16
        for name, c in (("k", kc), ("v", vc)):
            c.data.reshape(case.P, 2, 16, 64)[page, :, slot] = SENT
            c.sf.reshape(case.P, 2, 16, 8)[page, :, slot] = SENT
    for a, b in zip(caches, (kc.data, vc.data, kc.sf, vc.sf)):
        assert np.array_equal(a, b)
    indices[:] = case.P + 5
    st.zero_()
    got, caches = case.call(nv, status=st, indices=_t(indices))
    assert int(st.item()) == nv.DEV_BAD_PAGE and all((c == SENT).all() for c in caches)
    assert torch.equal(got.cpu(), q)


def test_device_scale_that_is_not_positive_finite(gpu_lib):
    nv = gpu_lib
    for bad in (0.0, -1.0, float("inf"), float("nan")):
        case = Case(31, 5, 4, 2, 64, 16, R.HND, torch.float16, 64, gs=(bad, 0.01))
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        _, caches = case.call(nv, status=st)
        assert int(st.item()) == nv.DEV_BAD_SCALE and all((c == SENT).all() for c in caches)


def test_zero_rows(gpu_lib):
    case = Case(32, 20, 4, 2, 128, 16, R.NHD, torch.bfloat16, 128)
    for x in case.rows:
        x[::2] = 0
    _same(case, *case.call(gpu_lib), case.expect())


def test_captured_graph(gpu_lib):
    nv = gpu_lib
    case = Case(33, 30, 8, 2, 128, 16, R.HND, torch.bfloat16, 128)
    q, k, v = (x.to(DEV) for x in case.rows)
    c = [torch.full((case.P, 2, 16, 128 // n), SENT, dtype=torch.uint8, device=DEV) for n in (2, 2, 16, 16)]
    w, tab, bi, pos, idx, ptr = (case.w[0].to(DEV), _t(case.table), _t(case.bi), _t(case.pos), _t(case.indices),
                                 _t(case.indptr))
    kw = case.w[1].to(DEV)
    call = lambda: nv.nvfp4_qk_norm_rope_append_paged(q, k, v, w, kw, tab, bi, pos, (c[0], c[1]), (c[2], c[3]), idx,
                                                      ptr, None, *case.gs, "HND", eps=1e-5)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    for x in c:
        x.fill_(SENT)
    g.replay()
    torch.cuda.synchronize()
    _same(case, out, [x.cpu().numpy().reshape(-1) for x in c], case.expect())
