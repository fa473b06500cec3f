"""Attention of one new token per request over the paged NVFP4 cache, dense and over selected
pages, against the 64-bit reference (tests/decode_reference.py), with the slots that no position
owns full of NaN scales."""
import numpy as np
import pytest
import torch

from tests import decode_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _cuda(gpu_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield


def _dev(c: R.Paged, pad_data=0, pad_sf=0, off_sf=0):
    """The caches on the device, with spare bytes between pages and an offset of the scales."""
    def put(x, pad, off):
        P, n = x.shape[0], x[0].size
        buf = torch.full((P * (n + pad) + off,), 0x7F, dtype=torch.uint8, device=DEV)
        t = buf[off:].as_strided(x.shape, (n + pad, x[0, 0].size, x.shape[3], 1))
        t.copy_(torch.as_tensor(x).to(DEV))
        return t
    return ((put(c.k, pad_data, 0), put(c.v, pad_data, 0)),
            (put(c.ks, pad_sf, off_sf), put(c.vs, pad_sf, off_sf)))


def _query(seed, B, Hq, D, dtype, scale=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((B, Hq, D), generator=g) * scale).to(dtype)


def _layout(c):
    return "NHD" if c.layout == R.NHD else "HND"


def _run(nv, c, q, dev=None, status=None, **kw):
    caches, sf = dev or _dev(c)
    st = torch.zeros(1, dtype=torch.int32, device=DEV) if status is None else status
    gk, gv = (torch.tensor([x], dtype=torch.float32, device=DEV) for x in (c.gk, c.gv))
    args = [q.to(DEV) if not q.is_cuda else q, caches, sf, torch.as_tensor(c.tables).to(DEV),
            torch.as_tensor(c.lens).to(DEV)]
    fn = nv.nvfp4_paged_attention_decode
    if "selected" in kw:
        fn = nv.nvfp4_sparse_paged_attention_decode
        args += [torch.as_tensor(kw.pop("selected")).to(DEV), torch.as_tensor(kw.pop("num_selected")).to(DEV)]
    out, lse = fn(*args, gk, gv, _layout(c), dev_status=st, **kw)
    torch.cuda.synchronize()
    return out, lse, int(st.item())


def _ref(c, q, sm=None, **kw):
    f32 = R.Paged(**{**c.__dict__, "gk": float(np.float32(c.gk)), "gv": float(np.float32(c.gv))})
    return R.attention(f32, q.double().numpy(), q.shape[-1] ** -0.5 if sm is None else sm, **kw)


CASES = [
    # lens, H, G, D, ps, layout, dtype
    ([1], 1, 1, 16, 2, R.NHD, torch.float16),
    ([0, 1, 2], 2, 1, 64, 16, R.HND, torch.bfloat16),
    ([0], 1, 4, 128, 16, R.HND, torch.float16),
    ([37, 64, 5], 2, 4, 64, 16, R.NHD, torch.bfloat16),
    ([31, 32, 33, 127, 128, 129], 2, 8, 128, 16, R.HND, torch.bfloat16),
    ([255, 256, 257, 511], 1, 7, 128, 64, R.NHD, torch.float16),
    ([300, 17], 3, 5, 96, 12, R.HND, torch.float16),
    ([200, 90], 2, 3, 80, 7, R.NHD, torch.bfloat16),
    ([130, 70], 2, 2, 48, 5, R.HND, torch.float16),
    ([77, 400], 1, 16, 128, 16, R.NHD, torch.bfloat16),
    ([333], 2, 9, 64, 32, R.HND, torch.float16),
    ([150, 1], 1, 12, 192, 8, R.NHD, torch.float16),
    ([260, 31], 2, 8, 256, 16, R.HND, torch.bfloat16),
    ([140], 1, 20, 256, 100, R.NHD, torch.float16),
    ([90, 65], 1, 33, 112, 4, R.HND, torch.bfloat16),
    ([4097, 3000, 1], 1, 4, 128, 16, R.HND, torch.float16),
    ([5000], 2, 1, 32, 3, R.NHD, torch.bfloat16),
    ([100] * 70, 3, 2, 64, 16, R.HND, torch.float16),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_dense_matches_reference(gpu_lib, i):
    lens, H, G, D, ps, layout, dtype = CASES[i]
    c = R.make_paged(i, lens, H, D, ps, layout)
    q = _query(i, c.B, H * G, D, dtype)
    out, lse, status = _run(gpu_lib, c, q)
    R.check_attention(out, lse, _ref(c, q), dtype)
    assert status == 0


@pytest.mark.parametrize("lens,H,D", [
    ([0, 700, 30, 390, 384, 385, 1, 416] * 12, 8, 64),   # more lists than CTAs, cut and whole ones mixed
    ([383, 384, 385, 3000], 1, 128),                     # twelve units and one more
    ([32 * n for n in range(15)], 2, 64),
    ([1] * 300, 2, 32),
])
def test_lists_about_the_length_that_is_cut(gpu_lib, lens, H, D):
    c = R.make_paged(len(lens), lens, H, D, 16, R.HND)
    q = _query(2, c.B, H * 2, D, torch.float16)
    out, lse, status = _run(gpu_lib, c, q)
    R.check_attention(out, lse, _ref(c, q), q.dtype)
    assert status == 0


@pytest.mark.parametrize("layout", [R.NHD, R.HND])
@pytest.mark.parametrize("D,off_sf,pad_sf,pad_data", [(128, 0, 16, 32), (128, 1, 3, 0), (128, 4, 4, 16),
                                                     (64, 2, 2, 0), (64, 0, 5, 48), (256, 8, 0, 0), (96, 0, 0, 16),
                                                     (32, 1, 1, 0)])
def test_strides_and_alignment(gpu_lib, layout, D, off_sf, pad_sf, pad_data):
    c = R.make_paged(40 + D, [75, 160, 33], 2, D, 16, layout, table_dtype=np.int64)
    q = _query(5, 3, 8, D, torch.bfloat16)
    wide = torch.zeros((3, 12, D), dtype=q.dtype, device=DEV)
    wide[:, 2:10] = q.to(DEV)
    out, lse, status = _run(gpu_lib, c, q, _dev(c, pad_data, pad_sf, off_sf))
    out2, lse2, _ = _run(gpu_lib, c, wide[:, 2:10], _dev(c, pad_data, pad_sf, off_sf))
    R.check_attention(out, lse, _ref(c, q), q.dtype)
    assert torch.equal(out, out2) and torch.equal(lse, lse2) and status == 0


def test_stacked_cache(gpu_lib):
    c = R.make_paged(7, [100, 3, 64], 4, 128, 16, R.HND)
    q = _query(7, 3, 8, 128, torch.float16)
    st = lambda a, b: torch.stack([torch.as_tensor(a), torch.as_tensor(b)], 1).to(DEV)
    out, lse, _ = _run(gpu_lib, c, q, (st(c.k, c.v), st(c.ks, c.vs)))
    R.check_attention(out, lse, _ref(c, q), q.dtype)


@pytest.mark.parametrize("window", [0, 1, 31, 32, 100, 5000])
@pytest.mark.parametrize("D", [64, 128])
def test_window(gpu_lib, window, D):
    c = R.make_paged(window, [0, 1, 33, 250, 700], 2, D, 16, R.NHD)
    q = _query(window, 5, 6, D, torch.float16)
    out, lse, _ = _run(gpu_lib, c, q, window_left=window)
    R.check_attention(out, lse, _ref(c, q, window=window), q.dtype)


@pytest.mark.parametrize("cap", [0.5, 5.0, 50.0])
def test_soft_cap_and_scale(gpu_lib, cap):
    c = R.make_paged(3, [40, 300], 2, 128, 16, R.HND)
    q = _query(3, 2, 8, 128, torch.bfloat16, scale=6.0)
    out, lse, _ = _run(gpu_lib, c, q, logits_soft_cap=cap, sm_scale=0.3)
    R.check_attention(out, lse, _ref(c, q, sm=0.3, soft_cap=cap), q.dtype)
    out, lse, _ = _run(gpu_lib, c, q, sm_scale=-0.05)
    R.check_attention(out, lse, _ref(c, q, sm=-0.05), q.dtype)


@pytest.mark.parametrize("scale,dtype", [(60.0, torch.float16), (3000.0, torch.bfloat16), (1e-3, torch.float16),
                                         (1e30, torch.bfloat16), (1e-30, torch.bfloat16)])
def test_peaked_and_flat_scores(gpu_lib, scale, dtype):
    """Scores that put all weight on one position, or the same on all; queries far from 1."""
    c = R.make_paged(11, [513, 20], 2, 128, 16, R.HND)
    q = _query(11, 2, 8, 128, dtype, scale=scale)
    sm = 0.09 if scale < 1e6 else 1e-29
    out, lse, _ = _run(gpu_lib, c, q, sm_scale=sm)
    R.check_attention(out, lse, _ref(c, q, sm=sm), dtype)


def test_query_of_zeros_and_one_huge_element(gpu_lib):
    c = R.make_paged(12, [200, 31], 1, 64, 16, R.NHD)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    q[0, 1, 5], q[1, 2, 63], q[1, 2, 0] = 3e38, -3e38, 1e-38
    out, lse, _ = _run(gpu_lib, c, q, sm_scale=1e-37)
    R.check_attention(out, lse, _ref(c, q, sm=1e-37), q.dtype)


def test_bad_pages_and_lengths(gpu_lib):
    nv = gpu_lib
    c = R.make_paged(21, [96, 50, 64, 20], 2, 128, 16, R.HND, width=6)
    c.tables[0, 2], c.tables[1, 0], c.tables[3, 0] = 10 ** 6, -5, c.k.shape[0]
    c.tables[3, 1] = -1                     # no page of request 3 is in the pool
    c.lens[0] = 1000                        # past the table's reach
    c.lens[2] = -3
    q = _query(21, 4, 8, 128, torch.float16)
    out, lse, status = _run(nv, c, q)
    c.tables = np.where(c.tables >= c.k.shape[0], -1, c.tables)
    R.check_attention(out, lse, _ref(c, q), q.dtype)
    assert status == nv.DEV_BAD_PAGE | nv.DEV_LEN_CLAMPED
    assert (out[3] == 0).all() and torch.isneginf(lse[3]).all() and (out[2] == 0).all()


def test_no_columns(gpu_lib):
    c = R.make_paged(22, [5], 1, 64, 16, R.HND)
    c.tables = np.zeros((1, 0), np.int32)
    q = _query(22, 1, 2, 64, torch.float16)
    out, lse, _ = _run(gpu_lib, c, q)
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("i", range(8))
def test_selected_pages(gpu_lib, i):
    nv = gpu_lib
    rng = np.random.Generator(np.random.PCG64(900 + i))
    H, G, D, ps, layout, dtype = [(2, 4, 128, 16, R.HND, torch.bfloat16), (3, 2, 64, 16, R.NHD, torch.float16),
                                  (1, 9, 128, 12, R.HND, torch.float16), (2, 8, 256, 4, R.NHD, torch.bfloat16),
                                  (8, 1, 64, 64, R.HND, torch.float16), (2, 4, 96, 1, R.NHD, torch.float16),
                                  (1, 16, 192, 33, R.HND, torch.bfloat16), (2, 4, 128, 16, R.NHD, torch.float16)][i]
    lens = [int(x) for x in rng.integers(1, 60 * ps + 2, 4)] + [1]
    c = R.make_paged(900 + i, lens, H, D, ps, layout, width=70)
    S = 24
    sel = np.full((5, H, S), -1, np.int32)
    num = np.zeros((5, H), np.int32)
    for b in range(5):
        n = -(-lens[b] // ps)
        for h in range(H):
            k = int(rng.integers(0, min(n, S) + 1))
            sel[b, h, :k] = np.sort(rng.permutation(n)[:k])
            num[b, h] = k
    expect = 0
    if i == 7:  # entries outside the table, in a page past the end, given twice; counts out of range
        sel[0, 0, :4], num[0, 0] = [3, 1 << 20, -1, 3], 4
        sel[1, 1, 0], num[1, 1] = 69, 1
        num[2, 0], num[3, 1] = -4, 1000
        sel[3, 1] = np.arange(S) % (-(-lens[3] // ps))
        expect = nv.DEV_BAD_PAGE
    q = _query(i, 5, H * G, D, dtype)
    out, lse, status = _run(nv, c, q, selected=sel, num_selected=num)
    R.check_attention(out, lse, _ref(c, q, selected=sel, num_selected=np.minimum(num, S)), dtype)
    assert status == expect


def test_selecting_every_page_is_the_dense_call(gpu_lib):
    c = R.make_paged(31, [500, 33, 160], 2, 128, 16, R.HND)
    q = _query(31, 3, 8, 128, torch.bfloat16)
    S = c.tables.shape[1]
    sel = np.broadcast_to(np.arange(S, dtype=np.int32), (3, 2, S)).copy()
    num = np.repeat(-(-c.lens // 16)[:, None], 2, 1).astype(np.int32)
    out, lse, _ = _run(gpu_lib, c, q)
    out2, lse2, _ = _run(gpu_lib, c, q, selected=sel, num_selected=num)
    ref = _ref(c, q)
    R.check_attention(out, lse, ref, q.dtype)
    R.check_attention(out2, lse2, ref, q.dtype)


def test_same_bits_every_time_on_any_stream(gpu_lib):
    c = R.make_paged(32, [3000, 1, 700, 2049] * 8, 2, 128, 16, R.HND)
    q = _query(32, 32, 8, 128, torch.bfloat16).to(DEV)
    dev = _dev(c)
    first = _run(gpu_lib, c, q, dev)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for s in streams * 3:
        with torch.cuda.stream(s):
            again = _run(gpu_lib, c, q, dev)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_captured_graph_follows_lengths(gpu_lib):
    nv = gpu_lib
    c = R.make_paged(33, [3000, 1, 700, 2049], 2, 128, 16, R.HND)
    q = _query(33, 4, 8, 128, torch.float16).to(DEV)
    caches, sf = _dev(c)
    tables, lens = torch.as_tensor(c.tables).to(DEV), torch.as_tensor(c.lens).to(DEV)
    gk, gv = (torch.tensor([x], dtype=torch.float32, device=DEV) for x in (c.gk, c.gv))
    call = lambda: nv.nvfp4_paged_attention_decode(q, caches, sf, tables, lens, gk, gv, "HND")
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = call()
    for lens_now in ([3000, 1, 700, 2049], [5, 0, 64, 2049], [2999, 1, 1, 1]):
        lens.copy_(torch.tensor(lens_now, dtype=torch.int32))
        for _ in range(2):
            g.replay()
        torch.cuda.synchronize()
        got = (out.clone(), lse.clone())
        want = call()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), lens_now


def test_pool_past_four_gigabytes(gpu_lib):
    """Pages whose byte offsets pass 2^32 in the codes."""
    P, H, ps, D = 600_000, 8, 16, 128
    small = R.make_paged(34, [100, 33], H, D, ps, R.HND)
    k, v = (torch.zeros((P, H, ps, D // 2), dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.full((P, H, ps, D // 16), 0x7F, dtype=torch.uint8, device=DEV) for _ in range(2))
    rng = np.random.Generator(np.random.PCG64(34))
    where = np.sort(rng.choice(np.arange(P - 70_000, P), small.k.shape[0], replace=False))
    at = torch.as_tensor(where).to(DEV)
    for big, x in ((k, small.k), (v, small.v), (ks, small.ks), (vs, small.vs)):
        big[at] = torch.as_tensor(x).to(DEV)
    moved = R.Paged(**{**small.__dict__, "tables": np.where(small.tables >= 0, where[small.tables], -1).astype(np.int64)})
    q = _query(34, 2, 16, D, torch.bfloat16)
    out, lse, status = _run(gpu_lib, moved, q, ((k, v), (ks, vs)))
    R.check_attention(out, lse, _ref(small, q), q.dtype)
    assert status == 0


def test_out_and_lse_given_and_reused_workspace(gpu_lib):
    """Calls of different shapes share one workspace; caller-owned outputs are used."""
    nv = gpu_lib
    for i in (4, 13, 9, 0, 15, 4):
        lens, H, G, D, ps, layout, dtype = CASES[i]
        c = R.make_paged(i, lens, H, D, ps, layout)
        q = _query(i, c.B, H * G, D, dtype)
        out = torch.full((c.B, H * G, D), 7.0, dtype=dtype, device=DEV)
        lse = torch.full((c.B, H * G), 7.0, device=DEV)
        got = _run(nv, c, q, out=out, lse=lse)
        assert got[0] is out and got[1] is lse
        R.check_attention(out, lse, _ref(c, q), dtype)
