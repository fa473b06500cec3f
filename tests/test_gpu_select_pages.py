"""Page bounds (exact) and page selection (equal, ties included) against tests/decode_reference.py."""
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


def _t(a):
    return torch.as_tensor(np.ascontiguousarray(a)).to(DEV)


BOUNDS = [
    # lens, H, D, ps, layout, table dtype
    ([1], 1, 16, 2, R.NHD, np.int32),
    ([0, 37, 64], 2, 64, 16, R.NHD, np.int32),
    ([33, 5, 0, 200], 8, 128, 16, R.HND, np.int64),
    ([100, 99], 3, 96, 12, R.HND, np.int32),
    ([70], 2, 80, 64, R.NHD, np.int32),
    ([130, 1, 2], 1, 256, 100, R.HND, np.int64),
    ([50, 31], 2, 512, 5, R.NHD, np.int32),
    ([700, 3], 16, 128, 32, R.NHD, np.int32),
]


def _bounds(nv, c, first=None, status=None):
    out = torch.full((c.k.shape[0], c.H, 2, c.D), 9.0, dtype=torch.float16, device=DEV)
    nv.nvfp4_page_key_bounds(_t(c.k), _t(c.ks), _t(c.tables), _t(c.lens), out,
                             None if first is None else _t(np.asarray(first, np.int32)),
                             "NHD" if c.layout == R.NHD else "HND", dev_status=status)
    torch.cuda.synchronize()
    return out.double().cpu().numpy()


@pytest.mark.parametrize("i", range(len(BOUNDS)))
@pytest.mark.parametrize("last", [False, True])
def test_bounds_are_exact(gpu_lib, i, last):
    lens, H, D, ps, layout, tdt = BOUNDS[i]
    c = R.make_paged(i, lens, H, D, ps, layout, table_dtype=tdt)
    c.ks[:, 0, 0, 0] |= np.uint8(0x80)  # a scale may carry a sign
    first = c.lens - 1 if last else None
    got = _bounds(gpu_lib, c, first)
    want = np.full(got.shape, 9.0)
    for p, (lo, hi) in R.key_bounds(c, first).items():
        want[p, :, 0], want[p, :, 1] = lo, hi
    assert np.array_equal(got, want)


def test_bounds_of_bad_pages_and_lengths(gpu_lib):
    nv = gpu_lib
    c = R.make_paged(50, [100, 50, 20], 2, 64, 16, R.HND, width=7)
    c.tables[0, 1], c.tables[1, 0] = -3, 10 ** 7
    c.lens[2] = 500
    c.tables[2, 2:] = c.k.shape[0]
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = _bounds(nv, c, [-5, 0, 0], st)
    p = c.tables[2, 1]  # the clamped length reaches past this page: its dead slots count as live
    want = np.full(got.shape, 9.0)
    for page, (lo, hi) in R.key_bounds(c, [0, 0, 0]).items():
        want[page, :, 0], want[page, :, 1] = lo, hi
    keep = np.arange(got.shape[0]) != p
    assert np.array_equal(got[keep], want[keep])
    assert int(st.item()) == nv.DEV_BAD_PAGE | nv.DEV_LEN_CLAMPED


RING = [
    # pages that bulk copies take: one, two and four lanes to a column, columns of several pages to a job
    ([3000, 1, 0, 77], 1, 64, 8, R.HND, np.int32),
    ([900, 31], 3, 96, 16, R.HND, np.int32),
    ([900, 31], 3, 96, 16, R.NHD, np.int64),
    ([700, 65, 64], 2, 80, 32, R.NHD, np.int32),
    ([130, 700, 2], 5, 48, 64, R.HND, np.int32),
    ([513] * 70, 2, 16, 16, R.NHD, np.int32),
    ([20000], 4, 64, 32, R.NHD, np.int32),
]


@pytest.mark.parametrize("i", range(len(RING)))
@pytest.mark.parametrize("last", [False, True])
def test_bounds_of_pages_in_bulk_copies(gpu_lib, i, last):
    lens, H, D, ps, layout, tdt = RING[i]
    assert ps * H * D // 16 % 16 == 0
    c = R.make_paged(i + 90, lens, H, D, ps, layout, table_dtype=tdt)
    first = c.lens // 2 if last else None
    got = _bounds(gpu_lib, c, first)
    want = np.full(got.shape, 9.0)
    for p, (lo, hi) in R.key_bounds(c, first).items():
        want[p, :, 0], want[p, :, 1] = lo, hi
    assert np.array_equal(got, want)


def _select_case(seed, lens, H, G, D, ps, dtype, quant=None):
    rng = np.random.Generator(np.random.PCG64(seed))
    lens = np.asarray(lens, np.int32)
    pages = (lens + ps - 1) // ps
    P = int(pages.sum()) + 5
    w = max(int(pages.max()), 1)
    tables = np.full((len(lens), w), -1, np.int32)
    perm, at = rng.permutation(P), 0
    for b, n in enumerate(pages):
        tables[b, :n] = perm[at:at + n]
        at += n
    mid = rng.standard_normal((P, H, D)) * 300
    half = rng.random((P, H, D)) * 500
    bounds = np.stack([mid - half, mid + half], 2).astype(np.float16)
    q = rng.standard_normal((len(lens), H * G, D))
    if quant:  # few different values: many equal scores
        bounds = (np.round(bounds.astype(np.float64) / quant) * quant).astype(np.float16)
        q = np.sign(q) * (rng.random(q.shape) < 0.05)
    return lens, tables, bounds, torch.as_tensor(q).to(dtype)


def _check_select(nv, case, ps, k, sink, recent, **kw):
    lens, tables, bounds, q = case
    B, Hq, D = q.shape
    H = bounds.shape[1]
    G = Hq // H
    sel, num = nv.nvfp4_select_pages(q.to(DEV), _t(bounds), _t(tables), _t(lens), ps, k, num_sink_pages=sink,
                                     num_recent_pages=recent, **kw)
    torch.cuda.synchronize()
    sel, num = sel.cpu().numpy(), num.cpu().numpy()
    qf = q.float().numpy()
    for b in range(B):
        n = -(-int(lens[b]) // ps) if lens[b] > 0 else 0
        for h in range(H):
            s = R.page_scores(qf[b, h * G:(h + 1) * G], bounds[tables[b, :n], h].astype(np.float32)) if n else []
            want = R.select(s, k, sink, recent)
            assert num[b, h] == len(want)
            assert sel[b, h, :len(want)].tolist() == want, (b, h)
            assert (sel[b, h, len(want):] == -1).all()


SELECT = [
    # lens, H, G, D, ps, dtype, k, sink, recent
    ([1], 1, 1, 16, 16, torch.float16, 1, 0, 0),
    ([0, 5, 100], 2, 2, 64, 4, torch.bfloat16, 8, 1, 1),
    ([3000, 4000, 17], 2, 4, 128, 16, torch.bfloat16, 64, 1, 2),
    ([900, 901], 3, 7, 96, 3, torch.float16, 100, 0, 0),
    ([5000], 2, 8, 128, 2, torch.float16, 256, 2, 4),
    ([640, 650], 1, 16, 256, 5, torch.bfloat16, 33, 1, 1),
    ([2000, 100], 2, 5, 192, 16, torch.float16, 7, 3, 9),
    ([40000], 1, 4, 64, 1, torch.bfloat16, 300, 1, 1),
    ([200, 16], 2, 33, 80, 1, torch.float16, 50, 1, 1),
    ([600, 16], 2, 20, 32, 1, torch.float16, 50, 0, 1),
]


@pytest.mark.parametrize("i", range(len(SELECT)))
def test_selection_is_equal(gpu_lib, i):
    lens, H, G, D, ps, dtype, k, sink, recent = SELECT[i]
    _check_select(gpu_lib, _select_case(i, lens, H, G, D, ps, dtype), ps, k, sink, recent)


@pytest.mark.parametrize("quant", [None, 500.0])
def test_many_short_lists(gpu_lib, quant):
    """More lists than wide CTAs fit at once: a small CTA to a list, the longest of 16 keys a thread."""
    lens = [(37 * i) % 400 for i in range(398)] + [8192, 8189]
    _check_select(gpu_lib, _select_case(5, lens, 2, 4, 16, 4, torch.float16, quant=quant), 4, 30, 1, 1)


@pytest.mark.parametrize("k", [1, 5, 64, 200])
def test_ties_go_to_the_lower_page(gpu_lib, k):
    _check_select(gpu_lib, _select_case(77, [3000, 700], 2, 4, 64, 4, torch.float16, quant=500.0), 4, k, 1, 1)
    lens, tables, bounds, q = _select_case(78, [3000, 700], 2, 4, 64, 4, torch.float16)
    _check_select(gpu_lib, (lens, tables, np.zeros_like(bounds), q), 4, k, 1, 1)
    _check_select(gpu_lib, (lens, tables, bounds, torch.zeros_like(q)), 4, k, 0, 0)


def test_forced_pages_past_the_count_and_beyond(gpu_lib):
    case = _select_case(79, [1000, 50, 3], 2, 2, 64, 4, torch.float16)
    _check_select(gpu_lib, case, 4, 6, 4, 4)     # more forced than selected: the lower ones
    _check_select(gpu_lib, case, 4, 6, 1000, 0)
    _check_select(gpu_lib, case, 4, 500, 1, 1)   # more than there are


def test_bad_pages_come_last(gpu_lib):
    nv = gpu_lib
    lens, tables, bounds, q = _select_case(80, [400], 1, 4, 64, 4, torch.float16)
    tables[0, 10:30] = 10 ** 8
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    sel, num = nv.nvfp4_select_pages(q.to(DEV), _t(bounds), _t(tables), _t(lens), 4, 80, num_sink_pages=0,
                                     num_recent_pages=0, dev_status=st)
    assert sel[0, 0, :80].tolist() == list(range(10)) + list(range(30, 100))
    assert int(st.item()) == nv.DEV_BAD_PAGE
    st.zero_()
    lens[0] = 10 ** 6
    nv.nvfp4_select_pages(q.to(DEV), _t(bounds), _t(tables), _t(lens), 4, 8, dev_status=st)
    assert int(st.item()) == nv.DEV_BAD_PAGE | nv.DEV_LEN_CLAMPED


def test_query_slice_given_output_and_graph(gpu_lib):
    nv = gpu_lib
    lens, tables, bounds, q = _select_case(81, [3000, 4000], 2, 4, 128, 16, torch.bfloat16)
    wide = torch.zeros((2, 12, 128), dtype=q.dtype, device=DEV)
    wide[:, 3:11] = q.to(DEV)
    want = nv.nvfp4_select_pages(q.to(DEV), _t(bounds), _t(tables), _t(lens), 16, 20)
    out = (torch.zeros((2, 2, 20), dtype=torch.int32, device=DEV), torch.zeros((2, 2), dtype=torch.int32, device=DEV))
    got = nv.nvfp4_select_pages(wide[:, 3:11], _t(bounds), _t(tables), _t(lens), 16, 20, out=out)
    assert got[0] is out[0] and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    bt, tt, lt = _t(bounds), _t(tables), _t(lens)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = nv.nvfp4_select_pages(wide[:, 3:11], bt, tt, lt, 16, 20)
    for n in ([3000, 4000], [100, 1], [16, 17]):
        lt.copy_(torch.tensor(n, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        _check_select(nv, (np.array(n, np.int32), tables, bounds, q), 16, 20, 1, 1, out=(cap[0].clone(), cap[1].clone()))
        want = nv.nvfp4_select_pages(q.to(DEV), bt, tt, lt, 16, 20)
        assert torch.equal(cap[0], want[0]) and torch.equal(cap[1], want[1])


def test_selected_scores_are_upper_bounds(gpu_lib):
    """Bounds from the cache, then selection: no position outside the selection beats what its page promises."""
    nv = gpu_lib
    c = R.make_paged(82, [1000], 1, 64, 16, R.HND)
    bounds = _bounds(nv, c).astype(np.float32)
    q = torch.randn((1, 2, 64), generator=torch.Generator().manual_seed(1)).half()
    n = -(-1000 // 16)
    s = R.page_scores(q.float().numpy()[0], bounds[c.tables[0, :n], 0])
    for j in range(n):
        x = c.rows("k", int(c.tables[0, j]), 0)[: 1000 - 16 * j] @ q[0].double().numpy().T
        assert x.max() <= s[j] + 64 * 2.0 ** -24 * np.abs(bounds).max() * 64
