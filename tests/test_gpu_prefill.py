"""Attention of the last tokens of each request over the paged NVFP4 cache against the 64-bit reference
(tests/prompt_reference.py), with the slots that no position owns full of NaN scales."""
import os

import numpy as np
import pytest
import torch

from tests import decode_reference as R
from tests import prompt_reference as PR
from tests.test_gpu_decode_attention import DEV, _dev, _layout, _query

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(gpu_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield


def _indptr(new, first=0):
    return (first + np.concatenate([[0], np.cumsum(new)])).astype(np.int32)


def _args(c, q, indptr, dev=None):
    caches, sf = dev or _dev(c)
    gk, gv = (torch.tensor([x], dtype=torch.float32, device=DEV) for x in (c.gk, c.gv))
    t = [torch.as_tensor(np.ascontiguousarray(x)).to(DEV) for x in (indptr, c.tables, c.lens)]
    return (q.to(DEV), caches, sf, *t, gk, gv, _layout(c))


def _run(nv, c, q, indptr, dev=None, **kw):
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = nv.nvfp4_paged_attention_prefill(*_args(c, q, indptr, dev), dev_status=st, **kw)
    torch.cuda.synchronize()
    return out, lse, int(st.item())


def _ref(c, q, indptr, sm=None, **kw):
    kw = {"window": kw.pop("window_left", -1), "sink": kw.pop("num_sink_tokens", 0), "soft_cap": kw.pop("logits_soft_cap", 0.0), **kw}
    return PR.attention(PR.with_f32_scales(c), q.double().numpy(), indptr, q.shape[-1] ** -0.5 if sm is None else sm, **kw)


def _both(nv, seed, new, lens, H, G, D, ps, layout, dtype, want_status=0, width=None, **kw):
    c = R.make_paged(seed, lens, H, D, ps, layout, width=width)
    q = _query(seed, sum(new), H * G, D, dtype)
    indptr = _indptr(new)
    out, lse, status = _run(nv, c, q, indptr, **kw)
    PR.check(out, lse, _ref(c, q, indptr, **kw), dtype)
    assert status == want_status


F16, BF16, NHD, HND = torch.float16, torch.bfloat16, R.NHD, R.HND
CASES = [
    # new, lens, H, G, D, ps, layout, dtype
    ([1], [1], 1, 1, 64, 16, HND, F16),
    ([1], [1], 1, 1, 16, 2, NHD, F16),
    ([1, 2, 0], [0, 1, 2], 2, 1, 64, 16, HND, BF16),                # a request without positions, one without tokens
    ([0], [300], 1, 4, 128, 16, HND, F16),
    ([3, 17, 5], [37, 64, 5], 2, 4, 64, 16, NHD, BF16),
    ([4, 4, 4, 4], [31, 129, 256, 257], 2, 8, 128, 16, HND, BF16),  # drafts
    ([127, 128, 129], [127, 128, 129], 1, 1, 128, 16, HND, F16),    # whole prompts about a tile
    ([300], [300], 2, 3, 128, 64, NHD, F16),                        # rows that split a token's heads between tiles
    ([200], [900], 1, 5, 96, 12, HND, BF16),
    ([70, 9], [200, 90], 2, 3, 80, 7, NHD, BF16),
    ([33, 40], [130, 70], 2, 2, 48, 5, HND, F16),
    ([60, 1], [77, 400], 1, 16, 128, 16, NHD, BF16),
    ([100], [333], 1, 9, 32, 32, HND, F16),
    ([45, 1], [150, 1], 1, 12, 192, 8, NHD, F16),
    ([130, 31], [260, 31], 2, 3, 256, 16, HND, BF16),
    ([2, 2], [140, 700], 1, 20, 256, 100, NHD, F16),
    ([9, 3], [90, 65], 1, 33, 112, 4, HND, BF16),
    ([4, 1, 2], [4097, 3000, 1], 1, 4, 128, 16, HND, F16),          # few rows over a long cache: cut
    ([130], [2500], 1, 2, 64, 3, NHD, BF16),
    ([2], [1500], 1, 1, 144, 16, HND, F16),
    ([2] * 70, [100] * 70, 3, 2, 64, 16, HND, F16),
    ([1, 600, 3], [2000, 640, 3], 1, 1, 128, 16, HND, BF16),        # one token, a chunk and a prompt in one call
]
MASKS = [dict(), dict(causal=False), dict(window_left=20, num_sink_tokens=4), dict(window_left=0),
         dict(window_left=130, num_sink_tokens=150, causal=False), dict(window_left=300, num_sink_tokens=129, logits_soft_cap=10.0),
         dict(logits_soft_cap=30.0, causal=False)]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_matches_reference(gpu_lib, i):
    _both(gpu_lib, i, *CASES[i])


@pytest.mark.parametrize("m", range(1, len(MASKS)))
@pytest.mark.parametrize("i", [4, 6, 8, 12, 14, 17, 21])
def test_masks(gpu_lib, i, m):
    _both(gpu_lib, 100 + i, *CASES[i], **MASKS[m])


@pytest.mark.parametrize("window,sink", [(127, 1), (128, 128), (129, 127), (383, 129), (1, 2000), (2 ** 31 - 1, 5), (500, 2 ** 31 - 1)])
def test_windows_about_tiles(gpu_lib, window, sink):
    _both(gpu_lib, window % 7, [140], [1100], 1, 2, 64, 16, HND, F16, window_left=window, num_sink_tokens=sink)


def test_more_tokens_than_positions(gpu_lib):
    """Rows before position 0 see nothing under causal: 0 and -inf."""
    c = R.make_paged(1, [10, 0, 200], 2, 128, 16, HND)
    new = [150, 7, 260]
    q = _query(1, sum(new), 4, 128, BF16)
    out, lse, status = _run(gpu_lib, c, q, _indptr(new))
    PR.check(out, lse, _ref(c, q, _indptr(new)), BF16)
    assert status == 0
    for r0, r1 in ((0, 140), (150, 157), (157, 217)):
        assert (out[r0:r1] == 0).all() and (lse[r0:r1] == -torch.inf).all()
    out, lse, _ = _run(gpu_lib, c, q, _indptr(new), causal=False)
    PR.check(out, lse, _ref(c, q, _indptr(new), causal=False), BF16)


@pytest.mark.parametrize("D,off_sf,pad_sf,pad_data", [(128, 0, 16, 32), (128, 1, 3, 0), (64, 2, 2, 0), (64, 3, 5, 48),
                                                     (256, 1, 0, 16), (96, 0, 0, 16), (80, 0, 1, 0)])
@pytest.mark.parametrize("layout", [NHD, HND])
def test_strides_and_alignment(gpu_lib, layout, D, off_sf, pad_sf, pad_data):
    c = R.make_paged(D + off_sf, [300, 41], 2, D, 16, layout)
    q = _query(D, 47, 4, D, F16)
    indptr = _indptr([40, 7])
    out, lse, _ = _run(gpu_lib, c, q, indptr, _dev(c, pad_data, pad_sf, off_sf))
    PR.check(out, lse, _ref(c, q, indptr), F16)


def test_rows_of_no_request_stay(gpu_lib):
    """Rows before the first request's, after the last one's, and out and lse given."""
    c = R.make_paged(2, [50, 300], 2, 64, 16, NHD)
    q = _query(2, 60, 4, 64, BF16)
    indptr = _indptr([20, 25], 5)
    out = torch.full((60, 4, 64), 7.0, dtype=BF16, device=DEV)
    lse = torch.full((60, 4), 9.0, device=DEV)
    o, s, status = _run(gpu_lib, c, q, indptr, out=out, lse=lse)
    assert o.data_ptr() == out.data_ptr() and s.data_ptr() == lse.data_ptr() and status == 0
    PR.check(out, lse, _ref(c, q, indptr), BF16)
    assert (out[:5] == 7).all() and (out[50:] == 7).all() and (lse[:5] == 9).all() and (lse[50:] == 9).all()


def test_query_slices_tables_of_64_bits_and_int8_scales(gpu_lib):
    c = R.make_paged(3, [50, 300], 2, 64, 16, HND, table_dtype=np.int64, width=40)
    q = _query(3, 45, 4, 64, BF16)
    indptr = _indptr([20, 25])
    wide = torch.zeros((45, 7, 64), dtype=BF16, device=DEV)
    wide[:, 1:5] = q.to(DEV)
    caches, sf = _dev(c)
    args = list(_args(c, q, indptr, (caches, tuple(x.view(torch.float8_e4m3fn) for x in sf))))
    args[0] = wide[:, 1:5]
    out, lse = gpu_lib.nvfp4_paged_attention_prefill(*args)
    PR.check(out, lse, _ref(c, q, indptr), BF16)


def test_pages_outside_the_pool(gpu_lib):
    c = R.make_paged(4, [400, 90], 1, 64, 16, NHD)
    for j, bad in ((0, 10 ** 6), (3, -5), (24, 99999)):
        c.tables[0, j] = bad
    c.tables[1, :] = -1  # all of a request
    q = _query(4, 60, 4, 64, F16)
    indptr = _indptr([50, 10])
    out, lse, status = _run(gpu_lib, c, q, indptr)
    PR.check(out, lse, _ref(c, q, indptr), F16)
    assert status == gpu_lib.DEV_BAD_PAGE and (out[50:] == 0).all()
    # where no row looks, nothing is reported
    kw = dict(window_left=100, num_sink_tokens=20)
    c = R.make_paged(4, [400], 1, 64, 16, NHD)
    c.tables[0, 5] = c.tables[0, 12] = -1
    out, lse, status = _run(gpu_lib, c, q[:50], _indptr([50]), **kw)
    PR.check(out, lse, _ref(c, q[:50], _indptr([50]), **kw), F16)
    assert status == 0


def test_lengths_past_the_table(gpu_lib):
    c = R.make_paged(5, [400], 1, 64, 16, NHD)
    c.tables = np.ascontiguousarray(c.tables[:, :10])
    q = _query(5, 30, 2, 64, F16)
    out, lse, status = _run(gpu_lib, c, q, _indptr([30]))
    PR.check(out, lse, _ref(c, q, _indptr([30])), F16)
    assert status == gpu_lib.DEV_LEN_CLAMPED


@pytest.mark.parametrize("indptr,taken", [([-3, 5, 9], [0, 5, 9]), ([0, 5, 1000], [0, 5, 12]), ([0, 7, 4], [0, 7, 7])])
def test_row_ranges_that_are_none(gpu_lib, indptr, taken):
    c = R.make_paged(6, [40, 90], 1, 64, 16, HND)
    q = _query(6, 12, 2, 64, F16)
    out = torch.full((12, 2, 64), 7.0, dtype=F16, device=DEV)
    out, lse, status = _run(gpu_lib, c, q, np.array(indptr, np.int32), out=out)
    assert status == gpu_lib.DEV_BAD_BATCH
    PR.check(out, lse, _ref(c, q, taken), F16)
    assert (out[taken[-1]:] == 7).all()


@pytest.mark.parametrize("D,G", [(128, 1), (128, 4), (64, 2), (256, 2)])
def test_nan_shows_where_the_formula_has_it(gpu_lib, D, G):
    """NaN block scales of K and of V in live slots: the rows that see the position, and of V's only that block."""
    new, lens = [200, 3, 90], [350, 1200, 90]
    c = R.make_paged(7, lens, 2, D, 16, HND)
    at = lambda b, t: (c.tables[b, t // 16], t % 16)  # noqa: E731
    p, s = at(0, 260)
    c.vs[p, 0, s, 1] = 0x7F
    c.vs[p, 1, s, D // 16 - 1] = 0xFF
    p, s = at(0, 320)
    c.ks[p, 0, s, 0] = 0xFF
    p, s = at(1, 700)
    c.vs[p, 1, s, 2] = 0x7F
    p, s = at(2, 89)   # the last position: the last row's alone
    c.vs[p, 0, s, :] = 0x7F
    q = _query(7, sum(new), 2 * G, D, BF16)
    for kw in (dict(), dict(window_left=60, num_sink_tokens=3)):
        out, lse, status = _run(gpu_lib, c, q, _indptr(new), **kw)
        ref = _ref(c, q, _indptr(new), **kw)
        assert np.isnan(ref[0]).any() and not np.isnan(ref[0]).all(-1).all()
        PR.check(out, lse, ref, BF16)
        assert status == 0


def test_queries_that_are_not_finite(gpu_lib):
    c = R.make_paged(8, [300], 1, 64, 16, HND)
    q = _query(8, 100, 2, 64, BF16)
    q[3, 0, 5] = torch.nan
    q[40, 1, 7] = torch.inf
    q[90, 0, 0] = -torch.inf
    q[91, 1] = 0
    clean = q.clone()
    clean[[3, 40, 90], [0, 1, 0]] = 0
    out, lse, _ = _run(gpu_lib, c, q, _indptr([100]))
    same, same_lse, _ = _run(gpu_lib, c, clean, _indptr([100]))
    for r, h in ((3, 0), (40, 1), (90, 0)):
        assert torch.isnan(out[r, h]).all() and torch.isnan(lse[r, h])
        out[r, h], lse[r, h] = same[r, h], same_lse[r, h]
    assert torch.equal(out, same) and torch.equal(lse, same_lse)
    PR.check(same, same_lse, _ref(c, clean, _indptr([100])), BF16)


@pytest.mark.parametrize("sm,scale", [(-0.1, 1.0), (0.0, 1.0), (1e-6, 3e4), (0.3, 1e-30), (2.0, 4.0)])
def test_scales_and_magnitudes(gpu_lib, sm, scale):
    c = R.make_paged(9, [280, 40], 2, 64, 16, HND)
    q = _query(9, 60, 4, 64, BF16, scale)
    out, lse, _ = _run(gpu_lib, c, q, _indptr([50, 10]), sm_scale=sm)
    PR.check(out, lse, _ref(c, q, _indptr([50, 10]), sm), BF16)


@pytest.mark.parametrize("gk,sm,scale", [(1e-22, 1e-20, 1e37), (1e20, 1e15, 1e-36), (-0.002, 0.1, 1.0), (0.0, 0.1, 1.0)])
def test_factors_whose_product_is_out_of_range(gpu_lib, gk, sm, scale):
    c = R.make_paged(9, [280, 40], 2, 64, 16, HND)
    c.gk = gk
    q = _query(9, 60, 4, 64, BF16, scale)
    out, lse, _ = _run(gpu_lib, c, q, _indptr([50, 10]), sm_scale=sm)
    PR.check(out, lse, _ref(c, q, _indptr([50, 10]), float(np.float32(sm))), BF16)


def test_growing_scores(gpu_lib):
    """The maximum rises all along a row, by more than the slack that it is given."""
    for D, G in ((64, 4), (128, 1), (256, 1)):
        c = R.make_paged(10, [1000, 700], 1, D, 16, HND)
        for b in range(2):
            for j in range(-(-int(c.lens[b]) // 16)):
                c.k[c.tables[b, j]] = 0x22   # 1.0 everywhere
                c.ks[c.tables[b, j]] = min(0x30 + j, 0x7A)
        q = torch.ones((200, G, D)).to(F16)
        out, lse, _ = _run(gpu_lib, c, q, _indptr([190, 10]), sm_scale=5.0 / D)
        PR.check(out, lse, _ref(c, q, _indptr([190, 10]), 5.0 / D), F16)


def test_a_row_does_not_depend_on_the_others(gpu_lib):
    """Rows' values, to the last bit, with other rows' queries changed; and from call to call."""
    c = R.make_paged(11, [900, 500], 2, 128, 16, HND)
    q = _query(11, 300, 4, 128, BF16)
    dev = _dev(c)
    indptr = _indptr([250, 50])
    out, lse, _ = _run(gpu_lib, c, q, indptr, dev)
    again, lse2, _ = _run(gpu_lib, c, q, indptr, dev)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    other = q.clone()
    other[::2] = 100 * other[::2].flip(0)
    got, lse3, _ = _run(gpu_lib, c, other, indptr, dev)
    assert torch.equal(out[1::2], got[1::2]) and torch.equal(lse[1::2], lse3[1::2])


def test_one_token_each_as_the_decode_call(gpu_lib):
    c = R.make_paged(12, [900, 1, 77, 0], 2, 128, 16, HND)
    q = _query(12, 4, 8, 128, BF16)
    kw = dict(window_left=100, num_sink_tokens=7)
    out, lse, _ = _run(gpu_lib, c, q, np.arange(5, dtype=np.int32), **kw)
    a = _args(c, q, np.arange(5, dtype=np.int32))
    want, want_lse = gpu_lib.nvfp4_paged_attention_decode(*a[:3], *a[4:], **kw)
    PR.check(out, lse, _ref(c, q, np.arange(5), **kw), BF16)
    assert torch.allclose(out.float(), want.float(), rtol=2 ** -7, atol=1e-4) and torch.allclose(lse, want_lse, rtol=1e-5, atol=1e-5)


def test_captured_and_replayed_on_other_lengths(gpu_lib):
    """Lengths, row ranges and queries change under a graph; another stream's calls run beside it."""
    c = R.make_paged(13, [1500, 900], 2, 128, 16, HND)
    q = _query(13, 300, 8, 128, BF16)
    args = list(_args(c, q, _indptr([100, 200])))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = gpu_lib.nvfp4_paged_attention_prefill(*args)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    for new, now in (([100, 200], [1500, 900]), ([1, 299], [1400, 299]), ([0, 4], [3, 880])):
        args[3].copy_(torch.as_tensor(_indptr(new)))
        args[5].copy_(torch.tensor(now))
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(other):
            beside, beside_lse = gpu_lib.nvfp4_paged_attention_prefill(*args)
        torch.cuda.synchronize()
        rows = sum(new)
        assert torch.equal(out[:rows], beside[:rows]) and torch.equal(lse[:rows], beside_lse[:rows])
        short = R.Paged(**{**c.__dict__, "lens": np.array(now, np.int32)})
        PR.check(out, lse, _ref(short, q, _indptr(new)), BF16)


def test_many_requests(gpu_lib):
    """More requests than threads, most of them of no tokens."""
    B = 3000
    new = [(i % 97 == 0) * (1 + i % 5) for i in range(B)]
    lens = [(i % 97 == 0) * (20 + i % 150) for i in range(B)]
    _both(gpu_lib, 14, new, lens, 1, 2, 64, 16, HND, F16)


def test_a_wait_that_runs_out(gpu_lib):
    """The tiles are withheld: the call comes back, reports it, and the next call is right."""
    c = R.make_paged(15, [300, 700], 2, 128, 16, HND)
    for new, D in (([300, 20], 128), ([20, 30], 128), ([50, 3], 256)):
        c = R.make_paged(15, [300, 700], 2, D, 16, HND)
        q = _query(15, sum(new), 4, D, BF16)
        os.environ["NVFP4KV_TEST_STALL_PIPELINE"] = "1"
        try:
            _, _, status = _run(gpu_lib, c, q, _indptr(new))
        finally:
            os.environ.pop("NVFP4KV_TEST_STALL_PIPELINE")
        assert status == gpu_lib.DEV_TIMEOUT
        out, lse, status = _run(gpu_lib, c, q, _indptr(new))
        PR.check(out, lse, _ref(c, q, _indptr(new)), BF16)
        assert status == 0


def test_refusals_by_the_tensors(gpu_lib):
    nv = gpu_lib
    c = R.make_paged(16, [50, 30], 2, 64, 16, HND)
    q = _query(16, 20, 4, 64, BF16)
    ok = list(_args(c, q, _indptr([10, 10])))

    def call(i, x, **kw):
        a = list(ok)
        a[i] = x
        return nv.nvfp4_paged_attention_prefill(*a, **kw)

    for i, x, text in ((0, ok[0][0], "n, heads, head_dim"), (0, ok[0].float(), "float16 or bfloat16"), (0, ok[0][:, :, :48], "heads of 64"),
                       (0, ok[0].transpose(0, 1), "contiguous heads"), (3, ok[3][:2], "one entry more"), (3, ok[3].long(), "Int"),
                       (4, ok[4][:1], "block_tables"), (5, ok[5].long(), "Int"), (6, 0.5, "k_scale"), (3, ok[3].cpu(), "cuda")):
        with pytest.raises(ValueError, match=text):
            call(i, x)
    with pytest.raises(ValueError, match="out must be"):
        call(0, ok[0], out=torch.empty((20, 4, 32), dtype=BF16, device=DEV))
    with pytest.raises(ValueError, match="lse must be"):
        call(0, ok[0], lse=torch.empty((20, 3), device=DEV))
    with pytest.raises(nv.NVFP4KVError, match="multiple of num_kv_heads"):
        call(0, ok[0][:, :3].contiguous())
    with pytest.raises(nv.NVFP4KVError, match="num_sink_tokens"):
        call(0, ok[0], num_sink_tokens=-1)
    out, lse = call(0, ok[0][:0])
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)


@pytest.mark.parametrize("window", [-1, 30])
def test_many_segments_with_an_empty_half(gpu_lib, window):
    """288 rows a KV head: the second segment's second half has none; several segments to a CTA."""
    new, lens = [72] * 130, [72 + 3 * i for i in range(130)]
    _both(gpu_lib, 17, new, lens, 2, 4, 64, 16, HND, BF16, window_left=window, num_sink_tokens=2)


FEW = [
    # few rows a request (and tables of more than 1024 positions): new, lens, H, G, D, ps, layout, dtype
    ([1, 1, 1], [40, 1, 333], 2, 8, 128, 16, HND, BF16),
    ([4] * 6, [31, 32, 33, 4, 700, 129], 2, 4, 128, 16, HND, BF16),      # drafts: sixteen rows
    ([2, 5, 1, 0, 3], [1, 64, 100, 7, 2], 1, 3, 64, 12, NHD, F16),       # more tokens than positions among them
    ([1, 1, 1, 1, 1, 40], [100, 30, 0, 400, 64, 300], 2, 2, 64, 16, HND, F16),   # a chunk beside single tokens
    ([2, 1, 3, 300], [1500, 40, 9, 640], 1, 1, 96, 16, NHD, BF16),       # and a prompt beside drafts
    ([3, 1, 3, 2], [200, 77, 5, 450], 2, 5, 80, 7, HND, BF16),
    ([8, 1, 4], [260, 31, 700], 2, 1, 256, 16, HND, F16),
    ([2, 4], [150, 90], 3, 2, 192, 8, NHD, BF16),
    ([16, 3], [3000, 18], 1, 1, 32, 16, HND, F16),
    ([2] * 90, [500 + i for i in range(90)], 4, 3, 64, 16, HND, BF16),   # lists that are cut
]


@pytest.mark.parametrize("m", range(len(MASKS)))
@pytest.mark.parametrize("i", range(len(FEW)))
def test_few_rows(gpu_lib, i, m):
    _both(gpu_lib, 200 + i, *FEW[i], width=4000 // FEW[i][5], **MASKS[m])


@pytest.mark.parametrize("window,sink", [(30, 33), (31, 32), (64, 1), (2, 70), (1000, 5)])
def test_few_rows_windows_about_units(gpu_lib, window, sink):
    _both(gpu_lib, window, [5, 3, 1], [400, 97, 32], 1, 2, 64, 16, HND, F16, width=100, window_left=window, num_sink_tokens=sink)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_few_rows_nan_shows_where_the_formula_has_it(gpu_lib, D):
    new, lens = [3, 1, 4], [350, 90, 1200]
    c = R.make_paged(18, lens, 2, D, 16, HND)
    at = lambda b, t: (c.tables[b, t // 16], t % 16)  # noqa: E731
    for b, t, h, block in ((0, 348, 0, 1), (0, 349, 1, 0), (2, 700, 1, 2), (2, 1197, 0, 3), (2, 1150, 0, 0)):
        p, s = at(b, t)
        c.vs[p, h, s, block] = 0x7F
    p, s = at(2, 1198)
    c.ks[p, 1, s, 0] = 0xFF
    q = _query(18, sum(new), 4 if D == 128 else 2, D, BF16)
    for kw in (dict(), dict(window_left=48, num_sink_tokens=3), dict(causal=False, window_left=47)):
        out, lse, status = _run(gpu_lib, c, q, _indptr(new), **kw)
        ref = _ref(c, q, _indptr(new), **kw)
        assert np.isnan(ref[0]).any() and not np.isnan(ref[0]).all(-1).all()
        PR.check(out, lse, ref, BF16)
        assert status == 0


def test_few_rows_captured_and_replayed(gpu_lib):
    """Under a graph a request grows from few rows to many and back."""
    c = R.make_paged(19, [1500, 900, 40], 2, 128, 16, HND)
    q = _query(19, 12, 8, 128, BF16)
    args = list(_args(c, q, _indptr([4, 4, 4])))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = gpu_lib.nvfp4_paged_attention_prefill(*args)
    for new, now in (([4, 4, 4], [1500, 900, 40]), ([1, 11, 0], [1400, 299, 0]), ([0, 4, 8], [3, 880, 17])):
        args[3].copy_(torch.as_tensor(_indptr(new)))
        args[5].copy_(torch.tensor(now))
        graph.replay()
        torch.cuda.synchronize()
        short = R.Paged(**{**c.__dict__, "lens": np.array(now, np.int32)})
        PR.check(out, lse, _ref(short, q, _indptr(new)), BF16)


@pytest.mark.parametrize("new,width", [([300, 40], None), ([3, 2], 100)])
def test_caches_of_more_than_4_gib(gpu_lib, new, width):
    """Pages 300 MB apart: offsets need 64 bits, for rows of 128 and for few."""
    c = R.make_paged(20, [400, 90], 2, 64, 16, HND, width=width)
    q = _query(20, sum(new), 4, 64, BF16)
    dev = _dev(c, pad_data=300_000_000)
    assert c.k.shape[0] * 300_000_000 > 1 << 32
    out, lse, status = _run(gpu_lib, c, q, _indptr(new), dev)
    PR.check(out, lse, _ref(c, q, _indptr(new)), BF16)
    assert status == 0


@pytest.mark.parametrize("width", [2, 70])
def test_largest_batch(gpu_lib, width):
    """16,384 requests, most of them without tokens, for rows of 128 and (tables of 1120 positions) for few."""
    B = 16384
    new = [1 + i % 4 if i % 911 == 0 else 0 for i in range(B)]
    lens = [1 + i % 30 if i % 3 == 0 else 0 for i in range(B)]
    _both(gpu_lib, 21, new, lens, 1, 2, 32, 16, HND, F16, width=width)
    with pytest.raises(gpu_lib.NVFP4KVError, match="16384"):
        c = R.make_paged(21, [1] * (B + 1), 1, 32, 16, HND)
        gpu_lib.nvfp4_paged_attention_prefill(*_args(c, _query(21, B + 1, 2, 32, F16), np.arange(B + 2, dtype=np.int32)))


def test_requests_that_share_pages(gpu_lib):
    """A common prompt: two requests' tables name the same pages."""
    c = R.make_paged(22, [160, 160, 200], 2, 64, 16, HND)
    c.tables[1] = c.tables[0]
    c.tables[2, :10] = c.tables[0, :10]
    q = _query(22, 90, 4, 64, F16)
    for new in ([30, 20, 40], [1, 2, 3]):
        out, lse, status = _run(gpu_lib, c, q[:sum(new)], _indptr(new))
        PR.check(out, lse, _ref(c, q[:sum(new)], _indptr(new)), F16)
        assert status == 0


def test_two_streams_at_once(gpu_lib):
    """Calls that run beside each other have workspaces of their own."""
    c = R.make_paged(23, [3000, 1700], 2, 128, 16, HND)
    dev = _dev(c)
    calls = []
    for i, new in enumerate(([200, 64], [130, 1000], [4, 4], [900, 30])):
        q = _query(30 + i, sum(new), 8, 128, BF16)
        calls.append((q, _indptr(new), _args(c, q, _indptr(new), dev)))
    alone = [gpu_lib.nvfp4_paged_attention_prefill(*a) for _, _, a in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        got = []
        for s, (_, _, a) in zip(streams, calls):
            with torch.cuda.stream(s):
                got.append(gpu_lib.nvfp4_paged_attention_prefill(*a))
        torch.cuda.synchronize()
        for (o, l), (wo, wl) in zip(got, alone):
            assert torch.equal(o, wo) and torch.equal(l, wl)


def test_row_ranges_that_overlap(gpu_lib):
    """After an entry below the one before it, requests may not take rows again: those before it keep theirs."""
    B, n = 4001, 300
    c = R.make_paged(24, [900] + [20] * (B - 1), 1, 64, 16, HND)
    q = _query(24, n, 2, 64, F16)
    indptr = np.array([0] + [n, 0] * (B // 2) + [n], np.int32)
    assert indptr.size == B + 1
    out, lse, status = _run(gpu_lib, c, q, indptr)
    first = R.Paged(**{**c.__dict__, "B": 1, "tables": np.ascontiguousarray(c.tables[:1]), "lens": c.lens[:1]})
    PR.check(out, lse, _ref(first, q, _indptr([n])), F16)
    assert status == gpu_lib.DEV_BAD_BATCH
