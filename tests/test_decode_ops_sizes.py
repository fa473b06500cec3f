"""Sizes whose counters inside the kernels would pass 32 bits are refused on the host (CPU: nothing is
launched, the addresses are made up)."""
import ctypes

import pytest

import nvfp4_paged_kv_02_gb300 as nv
from tests.test_decode_ops_refusals import UNS, attend, cache, err, select

TABLE = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    return nv.load()


@pytest.mark.parametrize("kw", [
    dict(B=1, maxp=TABLE),                       # a request's pages and a pass over them
    dict(B=1, maxp=2 ** 30 + 1),
    dict(B=16384, maxp=2 ** 20 + 1),             # groups of eight pages of all requests
    dict(B=17, maxp=2 ** 30),
    dict(B=16, maxp=2 ** 30),
])
def test_select_refuses_what_it_cannot_count(lib, kw):
    bytes_ = ctypes.c_int64(-1)
    assert select(lib, wsb=2 ** 62, **kw) == UNS
    assert "max_pages_per_request" in err(lib)
    assert lib.nvfp4_select_pages_workspace_bytes(kw["B"], 8, kw["maxp"], ctypes.byref(bytes_)) == UNS
    assert bytes_.value == -1


def test_select_workspace_bytes_do_not_wrap(lib):
    n = ctypes.c_int64(-1)
    assert lib.nvfp4_select_pages_workspace_bytes(1, 2 ** 31 - 1, 2 ** 30, ctypes.byref(n)) == UNS and n.value == -1
    assert lib.nvfp4_select_pages_workspace_bytes(2 ** 31 - 1, 2, 8, ctypes.byref(n)) == UNS
    assert lib.nvfp4_select_pages_workspace_bytes(1, 2 ** 26, 2 ** 30, ctypes.byref(n)) == nv.OK
    assert n.value == 2 ** 58
    assert lib.nvfp4_select_pages_workspace_bytes(15, 8, 2 ** 30, ctypes.byref(n)) == nv.OK


@pytest.mark.parametrize("kw", [
    dict(B=16384, maxp=TABLE), dict(B=16384, maxp=2 ** 20), dict(B=16384, S=2 ** 24, sel=1 << 20),
])
def test_attention_refuses_what_it_cannot_count(lib, kw):
    assert attend(lib, **kw) == UNS
    assert "2^43" in err(lib)


def test_attention_counts_every_list_of_a_wide_batch(lib):
    # below the limit the next check answers (here: no query)
    assert attend(lib, q=None, B=16384, maxp=2 ** 19 - 2 ** 10) == nv.ERR_INVALID_ARG and "query" in err(lib)
    assert attend(lib, q=None, B=1, maxp=TABLE) == nv.ERR_INVALID_ARG and "query" in err(lib)


def test_page_indices_are_32_bits(lib):
    huge = cache(pages=2 ** 31)
    assert select(lib, pages=2 ** 31) == UNS and "pages" in err(lib)
    assert attend(lib, kc=huge, vc=huge) == UNS and "pages" in err(lib)
    assert attend(lib, kc=huge, vc=huge, S=4, sel=1 << 20) == UNS and "pages" in err(lib)
    # the smaller of the two caches counts; the next check answers (here: no query)
    assert attend(lib, kc=huge, q=None) == nv.ERR_INVALID_ARG and "query" in err(lib)
