"""Norm, rotation and append with positions of several axes: query rows and cache bytes are exactly those of
the operator's binary32 order, each pair by the position on its axis, followed by the CPU oracle's append."""
import functools

import numpy as np
import pytest
import torch

from tests import decode_reference as R
from tests.test_gpu_norm_rope import DEV, Case, _same, _t

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(gpu_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield


class _ByToken:
    """A cos/sin table whose rows are the tokens', whatever their positions are."""
    def __init__(self, rows):
        self.rows, self.shape = rows, rows.shape

    def __getitem__(self, pos):
        return self.rows


class AxesCase(Case):
    def __init__(self, *args, axes=3, pair_axes=None, **kw):
        super().__init__(*args, **kw)
        rng = np.random.Generator(np.random.PCG64(args[0] + 100))
        self.table = R.cos_sin(500, self.rot)  # (more positions than the cache has)
        self.axis_pos = rng.integers(0, 500, (axes, self.nnz)).astype(np.int32)
        pairs = self.rot // 2
        self.pair_axes = rng.integers(0, axes, pairs).astype(np.uint8) if pair_axes is None else np.array(pair_axes, np.uint8)
        assert self.pair_axes.size == pairs

    def expect(self):
        table = self.table
        pair = np.arange(self.rot // 2)
        at = self.axis_pos[self.pair_axes].T  # [n, pairs]
        self.table = _ByToken(np.concatenate([table[at, pair], table[at, self.rot // 2 + pair]], -1))
        try:
            return super().expect()
        finally:
            self.table = table

    def call(self, nv, **kw):
        class Axes:
            NVFP44Over6Config = nv.NVFP44Over6Config
            nvfp4_qk_norm_rope_append_paged = staticmethod(functools.partial(
                nv.nvfp4_qk_norm_rope_append_paged, rotary_positions=kw.pop("axis_pos", _t(self.axis_pos)),
                rotary_axes=kw.pop("pair_axes", _t(self.pair_axes))))
        return super().call(Axes, **kw)


BLOCKED = [0] * 16 + [1] * 24 + [2] * 24
CASES = [
    # the case of the plain operator, axes, the pairs' axes (None: at random)
    ((1, 1, 1, 1, 16, 2, R.NHD, torch.float16, 16), 1, None),
    ((2, 64, 32, 8, 128, 16, R.HND, torch.bfloat16, 128), 3, BLOCKED),
    ((3, 33, 10, 2, 128, 16, R.NHD, torch.float16, 64, True), 3, [0, 1, 2] * 10 + [0, 0]),
    ((4, 17, 6, 3, 64, 12, R.HND, torch.bfloat16, 64, True, (256.0, 0, 0)), 2, None),
    ((5, 50, 5, 1, 80, 6, R.NHD, torch.float16, 80, False, (256.0, 1, 0)), 8, None),
    ((6, 9, 4, 4, 96, 16, R.HND, torch.bfloat16, 32, False, (448.0, 0, 1)), 3, [2] * 15 + [0]),
    ((7, 21, 7, 1, 192, 64, R.NHD, torch.float16, 192, False, (256.0, 1, 1)), 3, None),
    ((9, 5, 3, 1, 512, 4, R.NHD, torch.float16, 64, True), 4, None),
    ((10, 0, 4, 2, 64, 16, R.NHD, torch.bfloat16, 64), 3, None),
    ((12, 40, 4, 2, 64, 16, R.NHD, torch.bfloat16, 48, True, None, (True, False), False), 3, None),
]
MANY = [
    ((18, 3500, 6, 3, 64, 16, R.NHD, torch.bfloat16, 64), 3, None),
    ((19, 3300, 3, 1, 128, 16, R.HND, torch.float16, 128, True, (256.0, 0, 0)), 2, None),
    ((21, 3300, 4, 4, 128, 16, R.HND, torch.bfloat16, 128), 3, BLOCKED),
]


@pytest.mark.parametrize("i", range(len(CASES) + len(MANY)))
def test_same_bytes_as_rotation_by_axis_then_append(gpu_lib, i):
    args, axes, pair_axes = (CASES + MANY)[i]
    case = AxesCase(*args, axes=axes, pair_axes=pair_axes, **(dict(B=20) if i >= len(CASES) else {}))
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    got, caches = case.call(gpu_lib, status=st)
    assert int(st.item()) == 0
    _same(case, got, caches, case.expect())


def test_one_axis_is_the_plain_rotation(gpu_lib):
    case = Case(2, 64, 32, 8, 128, 16, R.HND, torch.bfloat16, 128)
    want, bytes_ = case.call(gpu_lib)
    same = AxesCase(2, 64, 32, 8, 128, 16, R.HND, torch.bfloat16, 128, axes=2)
    same.table, same.axis_pos = case.table, np.stack([case.pos, case.pos])
    got, other = same.call(gpu_lib, out="in place")
    assert torch.equal(got, want) and all(np.array_equal(x, y) for x, y in zip(bytes_, other))


@pytest.mark.parametrize("bad", [-1, 500, -2 ** 31, 2 ** 31 - 1])
def test_positions_outside_the_table(gpu_lib, bad):
    """A token with one is reported and nothing of it is written; one that no pair goes by does not count."""
    case = AxesCase(2, 64, 32, 8, 128, 16, R.HND, torch.bfloat16, 128, axes=4, pair_axes=BLOCKED)
    q, kc, vc = case.expect()
    pos = case.axis_pos.copy()
    pos[3] = bad
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    got, caches = case.call(gpu_lib, axis_pos=_t(pos), status=st)
    assert int(st.item()) == 0
    _same(case, got, caches, (q, kc, vc))
    pos[1, 10] = pos[2, 33] = bad
    out = torch.full((64, 32, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    got, caches = case.call(gpu_lib, axis_pos=_t(pos), status=st, out=out)
    assert int(st.item()) == gpu_lib.DEV_BAD_POSITION
    keep = np.ones(64, bool)
    keep[[10, 33]] = False
    assert (got[~torch.as_tensor(keep)] == 7.0).all() and torch.equal(got.cpu()[keep], q[keep])
    sub = AxesCase(2, 64, 32, 8, 128, 16, R.HND, torch.bfloat16, 128, axes=4, pair_axes=BLOCKED)
    sub.rows = [x[keep] for x in sub.rows]
    sub.nnz, sub.bi, sub.pos, sub.axis_pos = 62, sub.bi[keep], sub.pos[keep], sub.axis_pos[:, keep]
    _, kc, vc = sub.expect()
    _same(sub, torch.as_tensor(q[keep]), caches, (q[keep], kc, vc))


def test_an_axis_that_is_not_there(gpu_lib):
    case = AxesCase(2, 64, 32, 8, 128, 16, R.HND, torch.bfloat16, 128, axes=3, pair_axes=BLOCKED)
    axes = case.pair_axes.copy()
    axes[5] = 3
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full((64, 32, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    got, caches = case.call(gpu_lib, pair_axes=_t(axes), status=st, out=out)
    assert int(st.item()) == gpu_lib.DEV_BAD_POSITION and (got == 7.0).all()
    assert all((c == 0xA5).all() for c in caches)


def test_cache_positions_need_no_row_of_the_table(gpu_lib):
    """`positions` says only where the rows go: they may lie past the table's end."""
    case = AxesCase(2, 64, 32, 8, 128, 16, R.HND, torch.bfloat16, 128, axes=3, pair_axes=BLOCKED)
    case.table, case.axis_pos = case.table[:20], case.axis_pos % 20
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    got, caches = case.call(gpu_lib, status=st)
    assert int(st.item()) == 0
    _same(case, got, caches, case.expect())


def test_refusals(gpu_lib):
    nv = gpu_lib
    case = AxesCase(2, 64, 32, 8, 128, 16, R.HND, torch.bfloat16, 128, axes=3, pair_axes=BLOCKED)
    ok = dict(axis_pos=_t(case.axis_pos), pair_axes=_t(case.pair_axes))
    for kw, text in ((dict(axis_pos=None), "together"), (dict(pair_axes=None), "together"),
                     (dict(axis_pos=_t(case.axis_pos[0])), "axes, n"), (dict(axis_pos=_t(case.axis_pos[:, :9])), "axes, n"),
                     (dict(axis_pos=_t(case.axis_pos).long()), "Int"), (dict(axis_pos=_t(case.axis_pos).cpu()), "cuda"),
                     (dict(axis_pos=_t(case.axis_pos.T.copy()).T), "contiguous"), (dict(pair_axes=_t(case.pair_axes[:60])), "pairs"),
                     (dict(pair_axes=_t(case.pair_axes).int()), "Byte")):
        with pytest.raises(ValueError, match=text):
            case.call(nv, **{**ok, **kw})
    with pytest.raises(nv.NVFP4KVError, match="num_rotary_axes"):
        case.call(nv, **{**ok, "axis_pos": torch.zeros((9, 64), dtype=torch.int32, device=DEV)})
    with pytest.raises(nv.NVFP4KVError, match="num_rotary_axes"):
        case.call(nv, **{**ok, "axis_pos": torch.zeros((0, 64), dtype=torch.int32, device=DEV)})
