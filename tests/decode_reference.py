"""The decode-step operators in 64 bits (norm and rotation: in their own binary32 order), written
from their formulas on the CPU, and the inputs that their tests share."""
from __future__ import annotations

import math
from dataclasses import dataclass
from typing import Optional

import numpy as np
import torch

NHD, HND = 0, 1
MAG = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_values() -> np.ndarray:
    out = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[b] = math.nan if (b & 127) == 127 else (-v if b & 128 else v)
    return out


def decode(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """codes [..., D/2], scale bytes [..., D/16] -> e2m1 * S, float64 [..., D]."""
    val = np.concatenate([MAG, -MAG])
    x = np.stack([val[codes & 15], val[codes >> 4]], -1).reshape(*codes.shape[:-1], -1)
    with np.errstate(invalid="ignore"):
        return x * np.repeat(e4m3_values()[scales], 16, axis=-1)


@dataclass
class Paged:
    """A paged K and V cache on the host and its tables. Slots past a request's end and pages of
    no request hold garbage, NaN scales among it."""
    B: int
    H: int
    D: int
    ps: int
    layout: int
    lens: np.ndarray
    tables: np.ndarray
    k: np.ndarray    # codes [pages, ., ., D/2]
    ks: np.ndarray   # scales [pages, ., ., D/16]
    v: np.ndarray
    vs: np.ndarray
    gk: float
    gv: float

    def rows(self, which: str, page: int, h: int) -> np.ndarray:
        """e2m1 * S of one head's slots of a page, [ps, D]."""
        c, s = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        if self.layout == NHD:
            return decode(c[page, :, h], s[page, :, h])
        return decode(c[page, h], s[page, h])


def make_paged(seed: int, lens, H: int, D: int, ps: int, layout: int, spare: int = 3,
               table_dtype=np.int32, width: Optional[int] = None) -> Paged:
    rng = np.random.Generator(np.random.PCG64(seed))
    lens = np.asarray(lens, np.int32)
    pages = (np.maximum(lens, 0) + ps - 1) // ps
    P = int(pages.sum()) + spare
    w = max(int(pages.max(initial=0)), 1) if width is None else width
    tables = np.full((len(lens), w), -1, table_dtype)
    perm = rng.permutation(P)
    at = 0
    inner = (ps, H) if layout == NHD else (H, ps)
    k, v = (rng.integers(0, 256, (P, *inner, D // 2), dtype=np.uint8) for _ in range(2))
    ks, vs = (rng.integers(0x60, 0x7B, (P, *inner, D // 16), dtype=np.uint8) for _ in range(2))
    dead = np.ones((P, ps), bool)
    for b, n in enumerate(lens):
        for j in range(pages[b]):
            p = perm[at + j]
            tables[b, j] = p
            dead[p, : max(0, min(ps, n - j * ps))] = False
        at += pages[b]
    for s in (ks, vs):
        view = s if layout == NHD else s.transpose(0, 2, 1, 3)
        view[dead] = rng.choice(np.array([0x7F, 0xFF, 0x7E, 0x00], np.uint8), view[dead].shape)
    return Paged(len(lens), H, D, ps, layout, lens, tables, k, ks, v, vs, 0.0021, 0.0017)


def attention(c: Paged, q: np.ndarray, sm_scale: float, soft_cap: float = 0.0, window: int = -1,
              selected=None, num_selected=None, num_pages: Optional[int] = None):
    """(out, lse, mass, dx): mass = gs_v sum p |v| / sum p; dx bounds the binary32 error of a score."""
    P = c.k.shape[0] if num_pages is None else num_pages
    B, Hq, D = q.shape
    G = Hq // c.H
    out, mass = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    lse, dx = np.full((B, Hq), -np.inf), np.zeros((B, Hq))
    for b in range(B):
        n = min(int(c.lens[b]), c.tables.shape[1] * c.ps)
        lo = max(0, n - 1 - window) if window >= 0 else 0
        for h in range(c.H):
            cols = range(max(-(-n // c.ps), 0))
            if selected is not None:
                cols = [int(x) for x in selected[b, h, :max(0, int(num_selected[b, h]))]]
            kk, vv = [], []
            for j in cols:
                if not 0 <= j < c.tables.shape[1]:
                    continue
                p = int(c.tables[b, j])
                if not 0 <= p < P:
                    continue
                a, e = max(lo - j * c.ps, 0), min(c.ps, n - j * c.ps)
                if a < e:
                    kk.append(c.rows("k", p, h)[a:e])
                    vv.append(c.rows("v", p, h)[a:e])
            if not kk:
                continue
            kk, vv = np.concatenate(kk), np.concatenate(vv)
            for g in range(h * G, (h + 1) * G):
                f = sm_scale * c.gk
                x = f * (kk @ q[b, g])
                size = abs(f) * (np.abs(kk) @ np.abs(q[b, g])).max()
                if soft_cap > 0:
                    x = soft_cap * np.tanh(x / soft_cap)
                m = x.max()
                p = np.exp(x - m)
                out[b, g] = c.gv * (p @ vv) / p.sum()
                mass[b, g] = c.gv * (p @ np.abs(vv)) / p.sum()
                lse[b, g] = m + math.log(p.sum())
                # a sum of D products, the two factors and the cap's few operations, each 2^-24
                dx[b, g] = (D + 4) * 2.0 ** -24 * size + 8 * 2.0 ** -24 * max(abs(soft_cap), np.abs(x).max())
    return out, lse, mass, dx


def check_attention(got_out, got_lse, ref, dtype):
    out, lse, mass, dx = ref
    half = torch.finfo(dtype).eps / 2
    o = got_out.double().cpu().numpy()
    # the weights are rounded to binary16 (2^-11) and exp is a few 2^-22 off; both errors of a weight count
    # in the product and, but for the rounding, in the sum; then the output's rounding, subnormals included
    tol = half * np.abs(out) + (2.0 ** -11 + 2 * dx[..., None] + 2.0 ** -18) * mass * (1 + half) + 2.0 ** -25
    bad = ~(np.abs(o - out) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[0].tolist(), o[bad][0], out[bad][0], tol[bad][0])
    s = got_lse.double().cpu().numpy()
    fin = np.isfinite(lse)
    assert (s[~fin] == -np.inf).all()
    d = np.abs(s[fin] - lse[fin])
    assert (d <= dx[fin] + 2.0 ** -18 + 2.0 ** -22 * np.abs(lse[fin])).all(), d.max()


# ---- norm, rotation -------------------------------------------------------------------------

def _half_sum(t: np.ndarray) -> np.ndarray:
    while t.shape[-1] > 1:
        n = t.shape[-1] // 2
        t = t[..., :n] + t[..., n:]
    return t[..., 0]


def norm_rope(x: np.ndarray, w, eps: float, table, pos, inter: bool) -> np.ndarray:
    """Rows x [n, heads, D] float32 -> float32 before the final rounding, in the operator's order."""
    f = np.float32
    D = x.shape[-1]
    rot = 0 if table is None else table.shape[1]
    y = x.astype(f)
    if w is not None:
        groups = _half_sum((y * y).reshape(*y.shape[:-1], D // 8, 8))
        nr, nt = rot // 16, D // 16
        pair = np.stack([groups[..., j] + groups[..., j + nr] if j < nr
                         else groups[..., 2 * j] + groups[..., 2 * j + 1] for j in range(nt)], -1)
        full = np.zeros((*pair.shape[:-1], 1 << (nt - 1).bit_length()), f)
        full[..., :nt] = pair
        r = f(1) / np.sqrt(_half_sum(full) * f(1.0 / D) + f(eps))
        y = (y * r[..., None]) * w.astype(f)
    if rot:
        c, s = table[pos][:, None, :rot // 2], table[pos][:, None, rot // 2:]
        ia = np.arange(0, rot, 2) if inter else np.arange(rot // 2)
        ib = ia + (1 if inter else rot // 2)
        a, b = y[..., ia].copy(), y[..., ib].copy()
        y[..., ia] = a * c - b * s
        y[..., ib] = b * c + a * s
    assert y.dtype == f
    return y


def cos_sin(positions: int, rot: int, base: float = 10000.0) -> np.ndarray:
    ang = np.arange(positions)[:, None] * base ** (-np.arange(rot // 2) * 2.0 / rot)
    return np.concatenate([np.cos(ang), np.sin(ang)], -1).astype(np.float32)


# ---- pages ----------------------------------------------------------------------------------

def key_bounds(c: Paged, first=None):
    """{page: (lo [H, D], hi [H, D])} of the pages that the call writes."""
    out = {}
    for b in range(c.B):
        n = min(int(c.lens[b]), c.tables.shape[1] * c.ps)
        j0 = 0 if first is None else max(int(first[b]), 0) // c.ps
        for j in range(j0, -(-n // c.ps) if n > 0 else 0):
            p = int(c.tables[b, j])
            if not 0 <= p < c.k.shape[0]:
                continue
            x = np.stack([c.rows("k", p, h)[: n - j * c.ps] for h in range(c.H)])
            out[p] = (x.min(1), x.max(1))
    return out


def page_scores(q: np.ndarray, bounds: np.ndarray) -> np.ndarray:
    """q [G, D] float32, bounds [n, 2, D] float32 -> scores [n] float32 in the operator's order."""
    f = np.float32
    t = np.where(q[None] > 0, q[None] * bounds[:, None, 1], q[None] * bounds[:, None, 0]).astype(f)
    t = t.reshape(*t.shape[:-1], -1, 4, 2)
    chain = ((t[..., 0, :] + t[..., 1, :]) + t[..., 2, :]) + t[..., 3, :]
    s = chain[..., 0] + chain[..., 1]
    full = np.zeros((*s.shape[:-1], 1 << (s.shape[-1] - 1).bit_length()), f)
    full[..., : s.shape[-1]] = s
    return _half_sum(full).max(1)


def select(scores: np.ndarray, k: int, sink: int, recent: int) -> list:
    n = len(scores)
    forced = [j < sink or j >= n - recent for j in range(n)]
    order = sorted(range(n), key=lambda j: (not forced[j], 0.0 if forced[j] else -float(scores[j]), j))
    return sorted(order[:k])
