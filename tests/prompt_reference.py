"""Attention of several new tokens of each request, with sliding windows and first tokens that stay, in 64
bits, written from its formula; and the bounds of what the operators may be off."""
from __future__ import annotations

import math

import numpy as np
import torch

from tests import decode_reference as R


def attention(c: R.Paged, q: np.ndarray, indptr, sm_scale: float, causal: bool = True, soft_cap: float = 0.0,
              window: int = -1, sink: int = 0, num_pages=None):
    """(out, lse, mass, dx) for the rows q [nnz, Hq, D] of the requests' last tokens; rows of no request are NaN
    in `mass`. mass = gs_v sum p |v| / sum p; dx bounds the binary32 error of a score."""
    P = c.k.shape[0] if num_pages is None else num_pages
    nnz, Hq, D = q.shape
    G = Hq // c.H
    out, mass = np.zeros((nnz, Hq, D)), np.full((nnz, Hq, D), np.nan)
    lse, dx = np.full((nnz, Hq), -np.inf), np.zeros((nnz, Hq))
    for b in range(c.B):
        r0, r1 = int(indptr[b]), int(indptr[b + 1])
        L = min(max(int(c.lens[b]), 0), c.tables.shape[1] * c.ps)
        cols = [j for j in range(-(-L // c.ps)) if 0 <= int(c.tables[b, j]) < P]
        t = np.concatenate([np.arange(j * c.ps, min(L, (j + 1) * c.ps)) for j in cols] or [np.zeros(0, int)])
        for h in range(c.H):
            if len(t):
                kk, vv = (np.concatenate([c.rows(w, int(c.tables[b, j]), h)[:L - j * c.ps] for j in cols]) for w in "kv")
            for r in range(r0, r1):
                p = L - (r1 - r0) + (r - r0)
                live = np.ones(len(t), bool)
                if window >= 0:
                    live = (t >= p - window) | (t < sink)
                if causal:
                    live &= t <= p
                heads = slice(h * G, (h + 1) * G)
                mass[r, heads] = 0
                if not live.any():
                    continue
                k, v = kk[live], vv[live]
                f = sm_scale * c.gk
                for g in range(h * G, (h + 1) * G):
                    with np.errstate(invalid="ignore", over="ignore"):
                        x = f * (k @ q[r, g])
                        size = abs(f) * (np.abs(k) @ np.abs(q[r, g])).max()
                        if soft_cap > 0:
                            x = soft_cap * np.tanh(x / soft_cap)
                        m = x.max() if not np.isnan(x).any() else np.nan
                        if m == -np.inf:
                            continue
                        e = np.exp(x - m)
                        out[r, g] = c.gv * (e @ v) / e.sum()
                        mass[r, g] = c.gv * (e @ np.abs(v)) / e.sum()
                        lse[r, g] = m + math.log(e.sum())
                    # a sum of D products, the two factors and the cap's few operations, each 2^-24
                    dx[r, g] = (D + 4) * 2.0 ** -24 * size + 8 * 2.0 ** -24 * max(abs(soft_cap), np.abs(x).max())
    return out, lse, mass, dx


def check(got_out, got_lse, ref, dtype):
    """Equal where the formula is NaN or infinite, else within the roundings."""
    out, lse, mass, dx = ref
    rows = ~np.isnan(mass[:, 0]).all(-1) | np.isnan(out[:, 0]).all(-1)
    half = torch.finfo(dtype).eps / 2
    o, s = got_out.double().cpu().numpy()[rows], got_lse.double().cpu().numpy()[rows]
    out, lse, mass, dx = out[rows], lse[rows], mass[rows], dx[rows]
    nan = np.isnan(out)
    assert (np.isnan(o) == nan).all(), ("NaN", np.argwhere(np.isnan(o) != nan)[0].tolist())
    # the weights are rounded to binary16 (2^-11; 2^-25 of 2^8 where they are subnormal) and exp is a few 2^-22 off;
    # both errors of a weight count in the product and, but for the rounding, in the sum; then the output's rounding
    tol = half * np.abs(out) + (2.0 ** -11 + 2 * dx[..., None] + 2.0 ** -18) * mass * (1 + half) + 2.0 ** -25
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(o - out) <= tol) & ~nan
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[0].tolist(), o[bad][0], out[bad][0], tol[bad][0])
    nan, fin = np.isnan(lse), np.isfinite(lse)
    assert (np.isnan(s) == nan).all()
    assert (s[~fin & ~nan] == lse[~fin & ~nan]).all()
    d = np.abs(s[fin] - lse[fin])
    assert (d <= dx[fin] + 2.0 ** -18 + 2.0 ** -22 * np.abs(lse[fin])).all(), d.max()


def with_f32_scales(c: R.Paged) -> R.Paged:
    return R.Paged(**{**c.__dict__, "gk": float(np.float32(c.gk)), "gv": float(np.float32(c.gv))})
