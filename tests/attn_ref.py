"""64-bit references of the 4-bit cache and the attention calls (numpy, from
the definitions), and the error bounds their tests use.

Bounds.  u = half a unit of the 16-bit type relative to the value (2^-8 bf16,
2^-11 fp16).  A computed score differs from the exact one by at most
dx = (D + 16) 2^-24 S + |x| 2^-22, S the largest scale * sum |q_d k_d| of the
row: D products summed in FP32 in any order, the scaling, and exp2's argument.
Each weight is then off by a factor within 1 +- (dx + 2^-22) before it is
rounded to the 16-bit type (u; in fp16 also 2^-25 absolutely, below its normal
range).  The sum that the output is divided by is of the rounded weights, so
their roundings e_i (|e_i| <= u) enter as sum w_i e_i (v_i - out), w_i the
normalised weights: at most u (A + |out|), A = sum w_i |v_i|.  With the output's
own rounding, u |out|:
  |out - exact| <= A (u + 2 dx + 2^-21 + 2 N 2^-24) + 2 u |exact| + fp16's
  absolute terms,  |lse - exact| <= dx + 2^-21 + 2 N 2^-24 + |lse| 2^-22.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def quantise(x: np.ndarray):
    """x [..., D] float64 -> (codes [..., D/2], scale bytes [..., D/32]) uint8."""
    g = x.reshape(*x.shape[:-1], -1, 32)
    top = np.abs(g).max(-1)
    bad = ~np.isfinite(top)
    _, ex = np.frexp(np.where(bad | (top == 0), 1.0, top))
    e = np.clip(ex - 3, -120, 125)
    e = np.where(top == 0, -120, e)
    y = np.where(bad[..., None], 0.0, np.abs(np.where(np.isfinite(g), g, 0.0))) / np.ldexp(1.0, e)[..., None]
    d = np.abs(y[..., None] - E2M1)
    near = d == d.min(-1, keepdims=True)
    # the nearest value; of two equally near the even code
    code = np.where(near.sum(-1) == 1, near.argmax(-1), 0)
    first = near.argmax(-1)
    code = np.where(near.sum(-1) == 2, first + (first & 1), code)
    code = code + 8 * np.signbit(g)
    code = np.where(bad[..., None], 0, code).reshape(x.shape).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), np.where(bad, 255, e + 127).astype(np.uint8)


def dequantise(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = np.where(c >= 8, -1.0, 1.0) * E2M1[c & 7]
    unit = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return (v.reshape(*v.shape[:-1], -1, 32) * unit[..., None]).reshape(v.shape)


def attend_row(q, k, v, scale):
    """q [hq, D], k and v [n, hkv, D] of the keys the row sees, all float64.
    Returns out [hq, D], lse [hq] and per head (A [hq, D], dx [hq])."""
    hq, d = q.shape
    n, hkv = k.shape[:2]
    out, lse = np.zeros((hq, d)), np.full(hq, -np.inf)
    A, dx = np.zeros((hq, d)), np.zeros(hq)
    if n == 0:
        return out, lse, A, dx
    for h in range(hq):
        g = h // (hq // hkv)
        with np.errstate(invalid="ignore", over="ignore"):
            x = scale * (k[:, g] @ q[h])
            S = abs(scale) * (np.abs(k[:, g]) @ np.abs(q[h]))
            top = x.max()
            p = np.exp(x - top)
            out[h] = (p[:, None] * v[:, g]).sum(0) / p.sum()
            A[h] = (p[:, None] * np.abs(v[:, g])).sum(0) / p.sum()
            lse[h] = top + np.log(p.sum())
            dx[h] = (d + 16) * 2.0 ** -24 * S.max() + np.abs(x).max() * 2.0 ** -22
    return out, lse, A, dx


def check_rows(got, got_lse, want, kind, n_keys, vmax):
    """want: list of attend_row results; got [rows, hq, D] float64."""
    u = UNIT[kind]
    for r, (out, lse, A, dx) in enumerate(want):
        N = n_keys[r]
        tol = A * (u + 2 * dx[:, None] + 2.0 ** -21 + 2 * N * 2.0 ** -24) + 2 * u * np.abs(out) + 2.0 ** -40
        if kind == "f16":
            tol = tol + 2.0 ** -25 * (1 + N * vmax)
        fin = np.isfinite(out)
        assert np.array_equal(np.isnan(out), np.isnan(got[r])), f"row {r}: NaN pattern"
        assert np.array_equal(out[~fin & ~np.isnan(out)], got[r][~fin & ~np.isnan(out)]), f"row {r}: infinities"
        err = np.abs(np.where(fin, got[r], 0.0) - np.where(fin, out, 0.0))
        bad = fin & ~(err <= tol)
        assert not bad.any(), f"row {r}: {bad.sum()} values off, worst {np.max(np.where(fin, err / np.maximum(tol, 1e-300), 0))} tolerances"
        if got_lse is not None:
            f = np.isfinite(lse)
            assert np.array_equal(np.isneginf(lse), np.isneginf(got_lse[r])), f"row {r}: empty heads"
            el = np.abs(got_lse[r][f] - lse[f])
            assert np.all(el <= (dx + 2.0 ** -21 + 2 * N * 2.0 ** -24)[f] + np.abs(lse[f]) * 2.0 ** -22), f"row {r}: lse {el.max()}"
