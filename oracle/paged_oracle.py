"""Float64 oracle of the paged 8-bit cache: e4m3 rounding, page scales, position
rotation, appends into pages and reading them back.

Plain numpy from the definitions, sharing no code with the CUDA library.  The
attention over what is read back is aqua_oracle.decode / prefill.
"""
from __future__ import annotations

import numpy as np

SCALE_MIN_EXP = -60

# The 127 non-negative e4m3 numbers by code: four exponent bits (bias 7), three
# of mantissa, subnormals below 2^-6, no infinity; code 127 is NaN.
_POS = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7) for c in range(127)])


def e4m3_decode(code) -> np.ndarray:
    """Codes (uint8) -> the float64 numbers they stand for."""
    c = np.asarray(code, dtype=np.uint8).astype(np.int64)
    mag = np.append(_POS, np.nan)[c & 127]
    return np.where(c >= 128, -mag, mag)


def e4m3_round(x) -> np.ndarray:
    """The nearest e4m3 number of each x (ties to the even code, saturating at 448, NaN kept)."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    with np.errstate(invalid="ignore"):
        hi = np.searchsorted(_POS, np.where(np.isnan(a), 0.0, a), side="left")
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.where(np.isnan(x), np.nan, np.copysign(_POS[pick], x))


def page_scale(amax: float) -> float:
    """The smallest power of two s >= 2^-60 with amax <= 448 s."""
    e = SCALE_MIN_EXP
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def rotate(x, pos, cos_sin, interleaved: bool) -> np.ndarray:
    """Rows x [n, heads, d] with their first rot dimensions rotated to positions pos [n]."""
    x = np.asarray(x, dtype=np.float64).copy()
    if cos_sin is None:
        return x
    t = np.asarray(cos_sin, dtype=np.float64)
    rot = t.shape[1]
    for n, p in enumerate(pos):
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            c, s = t[p, i], t[p, rot // 2 + i]
            xa, xb = x[n, :, a].copy(), x[n, :, b].copy()
            x[n, :, a] = xa * c - xb * s
            x[n, :, b] = xa * s + xb * c
    return x


def finite_max(x) -> float:
    """The largest finite magnitude (0 if there is none): what sets a page's scale."""
    a = np.abs(np.asarray(x, dtype=np.float64))
    a = a[np.isfinite(a)]
    return float(a.max()) if a.size else 0.0


def append_to_block(old, old_scale: float, fill: int, new, scale: float) -> np.ndarray:
    """Code values of one page and head after an append, tokens first.

    old [page, dims]: code values before; new [n, dims]: the appended rows;
    scale: the page's scale afterwards.  Slots past fill + n keep their codes.
    """
    out = np.array(old, dtype=np.float64)
    if fill > 0 and scale != old_scale:
        out[:fill] = e4m3_round(out[:fill] * (old_scale / scale))
    out[fill:fill + len(new)] = e4m3_round(np.asarray(new, dtype=np.float64) / scale)
    return out


def read_sequence(k_codes, v_codes, k_scale, v_scale, table_row, n: int):
    """K~ [Hkv, n, m] and V [Hkv, n, d] of one sequence from the pages."""
    page = v_codes.shape[2]
    ks, vs = [], []
    for t in range(n):
        p, s = int(table_row[t // page]), t % page
        ks.append(e4m3_decode(k_codes[p, :, :, s]) * np.asarray(k_scale[p], dtype=np.float64)[:, None])
        vs.append(e4m3_decode(v_codes[p, :, s]) * np.asarray(v_scale[p], dtype=np.float64)[:, None])
    if not ks:
        return np.zeros((k_codes.shape[1], 0, k_codes.shape[2])), np.zeros((v_codes.shape[1], 0, v_codes.shape[3]))
    return np.stack(ks, 1), np.stack(vs, 1)
