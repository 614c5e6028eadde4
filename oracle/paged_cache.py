"""fp64 definition of the paged 8-bit key/value cache: appending, attention and page selection.

A cache is kept as plain arrays: e4m3 values as the numbers they are (without the scale) `vals` [n_pages, 2, hkv,
page, d], `scales` [n_pages, 2, hkv] and key bounds `bounds` [n_pages, hkv, 2, d].
"""
import numpy as np

from .msa_oracle import apply_rope

E4M3_MAX = 448.0
SCALE_MIN, SCALE_MAX = -50, 50


def decode_e4m3(b):
    """Values of e4m3 bytes: sign, 4 exponent bits (bias 7), 3 fraction bits; 0x7f and 0xff are NaN."""
    b = np.asarray(b, dtype=np.uint8).astype(np.int64)
    e, f = (b >> 3) & 15, b & 7
    x = np.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * 2.0 ** (e - 7.0))
    x = np.where((e == 15) & (f == 7), np.nan, x)
    return np.where(b >> 7, -x, x)


def round_e4m3(x):
    """To the nearest e4m3 value, halves to even, magnitudes above 448 to 448."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), E4M3_MAX)
    step = 2.0 ** (np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    return np.copysign(np.minimum(np.round(a / step) * step, E4M3_MAX), x)


def needed_scale(amax):
    """The smallest power of two s in range with amax <= 448 s."""
    amax = np.asarray(amax, dtype=np.float64)
    with np.errstate(divide="ignore"):
        e = np.ceil(np.log2(amax / E4M3_MAX))
    return 2.0 ** np.clip(e, SCALE_MIN, SCALE_MAX)


def append(vals, scales, bounds, pages, base, k, v, pos_offset=0, rope_base=1.0e6):
    """Appends k, v [n, hkv, d] to a sequence of `base` tokens kept in `pages`; the arrays are changed in place.
    Returns the rotated keys before rounding."""
    page = vals.shape[3]
    n = len(k)
    kr = apply_rope(np.asarray(k, np.float64), pos_offset + base + np.arange(n), rope_base)
    for p in range(base // page, -(-(base + n) // page) if n else 0):
        pid = pages[p]
        r0, r1 = max(base - p * page, 0), min(base + n - p * page, page)
        rows = np.stack((kr, np.asarray(v, np.float64)))[:, p * page + r0 - base:p * page + r1 - base]
        rows = rows.transpose(0, 2, 1, 3)                                   # [2, hkv, rows, d]
        fin = np.where(np.isfinite(rows), rows, 0.0)
        new = needed_scale(np.abs(fin).max((-1, -2)))
        if r0 > 0:
            new = np.maximum(new, scales[pid])
            vals[pid, :, :, :r0] = round_e4m3(vals[pid, :, :, :r0] * (scales[pid] / new)[..., None, None])
        rows = np.where(np.isnan(rows), 0.0, np.clip(rows, -1e300, 1e300))
        vals[pid, :, :, r0:r1] = round_e4m3(rows / new[..., None, None])
        scales[pid] = new
        keys = vals[pid, 0, :, :r1] * new[0][:, None, None]
        bounds[pid, :, 0], bounds[pid, :, 1] = keys.min(1), keys.max(1)
    return kr


def rows_of(vals, scales, pages, length, part, head):
    """Keys (part 0) or values (part 1) of a sequence of `length` tokens [length, d]."""
    pages = np.asarray(pages[:-(-length // vals.shape[3])], dtype=np.int64)
    x = vals[pages, part, head] * scales[pages, part, head][:, None, None]
    return x.reshape(-1, vals.shape[-1])[:length]


def attend(q, k, v, visible, scale):
    """One query row over keys k, v [len, d], of which `visible` [len] count -> (out [d], lse); (0, -inf) without any."""
    if not visible.any():
        return np.zeros(v.shape[1]), -np.inf
    s = k[visible] @ q * scale
    m = s.max()
    p = np.exp(s - m)
    return p @ v[visible] / p.sum(), m + np.log(p.sum())


def page_scores(q, lo, hi):
    """q [G, d], lo and hi [pages, d] -> [pages]: the largest dot product of any head with any key inside the bounds."""
    return np.maximum(q[:, None] * lo, q[:, None] * hi).sum(-1).max(0)


def pick(scores, k, recent):
    """The k best of the visible pages in ascending order, the `recent` newest first of all, ties to the lower page,
    padded with -1."""
    s = np.array(scores, dtype=np.float64)
    s[max(0, len(s) - recent):] = np.inf
    best = sorted(sorted(range(len(s)), key=lambda p: (-s[p], p))[:k])
    return np.array(best + [-1] * (k - len(best)), dtype=np.int32)
