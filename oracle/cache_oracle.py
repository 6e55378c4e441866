"""Plain float64 statement of the paged KV cache (test infrastructure only).

The cache of a sequence holds, per page and KV head, `page` slots of d values;
8-bit pages hold codes of a 4-exponent, 3-mantissa-bit float (bias 7, largest
448, no infinities) times one power-of-two scale per page and head.
"""
import numpy as np

E4M3_MAX = 448.0
#: the scale covers the finite magnitudes it is chosen for up to these; 316 for
#: keys before their rotation, since sqrt(2) * 316 < 448
LIM_K, LIM_V = 316.0, 448.0


def round_e4m3(x):
    """Nearest 8-bit value (ties to even), saturating; what is not finite gives NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    _, e = np.frexp(a)                              # a = m 2^e, m in [0.5, 1)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)  # 8 steps per binade, subnormals below 2^-6
    r = np.minimum(np.round(a / step) * step, E4M3_MAX)
    return np.where(np.isfinite(x), np.copysign(r, x), np.nan)


def page_scale(x, lim: float) -> float:
    """Smallest 2^e, -64 <= e <= 64, with |x| <= lim 2^e over the finite x."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x[np.isfinite(x)])
    top = float(a.max()) if a.size else 0.0
    for e in range(-64, 64):
        if top <= lim * 2.0 ** e:
            return 2.0 ** e
    return 2.0 ** 64


def rotate(x, pos, inv_freq, interleaved: bool):
    """x [n, h, d], pos [n]: pair i turned by pos * inv_freq[i]."""
    y = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    ang = np.asarray(pos, dtype=np.float64)[:, None] * np.asarray(inv_freq, dtype=np.float64)
    c, s = np.cos(ang)[:, None, :], np.sin(ang)[:, None, :]
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    u, v = y[..., a].copy(), y[..., b].copy()
    y[..., a], y[..., b] = u * c - v * s, u * s + v * c
    return y


def write_page(held, scale, first: int, raw, new, lim: float):
    """One head of one page: `held` [page, d] values before the write (multiples
    of `scale`), `new` [m, d] unrounded values for the slots from `first` on,
    `raw` the elements their scale is chosen for.  Returns (scale, exact): the
    values of the page before their rounding to 8-bit multiples of the scale,
    what it held below `first` being rounded already."""
    s = page_scale(raw, lim)
    out = np.array(held, dtype=np.float64)
    if first > 0:
        s = max(s, scale)
        out[:first] = round_e4m3(out[:first] / s) * s
    out[first:first + len(new)] = new
    return s, out
