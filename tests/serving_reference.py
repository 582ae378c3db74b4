"""Plain 64-bit implementations of the serving operators, for the tests: written from the
definitions, one row and one page at a time, on numpy arrays."""
import math

import numpy as np

MIN_SCALE = 2.0 ** -100


def e4m3_value(code):
    """The number that an e4m3 byte stands for: 1 sign, 4 exponent (bias 7), 3 mantissa bits."""
    sign = -1.0 if code & 0x80 else 1.0
    e, m = (code >> 3) & 15, code & 7
    if e == 15 and m == 7:
        return math.nan
    return sign * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))


VALUES = np.array([e4m3_value(c) for c in range(256)])
_FINITE = VALUES[:127]      # 0 .. 448, ascending; the index is the code


def e4m3_decode(codes):
    return VALUES[np.asarray(codes, dtype=np.uint8)]


def e4m3_round(x):
    """x (float64, |x| <= 448 or not finite) rounded to e4m3, ties to even; not finite -> NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    assert (a <= 448).all()
    hi = np.searchsorted(_FINITE, a)            # first value >= a
    lo = np.maximum(hi - 1, 0)
    down, up = a - _FINITE[lo], _FINITE[hi] - a
    # the code is even where the last mantissa bit is 0
    pick = np.where(_FINITE[hi] == a, hi, np.where(down < up, lo, np.where(
        up < down, hi, np.where(lo % 2 == 0, lo, hi))))
    return np.where(np.isfinite(x), np.copysign(_FINITE[pick], x), np.nan)


def scale_for(amax):
    """The smallest power of two s >= 2^-100 with amax <= 448 s."""
    s = MIN_SCALE
    while 448 * s < amax:
        s *= 2
    return s


def finite_amax(x):
    x = np.abs(x[np.isfinite(x)])
    return float(x.max()) if x.size else 0.0


def append(k, scale, x, pages, page, length, count):
    """One of K and V of one sequence: values k [num_pages, heads, page, d] and scales
    [num_pages, heads] (float64, changed in place) after tokens x [tokens, heads, d]."""
    start = length - count
    for at in range(start // page, -(-length // page)):
        lo, hi = max(start, at * page), min(length, (at + 1) * page)
        for h in range(k.shape[1]):
            pid = pages[at]
            new = x[lo - start:hi - start, h]
            s = scale_for(finite_amax(new))
            if lo > at * page:
                s = max(s, scale[pid, h])
                old = k[pid, h, :lo - at * page]
                k[pid, h, :lo - at * page] = e4m3_round(old * (scale[pid, h] / s))
            k[pid, h, lo - at * page:hi - at * page] = e4m3_round(new / s)
            scale[pid, h] = s


def seen(pos, n, window, sinks):
    """Which of the keys 0 .. n - 1 a query at position pos sees."""
    j = np.arange(n)
    see = j <= pos
    if window:
        see &= (j > pos - window) | (j < sinks)
    return see


def attend(q, k, v, window, sinks):
    """q [t, hq, d], k and v [n, hkv, d] in float64; query i stands at n - t + i.

    Returns o, the sums of w |v| and of w (per K/V head and key), and the largest
    sum of |q k| / sqrt(d) of each row: what the tolerances are made of."""
    t, hq, d = q.shape
    n, hkv = k.shape[:2]
    group = hq // hkv
    o, absv, mass = np.zeros(q.shape), np.zeros(q.shape), np.zeros((hkv, n))
    size = np.zeros((t, hq, 1))
    for i in range(t):
        see = seen(n - t + i, n, window, sinks)
        if not see.any():
            continue
        for h in range(hq):
            kk, vv = k[see, h // group], v[see, h // group]
            with np.errstate(invalid="ignore", over="ignore"):
                x = kk @ q[i, h] / math.sqrt(d)
                w = np.exp(x - x.max())
                w /= w.sum()
                o[i, h] = w @ vv
                absv[i, h] = w @ np.abs(vv)
            mass[h // group, see] += w
            size[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() / math.sqrt(d)
    return o, absv, mass, size


def weight_error(size, d):
    """Bound on the relative error of a softmax weight computed in 32 bits: a score sums d
    products (an addition on the tensor cores may cut off the last bit: 2^-23 of the running sum each)
    and is scaled and referred to the row's maximum (3 roundings of 2^-24); the weight
    and the sum that it is divided by both carry that error; 2^-21 for the exponentials."""
    return 2 * ((d + 3) * 2.0 ** -23 * size) + 2.0 ** -21


def keep(weights, n, budget, sinks, recent):
    """Positions of the tokens that an eviction keeps of n."""
    if n <= budget:
        return list(range(n))
    w = np.where(np.isnan(weights[:n]), -np.inf, weights[:n])
    middle = sorted(range(sinks, n - recent), key=lambda i: (-w[i], i))
    return sorted(list(range(sinks)) + list(range(n - recent, n))
                  + middle[:budget - sinks - recent])
