"""Plain 64-bit definitions of the int8 row products and the row sampler
(numpy, one row at a time where order matters), sharing no code with the
library."""
import numpy as np


def quantize_rows(x):
    """x float64 [m, k] holding values of the input type.  (codes int8, scale float64)."""
    with np.errstate(invalid="ignore"):
        amax = np.max(np.abs(x), axis=1)
    bad = ~np.isfinite(x).all(axis=1)
    with np.errstate(invalid="ignore", over="ignore"):
        scale = (amax.astype(np.float32) / np.float32(127)).astype(np.float32).astype(np.float64)
    scale[scale < 2.0 ** -126] = 0.0
    scale[bad] = np.nan
    codes = np.zeros(x.shape, np.int8)
    for i in range(x.shape[0]):
        if scale[i] > 0:
            s = scale[i]
            n = np.floor(x[i] / s)
            rest = 2.0 * (x[i] - n * s)  # exact: n has 8 bits, s 24
            up = (rest > s) | ((rest == s) & (n % 2 == 1))
            codes[i] = (n + up).astype(np.int8)
    return codes, scale


def product(a, a_scale, b, b_scale, bias=None):
    """(float64 result, float64 |product| before the bias)."""
    y = (a.astype(np.float64) @ b.astype(np.float64).T) * a_scale.astype(np.float64)[:, None] \
        * b_scale.astype(np.float64)[None, :]
    return (y if bias is None else y + bias.astype(np.float64)), np.abs(y)


def draw(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, probability, margin, error): margin is how far, as a share of the
    sums, the decisions stay from falling the other way (0 where one is an exact
    tie that whole weights decide); error is how far the shares of sums of whole
    weights can be off: each weight by half a unit of 2^-shift of the largest and
    2^-46 of itself, so a sum z of n weights by n unit / 2 + z 2^-46, and a
    running sum as a share of it by twice that over z; where top-p takes its
    sums from a histogram, 2^-37 of itself instead."""
    unit = 2.0 ** -min(46, 62 - int(np.ceil(np.log2(len(x)))))
    error = 0.0
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64))
    t, p, least, u = (float(np.float32(s)) for s in (temperature, top_p, min_p, u))
    top = x.max()
    if top == -np.inf:
        return -1, 0.0, 1.0, 0.0
    order = np.argsort(-x, kind="stable")
    if not t > 0:
        return int(order[0]), 1.0, 1.0, 0.0
    with np.errstate(invalid="ignore", under="ignore", over="ignore"):
        w = np.exp((x - top) / t)
    w = np.where(x == top, 1.0, np.where(x == -np.inf, 0.0, w))
    w = np.where(np.isnan(w), 0.0, w)
    margin = 1.0
    n = len(x) if top_k <= 0 else min(top_k, len(x))
    if not p >= 1:
        run = np.cumsum(w[order[:n]])
        before = np.concatenate([[0.0], run[:-1]])
        z = run[-1]
        inside = before < p * z
        error = (n * unit + z * 2.0 ** -36) / z
        inside[0] = True
        if p > 0:
            margin = min(margin, np.min(np.abs(before[1:] - p * z)) / z if n > 1 else 1.0)
        n = int(np.count_nonzero(inside))
    kept = np.zeros(len(x), bool)
    kept[order[:n]] = True
    if not least <= 0:
        ok = w >= least
        near = np.abs(w - least)[(w > 0) & (w != least)]
        if near.size:
            margin = min(margin, near.min())
        kept &= ok
        kept[order[0]] = True
        if not least <= 1:
            kept[:] = False
            kept[order[0]] = True
    wk = np.where(kept, w, 0.0)
    run = np.cumsum(wk)
    s = run[-1]
    error = max(error, (np.count_nonzero(kept) * unit + s * 2.0 ** -45) / s)
    if not u > 0:
        token = int(np.flatnonzero(wk > 0)[0])
    elif u >= 1:
        token = int(np.flatnonzero(wk > 0)[-1])
    else:
        token = int(np.argmax(run > u * s))
        live = run[wk > 0]
        margin = min(margin, np.min(np.abs(live - u * s)) / s)
    return token, float(wk[token] / s), float(margin), float(error)
