"""Comparison of the row sampler's answers with row_oracle's, within the bounds
that include/resident_topk.h states.

A weight w (of the largest, 1) becomes w (1 + d) + e with |d| <= 2^-43 and |e| at
most 1.1 units: half a unit where it is rounded alone; where a histogram sums it,
0.52 for the four roundings of its quartic and half a unit for its bin.  A sum S
of n weights is off by at most n 1.1 unit + S 2^-43, and so is a running part of
it; the part's share of the sum by twice that over S.  Every sum that decides is at
least that of the kept weights, so with S that one bounds them all."""
import numpy as np

import row_oracle

DEFAULTS = (("temperature", 1.0), ("top_k", 0), ("top_p", 1.0), ("min_p", 0.0))


def _column(value, r):
    return value.cpu().numpy() if hasattr(value, "cpu") else [value] * r


def share_error(x, token, prob, temperature):
    """The bound above for a row, from its drawn token's weight and share: S = w / prob."""
    v = len(x)
    unit = 2.0 ** -min(46, 62 - int(np.ceil(np.log2(v))))
    w = np.exp((x[token] - np.nanmax(x)) / temperature)
    return 2.0 * (v * 1.1 * unit * prob / w + 2.0 ** -43)


def check(token, prob, x, u, exact_ties=False, **settings):
    """token, prob (None: not looked at), x, u as host tensors: every row is the
    definition's.  Rows have to keep clear of the borders (asserted) unless
    exact_ties says that whole weights decide theirs."""
    token, rows, u = token.numpy(), x.double().numpy(), u.numpy()
    r = len(rows)
    s = {k: _column(settings.get(k, d), r) for k, d in DEFAULTS}
    for i in range(r):
        one = {k: s[k][i] for k in s}
        one["top_k"] = int(one["top_k"])
        e, p, margin, _ = row_oracle.draw(rows[i], u[i], **one)
        t = float(np.float32(one["temperature"]))
        error = share_error(rows[i], e, p, t) if e >= 0 and t > 0 else 0.0
        assert exact_ties or margin > error, ("the test's own row sits on a border", i, margin, error)
        assert token[i] == e, (i, token[i], e, margin)
        if prob is not None:  # the sum's error, the weight's own and one rounding to fp32
            assert abs(float(prob[i]) - p) <= p * (2.0 ** -24 + error) * 1.01 + 2.0 ** -149, (i, prob[i], p)
