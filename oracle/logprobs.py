"""Oracle: log probabilities of tokens under logits (test infrastructure), plain NumPy in 64 bits.

Per row z: log p = z - log sum e^z, entropy -sum p log p (a logit of -infinity adds nothing), and the columns in
descending order of z, ties to the lowest column, -0.0 just below +0.0.  A row with a NaN or +infinity, or with nothing
above -infinity, is no distribution: NaN everywhere, columns -1.  A token outside the row has NaN.

Parity unpinned by the pages: the benchmark's temperature 0 needs the argmax alone.
"""
from __future__ import annotations

import numpy as np


def row(z, token, top):
    """(log p of token, entropy, log p of the first `top`, their columns) of z float64 [N]."""
    if np.isnan(z).any() or np.isposinf(z).any() or not np.isfinite(z).any():
        return np.nan, np.nan, np.full(top, np.nan), np.full(top, -1)
    m = z.max()
    order = np.lexsort((np.arange(len(z)), np.signbit(z), -z))[:top]
    # the sum without one maximum, so that a sure row keeps its small digits
    rest = np.delete(z, np.argmax(z))
    with np.errstate(over="ignore", under="ignore"):
        e = np.exp(rest - m)
    a = e.sum()
    live = e > 0
    t = (e[live] * (rest[live] - m)).sum()
    lse = np.log1p(a)
    lp = z[token] - m - lse if 0 <= token < len(z) else np.nan
    return lp, lse - t / (1 + a), z[order] - m - lse, order
