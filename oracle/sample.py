"""Sampling of a row of bf16 logits, in float64 from its definition.

Tokens in order of (logit descending, id ascending), w = exp((x - max) / T);
top-k keeps the first k tokens (mass Z), top-p the shortest prefix of mass at
least p Z, min-p the tokens of w >= min_p; the shortest of the prefixes is
kept, and the pick is the first token whose cumulative mass exceeds u times
the kept mass.
"""

import math

import numpy as np

from .step import bf16_to_f64

NO_LOGITS, BAD_SETTING = 1, 2


def sample_row(bits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(pick, prob, flag) of one row of bf16 bit patterns."""
    x = bf16_to_f64(np.asarray(bits, dtype=np.uint16))
    flag = 0
    if np.isnan(x).any() or (x == np.inf).any() or (x == -np.inf).all():
        flag |= NO_LOGITS
    if not 0 <= temperature < math.inf or math.isnan(top_p) or not min_p <= 1 or not 0 <= u < 1:
        flag |= BAD_SETTING
    if flag:
        return -1, 0.0, flag
    order = np.lexsort((np.arange(len(x)), -x))
    if temperature == 0:
        return int(order[0]), 1.0, 0
    if 0 < top_k < len(x):
        order = order[:top_k]
    w = np.exp((x[order] - x.max()) / temperature)
    mass = np.cumsum(w)
    n = len(order)
    if top_p < 1:
        n = min(n, 1 + int(np.sum(mass < top_p * mass[-1])))
    if min_p > 0:
        n = min(n, int(np.sum(w >= min_p)))
    at = int(np.sum(mass[:n] <= u * mass[n - 1]))
    at = min(at, n - 1)
    return int(order[at]), float(w[at] / mass[n - 1]), 0


def sample_rows(bits, u, temperature=None, top_k=None, top_p=None, min_p=None):
    """sample_row over rows; a setting left None is off (temperature 1)."""
    R = len(bits)
    pick, prob, flag = np.zeros(R, np.int32), np.zeros(R), np.zeros(R, np.uint8)
    for r in range(R):
        kw = {n: float(v[r]) if n != "top_k" else int(v[r]) for n, v in
              (("temperature", temperature), ("top_k", top_k), ("top_p", top_p), ("min_p", min_p)) if v is not None}
        pick[r], prob[r], flag[r] = sample_row(bits[r], float(u[r]), **kw)
    return pick, prob, flag
