"""Top-k, top-p and min-p of a row of logits: the oracle (test infrastructure only).

A request that samples (oracle/sample.py; openinfer PR #626, Summary) may cut
the target's probabilities first. The tokens are sorted by logit, equal ones by
index, and walked through one by one.

Readings: top-k first, top-p as a share of what top-k leaves, min-p beside the
largest probability; top-p keeps the token that reaches the share; NaN, a top-k
outside [1, V], a top-p from 1 on and a min-p up to 0 limit nothing, a min-p
over 1 counts as 1.

Pins (tests/test_oracle_filter.py): hand-worked rows; each limit alone against
its one-line definition.
"""
from __future__ import annotations

import numpy as np

from .common import widen
from .sample import probabilities


def filtered(row, tau: float, k: int = 0, p: float = 1.0, m: float = 0.0):
    """(probabilities of the tokens that stay, zero elsewhere; how many stay)."""
    z = widen(row)
    full = probabilities(row, tau)
    order = [int(i) for i in np.lexsort((np.arange(len(z)), -np.where(np.isnan(z), -np.inf, z)))]
    order = [i for i in order if not np.isnan(z[i])]
    if not order or not full.any():
        return full, len(order)
    if 1 <= k <= len(z):
        order = order[:k]
    if p < 1:
        share, c, stay = max(float(p), 0.0) * float(np.sum(full[order])), 0.0, 0
        for i in order:
            if stay and c >= share:
                break
            c += full[i]
            stay += 1
        order = order[:stay]
    if m > 0:
        ratio = full / np.max(full)
        order = [i for i in order if ratio[i] >= min(m, 1.0)]
    out = np.zeros_like(full)
    out[order] = full[order]
    return out / np.sum(out), len(order)
