"""Acceptance of drafts by sampling: the oracle (test infrastructure only).

Greedy acceptance (accept.py) keeps a draft that equals the target's argmax
(openinfer PR #626, Summary). A request that samples keeps a draft with a
probability that leaves the target's distribution unchanged: with p the
target's and q the draft's distribution at the parent, a token x drawn from q
is kept when u q(x) < p(x), and otherwise the next token is drawn from
max(p - q, 0). A token that was picked rather than drawn has q = 1 at itself:
it is kept when u (mass left) < p(x), and leaves the rest when it is not.

All in float64. Readings: NaN logits have weight zero; +inf logits share the
weight; temperature 0 shares it among the largest logits; a row without any
finite or +inf logit has p = 0 and bonus 0; a rest of zero falls back to p;
the drawn token is the first whose cumulative weight passes u times the total,
the last positive one if none does.

Pins (tests/test_oracle_sample.py): scipy-free softmax identities; exact
enumeration over a grid of random numbers reproduces p on tiny vocabularies
for chains with and without draft probabilities and for trees.
"""
from __future__ import annotations

import dataclasses
from typing import Optional

import numpy as np

from .common import widen


def probabilities(row, tau: float) -> np.ndarray:
    z = widen(row).copy()
    ok = ~np.isnan(z)
    m = np.max(z[ok]) if ok.any() else -np.inf
    if m == -np.inf:
        return np.zeros_like(z)
    w = np.zeros_like(z)
    if tau == 0 or m == np.inf:
        w[ok & (z == m)] = 1.0
    else:
        fin = ok & (z > -np.inf)
        w[fin] = np.exp((z[fin] - m) / tau)
    return w / np.sum(w)


@dataclasses.dataclass
class SampleResult:
    accept_node: int
    accept_len: int
    path: np.ndarray
    bonus: int
    token_prob: np.ndarray
    accept_margin: float     # smallest |u q - p| / max over the decisions made
    bonus_margin: float      # distance of u from the drawn token's borders, in total weights


def draw(weights: np.ndarray, u: float):
    """(token, distance to the nearest border of its interval)."""
    c = np.cumsum(weights)
    hit = np.flatnonzero((weights > 0) & (c > u * c[-1]))
    v = int(hit[0]) if len(hit) else int(np.flatnonzero(weights > 0)[-1])
    lo = (c[v] - weights[v]) / c[-1]
    return v, min(abs(u - lo) if lo > 0 else 1.0, abs(c[v] / c[-1] - u) if c[v] < c[-1] else 1.0)


def accept(logits, tokens, uniforms, draft=None, tau: float = 1.0, parent: Optional[np.ndarray] = None) -> SampleResult:
    T, V = np.asarray(logits).shape
    parent = np.arange(-1, T - 1) if parent is None else np.asarray(parent)
    tokens = np.asarray(tokens)
    u = np.asarray(uniforms, dtype=np.float64)
    p = np.stack([probabilities(logits[t], tau) for t in range(T)])
    prob = np.ones(T)
    for t in range(1, T):
        x = int(tokens[t])
        prob[t] = p[parent[t], x] if 0 <= x < V else 0.0
    path, margin = [0], 1.0
    while True:
        node = path[-1]
        rest, nxt, left, gone = p[node].copy(), -1, 1.0, set()
        for t in range(node + 1, T):
            if parent[t] != node or nxt >= 0:
                continue
            x = int(tokens[t])
            if draft is not None:
                q = widen(draft[node])
                need = u[t] * q[x] if 0 <= x < V else np.inf
                if need < prob[t]:
                    nxt = t
                else:
                    rest = np.maximum(p[node] - q, 0.0)
            else:
                if x in gone:
                    continue
                need = u[t] * left
                if need < prob[t]:
                    nxt = t
                else:
                    left -= prob[t]
                    gone.add(x)
                    if 0 <= x < V:
                        rest[x] = 0.0
            big = max(need, prob[t])
            if 0 < big < np.inf:
                margin = min(margin, abs(need - prob[t]) / big)
        if nxt < 0:
            break
        path.append(nxt)
    node = path[-1]
    if not np.sum(rest) > 0:
        rest = p[node]
    bonus, bm = draw(rest, u[0]) if np.sum(rest) > 0 else (0, 1.0)
    full = np.full(T, -1, dtype=np.int32)
    full[:len(path)] = path
    return SampleResult(node, len(path) - 1, full, bonus, prob, margin, bm)
