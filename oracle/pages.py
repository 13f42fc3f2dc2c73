"""Page lists of the paged cache: the oracle (test infrastructure only).

A request's table grows from a stack of free pages before its new positions are
computed and shrinks back into it when they are rejected or the request ends
(openinfer PR #626, What Changed: the hybrid state includes the attention
layers' cache). One request after the other, one entry after the other.

Pins (tests/test_oracle_pages.py): hand-worked lists; what was reserved and is
released restores the list; no page is ever in two places.
"""
from __future__ import annotations

import numpy as np


def reserve(seq_len, n_new, table, held, free, n_free: int, page_size: int, n_pos: int, prefix=(), n_pages=None,
            clip=False, skip=None):
    """In place; returns (n_free, slot map [R, n_pos], requests that were refused or got nothing)."""
    R, P = table.shape
    if clip:
        n_new = [min(int(m), max(0, P * page_size - int(n))) if n >= 0 and 0 <= m <= n_pos else m
                 for n, m in zip(seq_len, n_new)]
    n_pages = len(free) if n_pages is None else n_pages
    have0, needs, ok = [], [], []
    for r in range(R):
        want = -(-(int(seq_len[r]) + int(n_new[r])) // page_size)
        good = seq_len[r] >= 0 and 0 <= n_new[r] <= n_pos and want <= P and 0 <= held[r] <= P
        good = good and (skip is None or not skip[r])
        have = max(int(held[r]), len(prefix))
        have0.append(have)
        needs.append(max(0, want - have) if good else 0)
        ok.append(good)
    left, gets, missed = n_free, [], 0
    for r in range(R):
        left -= needs[r]
        served = needs[r] == 0 or left >= 0
        gets.append(needs[r] if served else 0)
        missed += (skip is None or not skip[r]) and (not ok[r] or not served)
    at = n_free - sum(gets)
    n_free = at
    slots = np.full((R, n_pos), -1, dtype=np.int64)
    for r in range(R):
        if not ok[r]:
            continue
        for e in range(int(held[r]), len(prefix)):
            table[r, e] = prefix[e]
        for i in range(gets[r]):
            table[r, have0[r] + i] = free[at]
            at += 1
        held[r] = have0[r] + gets[r]
        for t in range(int(n_new[r])):
            j = int(seq_len[r]) + t
            e = j // page_size
            if e < held[r] and 0 <= table[r, e] < n_pages:
                slots[r, t] = int(table[r, e]) * page_size + j % page_size
    return n_free, slots, missed


def release(keep_len, table, held, free, n_free: int, page_size: int, n_prefix: int = 0):
    """In place; returns (n_free, refused requests)."""
    R, P = table.shape
    bad = 0
    for r in range(R):
        if keep_len[r] < 0 or not 0 <= held[r] <= P:
            bad += 1
            continue
        keep = max(-(-int(keep_len[r]) // page_size), n_prefix)
        for e in range(keep, int(held[r])):
            page = int(table[r, e])
            if 0 <= page < len(free) and n_free < len(free):
                free[n_free] = page
                n_free += 1
            table[r, e] = -1
        held[r] = min(int(held[r]), keep)
    return n_free, bad
