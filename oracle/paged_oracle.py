"""CPU oracle for the caches in pages: page-table calls on plain Python lists, quantisation in float64.

TEST INFRASTRUCTURE ONLY; shares no code with the CUDA path.
"""

from __future__ import annotations

import math
from typing import List

import numpy as np

E4M3_MAX = 448.0


class NoPages(Exception):
    pass


def _take_lowest(refs: List[int], n: int) -> List[int]:
    free = [p for p, r in enumerate(refs) if r == 0]
    if len(free) < n:
        raise NoPages
    return free[:n]


def reserve(table: List[List[int]], refs: List[int], page: int, entries: List[int]) -> None:
    places = [(r, lp) for r, e in enumerate(entries) for lp in range(-(-e // page)) if table[r][lp] < 0]
    for (r, lp), p in zip(places, _take_lowest(refs, len(places))):
        table[r][lp] = p
        refs[p] = 1


def fork(table: List[List[int]], refs: List[int], page: int, parent: List[int], entries: List[int]) -> List[tuple]:
    """The pages copied: [(from, to)] in slot order."""
    n = len(parent)
    new, partly, copies = [], [], []
    count = [0] * len(refs)
    for row in table:
        for p in row:
            if p >= 0:
                count[p] += 1
    outside = [r - c for r, c in zip(refs, count)]
    for r in range(n):
        s = parent[r]
        if s == r:
            new.append(list(table[r]))
            continue
        row = [-1] * len(table[r])
        if s >= 0:
            need = -(-entries[s] // page)
            row[:need] = table[s][:need]
            if entries[s] % page and row[need - 1] >= 0:
                partly.append((r, need - 1, row[need - 1]))
                row[need - 1] = -2
        new.append(row)
    after = list(outside)
    for row in new:
        for p in row:
            if p >= 0:
                after[p] += 1
    for r, lp, p in partly:
        if after[p] == 0:  # nobody else has it: the lowest slot keeps it
            new[r][lp] = p
            after[p] = 1
        else:
            copies.append((r, lp, p))
    dst = _take_lowest(after, len(copies))
    for (r, lp, src), p in zip(copies, dst):
        new[r][lp] = p
        after[p] = 1
    for r in range(n):
        table[r][:] = new[r]
    refs[:] = after
    return [(src, p) for (_, _, src), p in zip(copies, dst)]


def compact(table: List[List[int]], refs: List[int]):
    """([(from, to)], map, live)."""
    live = sum(1 for r in refs if r > 0)
    holes = [p for p in range(live) if refs[p] == 0]
    high = [p for p in range(live, len(refs)) if refs[p] > 0]
    where = [p if refs[p] > 0 else -1 for p in range(len(refs))]
    for a, b in zip(high, holes):
        where[a] = b
        refs[b], refs[a] = refs[a], 0
    for row in table:
        row[:] = [where[p] if p >= 0 else p for p in row]
    return list(zip(high, holes)), where, live


# The 127 finite magnitudes of e4m3 (code -> value), from the format: 4 exponent bits (bias 7), 3 of mantissa.
CODES = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)])


def e4m3(x: np.ndarray) -> np.ndarray:
    """The nearest e4m3 value (ties to the even code), |x| <= 448."""
    a = np.abs(x)
    hi = np.clip(np.searchsorted(CODES, a), 1, 126)
    lo = hi - 1
    mid = (CODES[lo] + CODES[hi]) / 2
    up = (a > mid) | ((a == mid) & (hi % 2 == 0))
    return np.copysign(np.where(up, CODES[hi], CODES[lo]), x)


def block_scale(amax: float) -> float:
    k = -100
    while 448.0 * math.ldexp(1.0, k) < amax:
        k += 1
    return math.ldexp(1.0, k)


def append(codes: np.ndarray, scales: np.ndarray, table, page: int, block: int, e0: int, e1: int, rows: np.ndarray) -> None:
    """Entries [e0, e1) of one request (table: its row) from rows[g] into codes [num_pages, page, d] (e4m3 values) and
    scales [num_pages, page // block], in float64."""
    for first in range(e0 // block * block, e1, block):
        new = [e for e in range(first, first + block) if e0 <= e < e1]
        old = [e for e in range(first, first + block) if e < e0]
        if not new:
            continue
        at = lambda e: (table[e // page], e % page)  # noqa: E731
        blk = (table[first // page], first % page // block)
        s = block_scale(max(np.max(np.abs(rows[e])) for e in new))
        if old:
            s = max(s, scales[blk])
            for e in old:
                codes[at(e)] = e4m3(codes[at(e)] * scales[blk] / s)
        scales[blk] = s
        for e in new:
            codes[at(e)] = e4m3(rows[e] / s)
