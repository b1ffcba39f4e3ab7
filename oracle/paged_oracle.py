"""Paged caches: plain fp64 / integer CPU oracle.

TEST INFRASTRUCTURE, like the rest of ``oracle/``: only ``tests/`` may import
it; the CUDA library shares nothing with it.

* ``attention``: one query per (layer, sequence, query head) over the first
  len rows of the sequence's pages (the decode oracle's formula; an empty
  sequence gives 0 and -inf), with bounds on what 32-bit arithmetic may be off;
* ``append``: norm and rotation of new rows;
* ``compact``: the cut of a cache to its kept rows, one (layer, sequence,
  head) at a time;
* ``update``: the page tables of a step, one sequence at a time in Python
  integers.

Parity status: pinned by ``tests/test_oracle_paged.py`` (an identity table
gives the decode oracle's results, rotations as complex products and by their
group law, invariants of the tables against a row-by-row replay).
"""

from __future__ import annotations

import math
from typing import List, Optional, Sequence, Tuple

import numpy as np

U32 = 2.0 ** -24          # half a step of fp32, relative


def rows_of(pool, table_row, n: int):
    """The first n rows of a sequence: pool [pages, page_size, H_kv, D] -> [n, H_kv, D]."""
    ps = pool.shape[1]
    j = np.arange(n)
    return pool[np.asarray(table_row)[j // ps], j % ps]


def attention(q, K, V, table, lens):
    """q [L, S, H, D], K, V [L, pages, ps, H_kv, D] (fp64), table [S, W], lens [S]:
    (out, lse, out_bound, lse_bound).

    Bounds of an fp32 computation: a logit is a sum of D products in any order, off by at most
    d = 2 (D + 4) u sum_i |q_i k_i| / sqrt(D) (the factor 2: an accumulator that truncates);
    weights are then off by 2 d + 2^-16 relative (the exponential's and the weights' own
    rounding included), and the sums over n rows, taken in runs, by another (n / 8 + 64) u."""
    L, S, H, D = q.shape
    G = H // K.shape[3]
    out = np.zeros(q.shape)
    lse = np.full((L, S, H), -np.inf)
    ob, lb = np.zeros(q.shape), np.zeros((L, S, H))
    for l in range(L):
        for b in range(S):
            n = int(lens[b])
            if n == 0:
                continue
            kr, vr = rows_of(K[l], table[b], n), rows_of(V[l], table[b], n)
            for h in range(H):
                k, v, x = kr[:, h // G], vr[:, h // G], q[l, b, h]
                z = k @ x / math.sqrt(D)
                m = z.max()
                p = np.exp(z - m)
                lse[l, b, h] = m + math.log(p.sum())
                p /= p.sum()
                out[l, b, h] = p @ v
                d = (2 * (D + 4) * U32 * (np.abs(k) @ np.abs(x)) / math.sqrt(D)).max()
                sums = (n / 8 + 64) * U32
                ob[l, b, h] = (2 * d + 2.0 ** -16 + sums) * (p @ np.abs(v)) + 1e-30
                lb[l, b, h] = d + 2.0 ** -16 + sums + abs(lse[l, b, h]) * 4 * U32
    return out, lse, ob, lb


def norm(x, weight, eps: float):
    """x [..., D] -> x / sqrt(mean(x^2) + eps) * weight."""
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight


def rotate(x, angles, interleaved: bool, scale: float = 1.0):
    """x [N, heads, D]; angles [N, rot / 2] in fp64."""
    half = angles.shape[1]
    y = np.array(x, np.float64)
    a, b = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved
            else (slice(0, half), slice(half, 2 * half)))
    c, s = scale * np.cos(angles)[:, None], scale * np.sin(angles)[:, None]
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y


def compact(want: Sequence[int], length: int) -> List[int]:
    """The row that each slot 0 .. n-1 holds after the cut to the n rows `want`."""
    n = len(want)
    if len(set(want)) != n or any(j < 0 or j >= length for j in want):
        raise ValueError("kept rows must be distinct and within the sequence")
    there = set(want)
    late = iter([j for j in want if j >= n])
    return [s if s in there else next(late) for s in range(n)]


def update(table, lens, parents: Optional[Sequence[int]], new_lens, num_pages: int, ps: int
           ) -> Tuple[List[List[int]], List[int], int, List[Tuple[int, int, int]]]:
    """(tables, references, free pages, copies (source, target, rows))."""
    width = len(table[0]) if len(table) else 0
    parents = list(range(len(new_lens))) if parents is None else list(parents)
    rows = [0 if p < 0 else min(lens[p], n) for p, n in zip(parents, new_lens)]
    out = [[-1] * width for _ in parents]
    ref = [0] * num_pages
    for b, p in enumerate(parents):
        for i in range(rows[b] // ps):
            out[b][i] = int(table[p][i])
            ref[out[b][i]] += 1
    for b, p in enumerate(parents):
        i = rows[b] // ps
        if rows[b] % ps and ref[table[p][i]] == 0:
            out[b][i] = int(table[p][i])
            ref[out[b][i]] = 1
    free = [x for x in range(num_pages) if ref[x] == 0]
    left, copies = len(free), []
    for b, p in enumerate(parents):
        for i in range(-(-new_lens[b] // ps)):
            if out[b][i] >= 0:
                continue
            left -= 1
            if not free:
                continue
            out[b][i] = free.pop(0)
            ref[out[b][i]] = 1
            if i == rows[b] // ps and rows[b] % ps:
                copies.append((int(table[p][i]), out[b][i], rows[b] % ps))
    return out, ref, left, copies
