"""Sums over many rows, put together from pieces that the plain 64-bit forms of
tests/_more_layers.py are called on one by one.

The forms bound a column sum over n rows by (n + 64) U times the sum of its terms'
absolute values, as if one thread added them in order; over tens of thousands of rows
that is as large as the sum.  A kernel's terms go through far fewer additions, `depth` of
them: the rows of one thread and the sums of threads, warps and blocks behind them.  A
piece of n rows with the bound e + (n + 64) U m (e: its terms' own errors, m: their
absolute sum) then counts with e + depth U m, which is at most its bound times
max(1, depth / (n + 64)).
"""
from __future__ import annotations

import torch


def tree(rows_of_a_thread):
    """Additions a term goes through: its thread's, then at most 5 of lanes, 8 of warps or
    teams, and of up to 4 blocks on each of 160 multiprocessors 20 of a warp's and 32 of the
    warps; 2 roundings of the term itself."""
    return rows_of_a_thread + 5 + 8 + 20 + 32 + 2


def summed(pieces, depth):
    """(value, bound) of a sum from those of its pieces, [(value, bound, rows)]."""
    value = sum(v for v, _, _ in pieces)
    return value, sum(e * max(1.0, depth / (n + 64)) for _, e, n in pieces)


def told_apart(pieces, depth):
    """The share of pieces of eight rows or more without which a sum would be found wrong in
    one entry at least: by twice the bound, since what is compared may be off by it too."""
    _, bound = summed(pieces, depth)
    seen = [bool((v.abs() > 2 * bound).any()) for v, _, n in pieces if n >= 8]
    return sum(seen) / len(seen)
