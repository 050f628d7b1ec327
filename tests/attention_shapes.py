"""Shapes of attention calls by the kernels that they run, and what the workspace says
of it.  Up to 16 rows (query tokens x query heads of a key/value head): eight waves of
one workgroup, or four waves a piece and a join of the pieces by one or four waves a
row.  More rows: 16 of them a wave up to 64 rows and for dim 256, else 32."""
import numpy as np


def lengths(B, seed, *first):
    return list(first) + [int(n) for n in np.random.default_rng(seed).integers(0, 24, B - len(first))]


# name: (lens, Lq, heads, group, whether the tokens are in pieces); not of every dim
SHAPES = {
    "eight waves": ([700, 0, 33], 1, 2, 5, False),
    "four waves, pieces": ([1500, 0, 1, 1030], 3, 2, 2, True),
    "four waves, many rows to join": (lengths(47, 1, 2150, 900), 1, 3, 15, True),
    "16 rows a wave": ([120, 0, 41], 5, 1, 7, False),
    "16 rows a wave, pieces": ([1100, 300], 9, 2, 4, True),
    "32 rows a wave": ([100, 7], 41, 1, 2, False),
    "32 rows a wave, pieces": ([1100, 90, 500], 75, 1, 2, True),
}


def case_of(name, dim):
    lens, Lq, heads, group, pieces = SHAPES[name]
    if dim == 256 and name == "eight waves":  # dim 256 never takes eight: four, in one piece
        lens = [200, 0, 33]
    return lens, Lq, heads, group, pieces
