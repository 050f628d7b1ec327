"""Error bounds of the layer operators that hold for any order of their sums.

u is fp32's unit roundoff.  A sum of n terms in any order is off by at most n * 2 u *
sum|terms| to first order, where an addition may also cut its result short (2 u) instead
of rounding it (u)."""
import numpy as np

U = 2.0 ** -24


def half_step_bf16(x):
    """Half the distance between bf16 values (8 significant bits) at |x|."""
    e = np.frexp(np.maximum(np.abs(x), 2.0 ** -126))[1] - 1
    return np.ldexp(1.0, e - 8)


def attention(q, k, v, limits, scale):
    """(o, lse, bound of o's error before its rounding, bound of lse's) in 64 bits, for queries
    q [n, dim], the row i of which sees the first limits[i] of the keys k [tokens, dim].

    Scores: products of bf16 values are exact in fp32; dim of them are summed, and the
    scaling rounds twice.  A weight takes the error of its score and of the score that
    it is taken from, and less than 2^-20 from the exponential and its argument.  For
    the product with v it is two terms of 8 bits, the first cut (less than 2^-7 is left),
    the second rounded (2^-8 of that): 2^-15, and 2^-20 by which the second is raised.
    2 e terms are summed then, and their sums joined with factors of 2 roundings each."""
    n, dim = q.shape
    o, lse = np.zeros((n, v.shape[1])), np.full(n, -np.inf)
    bo, bl = np.zeros_like(o), np.zeros(n)
    for i in range(n):
        e = int(min(max(limits[i], 0), k.shape[0]))
        if e == 0:
            continue
        a = scale * (k[:e] @ q[i])
        ds = 2 * U * (dim + 4) * abs(scale) * (np.abs(k[:e]) @ np.abs(q[i])) + 4 * U * np.abs(a)
        m = a.max()
        p = np.exp(a - m)
        l = p.sum()
        rel = 2 * ds.max() + 2.0 ** -20 + 2 * U * (2 * e + 64)
        o[i] = (p @ v[:e]) / l
        lse[i] = m + np.log(l)
        bo[i] = (2 * rel + 2.0 ** -15 + 2.0 ** -20) * (p @ np.abs(v[:e])) / l
        bl[i] = rel + 4 * U * (abs(m) + abs(np.log(l)) + 1)
    return o, lse, bo, bl
