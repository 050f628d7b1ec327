"""Plain references of the decoder-layer operators in 64 bits (numpy), and the error
bounds of their fp32 evaluation.  No code of the library or of the oracle.

u is fp32's unit roundoff.  A sum of n terms taken in chains of at most `depth`
additions is off by at most depth * u * sum|terms| (to first order)."""
import numpy as np

U = 2.0 ** -24
HALF_BF16 = 2.0 ** -8   # half a step of bf16 (8 significant bits), relative


def f64_of_bf16(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def norm_depth(cols):
    """Additions in a row's chain: a lane's own elements (512 lanes at most share a
    row of more than 2048), then lanes and waves."""
    return 8 * -(-cols // 4096) + 24


def norm(h, w, eps):
    """(rstd, y) of rows h [rows, cols]."""
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return rstd, h * rstd[:, None] * w


def norm_loss(x, r, w, eps, c, d):
    """A scalar of the norm's outputs: sum(c * y) + sum(d * h)."""
    h = x + r
    return (c * norm(h, w, eps)[1]).sum() + (d * h).sum()


def norm_grad(dy, h, w, rstd, dh):
    """(dx, dw) by the formula, and bounds of their error in fp32 before the output's
    rounding."""
    n = h.shape[1]
    xhat = h * rstd[:, None]
    g = dy * w
    mean = (g * xhat).mean(1, keepdims=True)
    dx = rstd[:, None] * (g - xhat * mean) + dh
    dw = (dy * xhat).sum(0)
    # mean: its terms carry 3 roundings, its sum `depth`, the division 2
    dmean = (norm_depth(n) + 5) * U * np.abs(g * xhat).mean(1, keepdims=True)
    r = np.abs(rstd)[:, None]
    bx = r * (np.abs(xhat) * dmean + 6 * U * (np.abs(g) + np.abs(xhat * mean))) + 2 * U * np.abs(dx) + 2 * U * np.abs(dh)
    # rows of a column: at most ceil(rows / 256) in a workgroup's chain, 8 groups, then the partial sums
    depth = -(-h.shape[0] // 256) + 8 + 32 + 16
    bw = (depth + 3) * U * np.abs(dy * xhat).sum(0)
    return dx, dw, bx, bw


def e8m0(codes):
    return np.ldexp(1.0, np.asarray(codes, np.int64) - 127)


def attention(q, k, v, limits, scale):
    """(o, lse, bound of o's error, bound of lse's) for queries q [n, dim], the row i
    of which sees the first limits[i] of the keys k [tokens, dim].

    Scores: products of bf16 values are exact in fp32, a chain of dim + 8 additions,
    two roundings of the scaling.  p: the score's error enters as a relative one, the
    exponential and its argument's rounding add less than 2^-20; it is then rounded
    to bf16 for the product with v.  Sums over tokens: four waves at least share them,
    32 at a time, so a chain is at most tokens / 128 + 64 additions."""
    n, dim = q.shape
    o, lse = np.zeros((n, v.shape[1])), np.full(n, -np.inf)
    bo, bl = np.zeros_like(o), np.zeros(n)
    for i in range(n):
        e = int(min(max(limits[i], 0), k.shape[0]))
        if e == 0:
            continue
        a = scale * (k[:e] @ q[i])
        ds = (dim + 8 + 4) * U * abs(scale) * (np.abs(k[:e]) @ np.abs(q[i])) + 4 * U * np.abs(a)
        m = a.max()
        p = np.exp(a - m)
        l = p.sum()
        chain = (e / 128 + 64) * U
        rel = 2 * ds.max() + 2.0 ** -20 + chain
        o[i] = (p @ v[:e]) / l
        lse[i] = m + np.log(l)
        bo[i] = (HALF_BF16 + 2 * rel) * (p @ np.abs(v[:e])) / l
        bl[i] = rel + 4 * U * (abs(m) + abs(np.log(l)) + 1)
    return o, lse, bo, bl
