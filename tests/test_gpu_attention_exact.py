"""Attention against the 64-bit softmax to the rounding of its outputs alone: a bf16
output may be half a step from the 64-bit one, and further by what fp32 sums and weights
of 15 bits leave (layer_bounds).  Every kernel variant: dims, formats and the shapes of
attention_shapes."""
import numpy as np
import pytest
import torch

import layer_bounds as bounds
from attention_shapes import SHAPES, case_of
from gpu_util import Guarded, dev, host, say
from test_gpu_attention import Case

pytestmark = pytest.mark.gpu
PAGE = 16


@pytest.fixture(scope="module")
def mx():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    from microscaling_block_scaled_amd import mx as m
    return m


def reference(c, scale):
    B, Lq, hq, dim = c.q.shape
    o, lse = np.zeros(c.q.shape), np.zeros((B, Lq, hq))
    bo, bl = np.zeros_like(o), np.zeros_like(lse)
    for b in range(B):
        limits = [c.lens[b] - Lq + 1 + i for i in range(Lq)]
        for h in range(hq):
            o[b, :, h], lse[b, :, h], bo[b, :, h], bl[b, :, h] = bounds.attention(
                c.q[b, :, h].astype(np.float64), c.k[b][:, h // c.group], c.v[b][:, h // c.group], limits, scale)
    return o, lse, bo, bl


def outside(got, o, bo):
    g = host(got.float()).astype(np.float64)
    return np.abs(g - o) / (bounds.half_step_bf16(np.abs(o) + bo) + bo + 2.0 ** -120)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("name", SHAPES)
def test_outputs_are_rounded_once(mx, oracle, name, dim, fmt):
    lens, Lq, heads, group, _ = case_of(name, dim)
    c = Case(oracle, np.random.default_rng(len(name) + dim + fmt), lens, Lq, heads, group, dim, PAGE, fmt)
    q = c.device()
    out = {"o": Guarded(q.shape, torch.bfloat16), "lse": Guarded(q.shape[:3], torch.float32)}
    say("attention", name, dim, fmt)
    mx.attention(q, c.dcache, fmt, c.dtable, c.dlens, out={n: g.t for n, g in out.items()})
    torch.cuda.synchronize()
    for n, g in out.items():
        g.check(n)
    o, lse, bo, bl = reference(c, dim ** -0.5)
    far = outside(out["o"].t, o, bo)
    assert (far <= 1).all(), ((far > 1).sum(), far.size, far.max())
    gl, empty = host(out["lse"].t).astype(np.float64), np.isneginf(lse)
    assert np.array_equal(np.isneginf(gl), empty)
    assert (np.abs(gl[~empty] - lse[~empty]) <= bl[~empty]).all()


@pytest.mark.parametrize("name", ["four waves, pieces", "16 rows a wave, pieces", "32 rows a wave, pieces"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_beside_values_that_are_not_finite(mx, oracle, dim, name):
    """A NaN value and an infinite one in the last tokens: the dims beside them, and the
    queries before them, are as exact as without them; an infinite value that is seen is
    infinite in the output, as a positive weight times it."""
    lens, Lq, heads, group, _ = case_of(name, dim)
    fmt = 1
    c = Case(oracle, np.random.default_rng(dim + Lq), lens[:1], Lq, heads, group, dim, PAGE, fmt)
    q = c.device()
    n = lens[0]
    for d, tok, byte in ((5, n - 1, 0x7E), (dim - 9, n - 2, 0x7C), (34, 100, 0xFC)):
        c.dcache["v_q"][c.table[0, tok // PAGE], 0, tok % PAGE, d] = byte
    say("attention beside NaN", name, dim)
    got = mx.attention(q, c.dcache, fmt, c.dtable, c.dlens)
    o, lse, bo, bl = reference(c, dim ** -0.5)
    mine = slice(0, group)  # the rows of the first key/value head
    g = host(got["o"].float())
    assert np.isnan(g[0, -1, mine, 5]).all()
    assert np.isposinf(g[0, Lq - 2:, mine, dim - 9]).all()
    assert np.isneginf(g[0, :, mine, 34]).all()
    seen = np.zeros(o.shape, bool)
    seen[0, -1, mine, 5] = seen[0, Lq - 2:, mine, dim - 9] = seen[0, :, mine, 34] = True
    far = outside(got["o"], o, bo)
    assert (far[~seen] <= 1).all(), far[~seen].max()
    assert (np.abs(host(got["lse"]) - lse) <= bl).all()


def test_infinite_values_of_single_queries(mx, oracle):
    """One query token, for which no step asks whether its values are finite."""
    for dim in (64, 128, 256):
        c = Case(oracle, np.random.default_rng(dim), [90, 40], 1, 1, 4, dim, PAGE, 1)
        q = c.device()
        c.dcache["v_q"][c.table[0, 1], 0, 3, 7], c.dcache["v_q"][c.table[0, 2], 0, 0, 40] = 0x7C, 0xFC
        say("attention infinite values", dim)
        got = mx.attention(q, c.dcache, 1, c.dtable, c.dlens)
        o, lse, bo, _ = reference(c, dim ** -0.5)
        g = host(got["o"].float())
        assert np.isposinf(g[0, ..., 7]).all() and np.isneginf(g[0, ..., 40]).all()
        seen = np.zeros(o.shape, bool)
        seen[0, ..., 7] = seen[0, ..., 40] = True
        assert (outside(got["o"], o, bo)[~seen] <= 1).all()


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_tiny_and_zero_values(mx, oracle, dim):
    """Blocks of zeros (scale code 0) and scales down to code 0: what bf16 cannot hold of
    an element times its scale is less than 2^-133."""
    for Lq in (1, 30):
        c = Case(oracle, np.random.default_rng(dim), [70], Lq, 1, 2, dim, PAGE, 0)
        c.cache["k_q"][c.table[0, 0], 0, 3] = c.cache["v_q"][c.table[0, 0], 0, 3] = 0
        c.cache["k_s"][c.table[0, 0], 0, 3] = c.cache["v_s"][c.table[0, 0], 0, 3] = 0
        c.k[0][3] = c.v[0][3] = 0.0
        for tok in range(16, 32):  # codes 0 .. 15
            at = (c.table[0, 1], 0, tok - 16)
            for name, kv in (("k", c.k[0]), ("v", c.v[0])):
                kv[tok, 0] *= np.repeat(np.exp2(tok - 16.0 - c.cache[name + "_s"][at]), 32)
                c.cache[name + "_s"][at] = tok - 16
        q = c.device()
        say("attention tiny values", dim, Lq)
        got = mx.attention(q, c.dcache, 0, c.dtable, c.dlens)
        o, lse, bo, bl = reference(c, dim ** -0.5)
        assert (outside(got["o"], o, bo) <= 1).all()
        assert (np.abs(host(got["lse"]) - lse) <= bl).all()
