"""Few-token products with 4-bit MX weights on the GPU, against the 64-bit product of
the oracle's dequantized weights at the GEMM's bound (1e-5 of the sum of the
products' sizes, half a bf16 step more for bf16 outputs)."""
import numpy as np
import pytest
import torch

from gpu_util import Guarded, dev, gemm_tolerance, host, say
from microscaling_block_scaled_amd.synth import bf16_bits, bf16_to_f32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    from microscaling_block_scaled_amd import mx as m
    return m


def packed(oracle, rng, N, K, spread=0):
    w = rng.standard_normal((N, K)) * 0.02
    if spread:
        w *= np.exp2(rng.integers(-spread, spread + 1, (N, K)))
    o = oracle.quantize(w.astype(np.float32), oracle.E2M1, oracle.LAYOUT_ROW)
    return o["q_row"], o["s_row"]


def dequantized(oracle, q, s, N, K):
    return oracle.dequantize(q, s, oracle.E2M1, N, K).astype(np.float64)


def check(y, x, w, what):
    c, t = x @ w.T, np.abs(x) @ np.abs(w).T
    tol = gemm_tolerance(t)
    if y.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(c) + tol) + 2.0 ** -134
    err = np.abs(host(y.float()).astype(np.float64) - c)
    assert (err <= tol).all(), f"{what}: {(err > tol).sum()} outside, worst {(err / tol).max()}"


# tokens around each workgroup shape; rows off 16 and 64; K off 32, 256 and 8
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9, 16, 17, 32, 33, 70])
@pytest.mark.parametrize("N,K", [(1, 1), (16, 32), (17, 31), (40, 256), (65, 300), (100, 1111), (48, 4100)])
def test_product(mx, oracle, M, N, K):
    rng = np.random.default_rng(M * 1000003 + N * 1009 + K)
    q, s = packed(oracle, rng, N, K, spread=3)
    x = bf16_to_f32(bf16_bits(rng.standard_normal((M, K)).astype(np.float32)))
    w = dequantized(oracle, q, s, N, K)
    xd, qd, sd = dev(bf16_bits(x)), dev(q), dev(s)
    say("gemv", M, N, K)
    for call, kind in ((mx.gemv, torch.float32), (mx.gemv_bf16, torch.bfloat16)):
        y = Guarded((M, N), kind)
        call(xd, qd, sd, mx.E2M1, M, N, K, y=y.t)
        torch.cuda.synchronize()
        y.check("y")
        check(y.t, x.astype(np.float64), w, f"{M} x {N} x {K}")


# more row groups than two for each CU: the other workgroup shapes
@pytest.mark.parametrize("M", [1, 2, 4, 7, 16, 21])
def test_many_rows(mx, oracle, M):
    rng = np.random.default_rng(M)
    N, K = 8195, 600
    q, s = packed(oracle, rng, N, K)
    x = bf16_to_f32(bf16_bits(rng.standard_normal((M, K)).astype(np.float32)))
    say("gemv many rows", M)
    y = mx.gemv(dev(bf16_bits(x)), dev(q), dev(s), mx.E2M1, M, N, K)
    check(y, x.astype(np.float64), dequantized(oracle, q, s, N, K), "many rows")


def test_strides_and_alignment(mx, oracle):
    """x as a slice that starts on 2 bytes, in rows of any length; y in wider rows."""
    rng = np.random.default_rng(3)
    M, N, K = 3, 50, 333
    q, s = packed(oracle, rng, N, K)
    x = bf16_to_f32(bf16_bits(rng.standard_normal((M, K)).astype(np.float32)))
    big = torch.full((M, 2 * K + 5), float("nan"), dtype=torch.bfloat16, device="cuda")
    big[:, 3:3 + K] = dev(bf16_bits(x))
    out = torch.full((M, N + 7), 2.5, device="cuda")
    say("gemv strides")
    mx.gemv(big[:, 3:3 + K], dev(q), dev(s), mx.E2M1, M, N, K, y=out[:, 2:2 + N])
    check(out[:, 2:2 + N], x.astype(np.float64), dequantized(oracle, q, s, N, K), "strides")
    assert (out[:, :2] == 2.5).all() and (out[:, 2 + N:] == 2.5).all()


def test_scales_over_their_range(mx, oracle):
    """Scale codes 1 .. 250 against tokens of the opposite size; every element code."""
    N, K = 250, 64
    codes = np.arange(N * K, dtype=np.int64).reshape(N, K) % 16
    q = (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
    s = np.repeat(np.arange(1, N + 1, dtype=np.uint8)[:, None], 2, axis=1)
    rng = np.random.default_rng(4)
    x = bf16_to_f32(bf16_bits((rng.standard_normal((2, K)) * np.array([[2.0 ** 30], [2.0 ** -30]])).astype(np.float32)))
    say("gemv scales")
    y = host(mx.gemv(dev(bf16_bits(x)), dev(q), dev(s), mx.E2M1, 2, N, K)).astype(np.float64)
    w = dequantized(oracle, q, s, N, K)
    c, t = x.astype(np.float64) @ w.T, np.abs(x).astype(np.float64) @ np.abs(w).T
    fits = t < 2.0 ** 127
    assert fits.sum() > 2 * N - 60
    assert (np.abs(y - c)[fits] <= gemm_tolerance(t)[fits]).all()


def test_not_finite_stays_in_its_place(mx, oracle):
    """A NaN scale reaches its row alone, a NaN or Inf token its own outputs alone."""
    rng = np.random.default_rng(6)
    M, N, K = 5, 40, 512
    q, s = packed(oracle, rng, N, K)
    x = bf16_to_f32(bf16_bits(rng.standard_normal((M, K)).astype(np.float32)))
    s2, x2 = s.copy(), x.copy()
    s2[7, 3] = 0xFF
    x2[2, 100], x2[3, 9] = np.nan, np.inf
    say("gemv NaN")
    y = host(mx.gemv(dev(bf16_bits(x2)), dev(q), dev(s2), mx.E2M1, M, N, K))
    clean = host(mx.gemv(dev(bf16_bits(x)), dev(q), dev(s), mx.E2M1, M, N, K))
    assert np.isnan(y[:, 7]).all() and np.isnan(y[2]).all() and not np.isfinite(y[3]).any()
    rest = np.ones((M, N), bool)
    rest[:, 7] = rest[2] = rest[3] = False
    assert np.array_equal(y[rest], clean[rest])


def test_past_4_gib(mx, oracle):
    """Weights past 32-bit offsets: 1.3 M rows of K = 7168 (4.6 GB), the last ones set."""
    rng = np.random.default_rng(7)
    N, K, last = 1300000, 7168, 20
    q, s = packed(oracle, rng, last, K)
    qd = torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda")
    sd = torch.full((N, K // 32), 127, dtype=torch.uint8, device="cuda")
    qd[-last:], sd[-last:] = dev(q), dev(s)
    x = bf16_to_f32(bf16_bits(rng.standard_normal((2, K)).astype(np.float32)))
    say("gemv past 4 GiB")
    y = mx.gemv(dev(bf16_bits(x)), qd, sd, mx.E2M1, 2, N, K)
    assert (y[:, :-last] == 0).all()
    check(y[:, -last:], x.astype(np.float64), dequantized(oracle, q, s, last, K), "past 4 GiB")


def test_empty_and_refusals(mx):
    e = lambda *s, t=torch.uint8: torch.zeros(s, dtype=t, device="cuda")
    bf = torch.bfloat16
    assert mx.gemv(e(0, 64, t=bf), e(8, 32), e(8, 2), mx.E2M1, 0, 8, 64).shape == (0, 8)
    y = mx.gemv(e(2, 0, t=bf), e(8, 0), e(8, 0), mx.E2M1, 2, 8, 0, y=torch.ones((2, 8), device="cuda"))
    assert (y == 0).all()  # a sum of nothing
    x, q, s = e(2, 64, t=bf), e(8, 32), e(8, 2)
    for bad in (dict(x=e(2, 64, t=torch.float32)), dict(x=e(2, 65, t=bf)), dict(q=e(8, 33)), dict(s=e(8, 3)),
                dict(y=e(2, 8, t=bf)), dict(fmt=11)):
        a = dict(x=x, q=q, s=s, fmt=mx.E2M1, y=None) | bad
        with pytest.raises(ValueError):
            mx.gemv(a["x"], a["q"], a["s"], a["fmt"], 2, 8, 64, y=a["y"])
    with pytest.raises(mx.MXError) as err:
        mx.gemv(x, e(8, 64), s, mx.E4M3, 2, 8, 64)
    assert err.value.status == mx.MX_ERR_UNSUPPORTED
    off = torch.zeros(8 * 32 + 8, dtype=torch.uint8, device="cuda")[8:].view(8, 32)
    with pytest.raises(mx.MXError) as err:
        mx.gemv(x, off, s, mx.E2M1, 2, 8, 64)
    assert err.value.status == mx.MX_ERR_ALIGN
