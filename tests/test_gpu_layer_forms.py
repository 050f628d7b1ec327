"""Forms of the norm and of the few-token products that no other test runs: every output
format at every number of waves and chunks a row, bf16 outputs of many rows of weights."""
import numpy as np
import pytest
import torch

from gpu_util import dev, host, say
from microscaling_block_scaled_amd.synth import bf16_bits, bf16_to_f32
from test_gpu_gemv_long import weights
from test_gpu_norm import EPS, pitch_of, round_to, to_dev, values

pytestmark = pytest.mark.gpu


# 1, 2, 4, 8 waves of one chunk a lane, 8 of two and of four, two passes
@pytest.mark.parametrize("cols", [500, 1000, 2001, 4090, 8001, 16380, 16400])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_norm_formats(oracle, cols, kind):
    from microscaling_block_scaled_amd import mx
    rng = np.random.default_rng(cols)
    rows = 3
    x, r, w = values(rng, (rows, cols), kind), values(rng, (rows, cols), kind, 3.0), values(rng, (cols,), kind)
    h = round_to(x + r, kind)
    tx, tr = (to_dev(a, kind, pitch_of(cols, kind)) for a in (x, r))
    tw = dev(bf16_bits(w) if kind == "bf16" else w)
    for fmt in range(6):
        say("norm", cols, kind, fmt)
        got = mx.rmsnorm_quantize(tx, tw, fmt, EPS, residual=tr, want_y=True)
        y = (h * host(got["rstd"])[:, None]) * w
        assert np.array_equal(host(got["h"].float()), h) and np.array_equal(host(got["y"].float()), round_to(y, kind))
        q = oracle.quantize(y, fmt, oracle.LAYOUT_ROW)
        assert np.array_equal(host(got["q_row"]), q["q_row"]) and np.array_equal(host(got["s_row"]), q["s_row"]), fmt


@pytest.mark.parametrize("M", [1, 2, 3, 8, 13, 32])
def test_bf16_products_of_many_rows(M):
    from microscaling_block_scaled_amd import mx
    N, K = 8203, 520
    q, s, w = weights(N, K, M)
    x = torch.randn((M, K), device="cuda").to(torch.bfloat16)
    say("gemv bf16", M, N, K)
    y = mx.gemv_bf16(x, q, s, mx.E2M1, M, N, K).double()
    w = w.t().contiguous()
    c, t = x.double() @ w, x.double().abs() @ w.abs()
    tol = 1e-5 * t + 2.0 ** -126
    assert ((y - c).abs() <= tol + 2.0 ** -8 * (c.abs() + tol)).all()
