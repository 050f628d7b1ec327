"""Edges of the layer operators on the GPU: rows without columns, a layer without tokens."""
import pytest
import torch

from gpu_util import Guarded, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [1, 9, 1030])
def test_norm_of_rows_without_columns(rows, kind):
    """The mean of nothing is 0 / 0: rstd is NaN, and written."""
    from microscaling_block_scaled_amd import mx
    e = lambda *s: torch.empty(s, dtype=kind, device="cuda")
    rstd = Guarded((rows,), torch.float32)
    rstd.t.fill_(2.5)
    say("norm of no columns", rows, kind)
    o = mx.rmsnorm_quantize(e(rows, 0), e(0), mx.E4M3, residual=e(rows, 0), want_y=True, out={"rstd": rstd.t})
    torch.cuda.synchronize()
    rstd.check("rstd")
    assert torch.isnan(rstd.t).all()
    assert o["q_row"].shape == (rows, 0) and o["s_row"].shape == (rows, 0) and o["y"].shape == o["h"].shape == (rows, 0)


@pytest.mark.parametrize("B", [0, 2])
def test_decoder_step_without_tokens(B):
    """No request, and requests without new tokens."""
    from microscaling_block_scaled_amd import decoder, mx
    layer = decoder.random_layer(64, 2, 1, 64, 64)
    z = lambda *s, t=torch.int32: torch.zeros(s, dtype=t, device="cuda")
    say("decoder step without tokens", B)
    x, h = decoder.step(layer, z(0, 64, t=torch.bfloat16), z(0, 64, t=torch.bfloat16), mx.kv_cache(2, 1, 16, 64), z(B, 1),
                        z(B), z(0, t=torch.int64))
    assert x.shape == h.shape == (0, 64)
