"""Few-token products whose waves take more of K than one load of scales serves (2048
elements: K past 16384 by eight waves, past 8192 by four), on the GPU, against the
product in 64 bits at the bound of test_gpu_gemv (1e-5 of the sum of the products'
sizes)."""
import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def weights(N, K, seed):
    """Every element and 16 scales, at random; the padding of a short last block is zeros."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    nb = -(-K // 32)
    codes = torch.randint(0, 16, (N, nb * 32), device="cuda", generator=g, dtype=torch.uint8)
    codes[:, K:] = 0
    s = torch.randint(112, 128, (N, nb), device="cuda", generator=g, dtype=torch.uint8)
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device="cuda")
    w = table[codes.int()] * torch.exp2(s.double() - 127).repeat_interleave(32, 1)
    return codes[:, 0::2] | (codes[:, 1::2] << 4), s, w[:, :K]


# around the ends of 64 blocks of scales a wave: 8 x 2048 and 4 x 2048 elements, twice them,
# and a K whose last block, step and run of 16 scales are short
@pytest.mark.parametrize("N,K", [(40, 16384), (40, 16400), (33, 16500), (40, 18433), (40, 33000), (17, 49153),
                                 (8195, 8192), (8195, 8300), (8195, 10241), (8211, 16500)])
def test_scales_are_loaded_again(N, K):
    from microscaling_block_scaled_amd import mx
    q, s, w = weights(N, K, N + K)
    size = w.abs().t().contiguous()
    w = w.t().contiguous()
    for M in (1, 2, 4, 7, 16, 32):
        g = torch.Generator(device="cuda").manual_seed(M)
        x = torch.randn((M, K), device="cuda", generator=g).to(torch.bfloat16)
        say("gemv", M, N, K)
        y = mx.gemv(x, q, s, mx.E2M1, M, N, K).double()
        c, t = x.double() @ w, x.double().abs() @ size
        bad = (y - c).abs() > 1e-5 * t + 2.0 ** -126
        assert not bad.any(), (M, int(bad.sum()), float(((y - c).abs() / t).max()))
