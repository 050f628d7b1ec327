"""The layer operators together: the decoder example run token by token, by a prompt
in one piece and in both ways, and a normed linear layer's training step."""
import numpy as np
import pytest
import torch

import layer_ref as ref
from gpu_util import dev, host, say
from test_gpu_linear import bf16_close, oracle_step
from microscaling_block_scaled_amd.synth import bf16_bits, bf16_to_f32

pytestmark = pytest.mark.gpu


def plain_step(layer, x, residual, weights, eps=1e-5):
    """The layer on one request's whole prompt in fp32 torch, without any MX rounding
    of activations (weights as stored)."""
    def norm(h, w):
        return h * torch.rsqrt(h.square().mean(-1, keepdim=True) + eps) * w.float()
    h = x.float() + (0 if residual is None else residual.float())
    T = h.shape[0]
    qkv = (norm(h, layer.norm1) @ weights["wqkv"].t()).view(T, -1, layer.dim)
    q, k, v = qkv.split((layer.heads_q, layer.heads, layer.heads), dim=1)
    g = layer.heads_q // layer.heads
    k, v = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
    s = torch.matmul(q.transpose(0, 1), k.permute(1, 2, 0).contiguous()) * layer.dim ** -0.5
    s = s.masked_fill(torch.ones(T, T, dtype=torch.bool, device=s.device).triu(1), float("-inf"))
    a = torch.matmul(s.softmax(-1), v.transpose(0, 1).contiguous()).transpose(0, 1).reshape(T, -1)
    x = a @ weights["wo"].t()
    h = x + h
    gate, up = (norm(h, layer.norm2) @ weights["wgu"].t()).chunk(2, dim=1)
    return (torch.nn.functional.silu(gate) * up) @ weights["wd"].t(), h


def test_decoder_layer():
    """A prompt of 40 tokens (GEMM path), then 3 single tokens of two requests, equal
    the plain layer on the whole sequences up to the formats' rounding: an FP8
    activation is off by up to 2^-4 of itself, on average 2 %, and three such products
    and a cache follow each other."""
    from microscaling_block_scaled_amd import decoder, mx
    layer = decoder.random_layer(256, 4, 2, 64, 512)
    weights = {n: mx.dequantize(w.q, w.s, mx.E2M1, w.n, w.k) for n, w in
               (("wqkv", layer.wqkv), ("wo", layer.wo), ("wgu", layer.wgu), ("wd", layer.wd))}
    g = torch.Generator(device="cuda").manual_seed(1)
    B, n, more, page = 2, 40, 3, 16
    x = torch.randn((B, n + more, 256), device="cuda", generator=g).to(torch.bfloat16)
    cache = mx.kv_cache(8, 2, page, 64)
    table = torch.tensor([[5, 0, 3], [1, 7, 2]], dtype=torch.int32, device="cuda")

    def slots(t0, t1):
        t = torch.arange(t0, t1, device="cuda")
        return (table[:, t // page].long() * page + t % page).reshape(-1)

    outs, res = [], []
    say("decoder prompt")
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    y, h = decoder.step(layer, x[:, :n].reshape(-1, 256), None, cache, table, lens, slots(0, n))
    outs.append(y.view(B, n, 256)), res.append(h.view(B, n, 256))
    for t in range(n, n + more):
        say("decoder token", t)
        lens = lens + 1
        y, h = decoder.step(layer, x[:, t].contiguous(), None, cache, table, lens, slots(t, t + 1))
        outs.append(y.view(B, 1, 256)), res.append(h.view(B, 1, 256))
    y, h = torch.cat(outs, 1).float(), torch.cat(res, 1).float()
    for b in range(B):
        py, ph = plain_step(layer, x[b], None, weights)
        assert (h[b] - ph).norm() < 0.03 * ph.norm()
        assert (y[b] - py).norm() < 0.1 * py.norm()
    # the tokens one by one from the start: the bf16 products and the same cache
    cache2 = mx.kv_cache(8, 2, page, 64)
    for t in range(n + more):
        lens = torch.full((B,), t + 1, dtype=torch.int32, device="cuda")
        y1, h1 = decoder.step(layer, x[:, t].contiguous(), None, cache2, table, lens, slots(t, t + 1))
    assert (y1.float() - y[:, -1]).norm() < 0.1 * y1.float().norm()
    assert (h1.float() - h[:, -1]).norm() < 0.03 * h1.float().norm()


@pytest.mark.parametrize("fmt,T,H,O", [(4, 288, 160, 96), (0, 512, 512, 512)])
def test_normed_linear_step(oracle, fmt, T, H, O):
    """forward_normed hands the product the very codes that quantizing N gives up to
    N's rounding to bf16; the backward equals the linear layer's followed by the norm's
    formula."""
    from microscaling_block_scaled_amd import linear, mx
    rng = np.random.default_rng(T + fmt)
    x, r = (bf16_to_f32(bf16_bits(rng.standard_normal((T, H)).astype(np.float32))) for _ in range(2))
    w = (rng.standard_normal((O, H)) * 0.02).astype(np.float32)
    wn = (1 + 0.1 * rng.standard_normal(H)).astype(np.float32)
    dy, dh = (bf16_to_f32(bf16_bits((rng.standard_normal(s) * 1e-3).astype(np.float32))) for s in ((T, O), (T, H)))
    rec = linear.Recipe(fmt=fmt, seed=42, hadamard_signs=0x5A5A0F0F)
    b = lambda a: dev(bf16_bits(a))
    say("normed linear", fmt, T, H, O)
    y, h, saved = linear.forward_normed(b(x), b(r), b(wn), b(w), rec)
    dx, dwn, dw = linear.backward_normed(b(dy), b(dh), saved, rec)
    # the forward: the norm's fp32 y quantized, then the oracle's product
    hh = bf16_to_f32(bf16_bits(x + r))
    assert np.array_equal(host(h.float()), hh)
    wn32 = bf16_to_f32(bf16_bits(wn))
    n = (hh * host(saved.rstd)[:, None]) * wn32
    q = oracle.quantize(n, fmt, oracle.LAYOUT_ROW)
    ow = oracle.quantize(bf16_bits(w), fmt, oracle.LAYOUT_ROW)
    c, t = oracle.gemm_f64(q["q_row"], q["s_row"], fmt, ow["q_row"], ow["s_row"], fmt, T, O, H)
    bf16_close(host(y.float()), c, 1e-5 * t + 2.0 ** -126 if fmt == 4 or H >= 512 else None, "forward")
    # the backward: the linear layer's gradient of the bf16 n ...
    n16 = bf16_bits(n)
    step = oracle_step(oracle, fmt, n16, bf16_bits(w), bf16_bits(dy), rec.seed, rec.hadamard_signs)
    cw, tol = step["dw"]
    assert (np.abs(host(dw).astype(np.float64) - cw) <= tol).all()
    # ... whose dX goes through the norm's formula
    lin_dx, _ = linear.backward(b(dy), saved.linear, rec)
    wx, ww, bx, bw = ref.norm_grad(host(lin_dx.float()).astype(np.float64), hh.astype(np.float64),
                                   wn32.astype(np.float64), host(saved.rstd).astype(np.float64), dh.astype(np.float64))
    assert (np.abs(host(dx.float()) - wx) <= bx + ref.HALF_BF16 * (np.abs(wx) + bx) + 2.0 ** -133).all()
    assert (np.abs(host(dwn) - ww) <= bw + 2.0 ** -148).all()


def test_linear_forward_with_given_codes():
    from microscaling_block_scaled_amd import linear, mx
    x, w = torch.randn((96, 160), device="cuda").to(torch.bfloat16), torch.randn((64, 160), device="cuda").to(torch.bfloat16)
    r = linear.Recipe()
    y, _ = linear.forward(x, w, r)
    z, _ = linear.forward(x, w, r, qx=mx.quantize(x, r.fmt))
    assert torch.equal(y, z)
