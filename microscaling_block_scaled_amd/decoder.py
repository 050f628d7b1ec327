"""A decoder layer over MX weights and an 8-bit MX key/value cache, built from the
calls of ``mx``: one ``step`` for prompts and for single new tokens.

    h = x + residual;  n = norm(h)                      rmsnorm_quantize
    q, k, v = n Wqkv^T                                  gemv_bf16 / gemm_bf16
    k, v -> cache                                       cache_write
    a = attention(q, cache)                             attention
    x = a Wo^T                                          gemv_bf16 / gemm_bf16
    h = x + h;  n = norm(h)                             rmsnorm_quantize
    x = (silu(n Wg^T) * (n Wu^T)) Wd^T                  gemv_bf16 / gemm_bf16

Weights are MXFP4 (E2M1).  Up to GEMV_TOKENS tokens take the products that read the
weights once with bf16 activations; more take the MX GEMM, whose A operand the norm
has written in MXFP8 (E4M3) already.  A position enters through the cache's order
alone (no rotary embedding).  Everything here is call order; the gating between
the two halves of the MLP is torch's."""
from dataclasses import dataclass

import torch

from . import mx

GEMV_TOKENS = 32   # tokens up to which the weights' reading is the work
ACT = mx.E4M3      # format of the GEMM's activations and of the cache


@dataclass
class Weight:
    """A weight [n, k] in row-wise MXFP4."""
    q: torch.Tensor
    s: torch.Tensor
    n: int
    k: int


@dataclass
class Layer:
    heads_q: int
    heads: int          # key/value heads
    dim: int
    norm1: torch.Tensor  # bf16 [hidden]
    wqkv: Weight        # [(heads_q + 2 heads) dim, hidden]
    wo: Weight          # [hidden, heads_q dim]
    norm2: torch.Tensor
    wgu: Weight         # gate and up: [2 inter, hidden]
    wd: Weight          # [hidden, inter]


def pack(w: torch.Tensor) -> Weight:
    """A bf16 or fp32 weight [n, k] in MXFP4."""
    o = mx.quantize(w, mx.E2M1, mx.LAYOUT_ROW, mx.RNE)
    return Weight(o["q_row"], o["s_row"], w.shape[0], w.shape[1])


def random_layer(hidden: int, heads_q: int, heads: int, dim: int, inter: int, seed: int = 0) -> Layer:
    """A layer of N(0, 1 / k) weights."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def weight(n, k):
        return pack((torch.randn((n, k), device="cuda", generator=g) * k ** -0.5).to(torch.bfloat16))

    def norm():
        return (1 + 0.1 * torch.randn(hidden, device="cuda", generator=g)).to(torch.bfloat16)

    return Layer(heads_q, heads, dim, norm(), weight((heads_q + 2 * heads) * dim, hidden),
                 weight(hidden, heads_q * dim), norm(), weight(2 * inter, hidden), weight(hidden, inter))


def product(x: torch.Tensor, w: Weight, qx: dict | None = None) -> torch.Tensor:
    """x W^T in bf16 for x [tokens, k]; ``qx``: x's row blocks where its producer
    has written them."""
    T = x.shape[0]
    if T <= GEMV_TOKENS:
        return mx.gemv_bf16(x, w.q, w.s, mx.E2M1, T, w.n, w.k)
    if qx is None:
        qx = mx.quantize(x, ACT, mx.LAYOUT_ROW, mx.RNE)
    return mx.gemm_bf16(qx["q_row"], qx["s_row"], ACT, w.q, w.s, mx.E2M1, T, w.n, w.k)


def step(layer: Layer, x: torch.Tensor, residual: torch.Tensor | None, cache: dict, table: torch.Tensor,
         lens: torch.Tensor, slots: torch.Tensor, eps: float = 1e-5):
    """The layer on Lq new tokens of each of B requests: x, residual bf16 [B * Lq,
    hidden] (residual None: x is the stream itself); lens [B] int32 counts the
    new tokens, slots [B * Lq] int64 are their places in the cache (slot = page *
    page size + place).  Returns (x, residual) for the next layer."""
    T, B = x.shape[0], lens.shape[0]
    hq, hk, d = layer.heads_q, layer.heads, layer.dim
    n = mx.rmsnorm_quantize(x, layer.norm1, ACT, eps, residual=residual, want_y=True)
    h = n.get("h", x)
    qkv = product(n["y"], layer.wqkv, n).view(T, hq + 2 * hk, d)
    mx.cache_write(qkv[:, hq:hq + hk], qkv[:, hq + hk:], slots, cache, ACT)
    a = mx.attention(qkv[:, :hq].unflatten(0, (B, T // max(B, 1))), cache, ACT, table, lens)
    x = product(a["o"].view(T, hq * d), layer.wo)
    n = mx.rmsnorm_quantize(x, layer.norm2, ACT, eps, residual=h, want_y=True)
    gate, up = product(n["y"], layer.wgu, n).chunk(2, dim=1)
    return product(torch.nn.functional.silu(gate) * up, layer.wd), n["h"]
