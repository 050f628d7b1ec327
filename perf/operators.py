"""The decoder-layer operators as a user's program calls them, and their plain forms.

Operators: the root-mean-square norm with the residual's addition and an MX FP8 output, and its
gradient; products of a few tokens with 4-bit MX weights; the paged 8-bit MX key/value cache's write;
and attention over that cache.  ``listed()`` holds the cases that are measured, ``draw()`` gives more of
the same ranges.  ``run()`` computes a case with elementary torch operations in 32 bits, or, where
``own`` is true, with this repository's kernels.

An MX block is 32 consecutive values that share one power of two X (an E8M0 byte, X = 2^(code - 127));
a value is X times its 8- or 4-bit element.  Elements in 8 bits and scales are returned as tensors of
torch's float8 types, that is, as the values that they stand for.
"""
import math

import torch

own = False

BLOCK = 32
FP8 = {"e4m3": (torch.float8_e4m3fn, 8, 448.0), "e5m2": (torch.float8_e5m2, 15, 57344.0)}
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def blocks(n):
    return (n + BLOCK - 1) // BLOCK


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token's hidden state on its way through a layer: latency counts
        {"name": "norm, 1 x 4096", "op": "norm", "rows": 1, "cols": 4096, "type": "bf16",
         "fmt": "e4m3", "residual": True, "y": True},
        # the activations of a prefill or a training batch
        {"name": "norm, 16384 x 4096", "op": "norm", "rows": 16384, "cols": 4096, "type": "bf16",
         "fmt": "e4m3", "residual": True, "y": False},
        # the backward pass of a training batch, with the gradient that comes along the residual
        {"name": "norm gradient, 8192 x 4096", "op": "norm_grad", "rows": 8192, "cols": 4096,
         "type": "bf16", "dh": True},
        # fp32, an odd width in rows that are padded to 16 bytes, a ragged number of rows
        {"name": "norm gradient, 1001 x 2050", "op": "norm_grad", "rows": 1001, "cols": 2050,
         "type": "fp32", "dh": False},
        # one token's attention output projection
        {"name": "4-bit product, 1 x 4096 x 4096", "op": "gemv", "M": 1, "N": 4096, "K": 4096, "out": "bf16"},
        # the up projection of a few requests that are served together
        {"name": "4-bit product, 4 x 14336 x 4096", "op": "gemv", "M": 4, "N": 14336, "K": 4096, "out": "bf16"},
        # the down projection of a larger batch, with the full sums
        {"name": "4-bit product, 16 x 4096 x 14336", "op": "gemv", "M": 16, "N": 4096, "K": 14336, "out": "fp32"},
        # one request early in its answer
        {"name": "attention, 1 request of 1000", "op": "attention", "B": 1, "Lq": 1, "L": 1000, "Hkv": 8,
         "G": 4, "D": 128, "page": 16, "fmt": "e4m3"},
        # a batch of long requests of many lengths
        {"name": "attention, 32 requests to 16384", "op": "attention", "B": 32, "Lq": 1, "L": 16384,
         "Hkv": 8, "G": 4, "D": 128, "page": 64, "fmt": "e4m3"},
        # a piece of each prompt behind what is cached of it already
        {"name": "attention, 4 x 64 tokens to 4096", "op": "attention", "B": 4, "Lq": 64, "L": 4096,
         "Hkv": 8, "G": 4, "D": 128, "page": 32, "fmt": "e4m3"},
        # one new token each for a batch of requests
        {"name": "cache write, 32 tokens", "op": "write", "T": 32, "Hkv": 8, "D": 128, "page": 64,
         "pages": 64, "type": "bf16", "fmt": "e4m3"},
        # the prompt tokens of a prefill
        {"name": "cache write, 8192 tokens", "op": "write", "T": 8192, "Hkv": 8, "D": 128, "page": 64,
         "pages": 256, "type": "bf16", "fmt": "e4m3"},
    ]


def spread(rng, lo, hi):
    """A whole number from lo to hi, uniform over the logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("norm", "norm_grad", "gemv", "gemv", "attention", "attention", "write"))
    if op in ("norm", "norm_grad"):
        cols = spread(rng, 64, 14336)
        if rng.random() < 0.5:
            cols = max(64, cols // 64 * 64)
        rows = spread(rng, 1, max(1, min(16384, (1 << 25) // cols)))
        kind = rng.choice(("bf16", "bf16", "fp32"))
        if op == "norm":
            return {"op": op, "rows": rows, "cols": cols, "type": kind, "fmt": rng.choice(("e4m3", "e5m2")),
                    "residual": rng.random() < 0.7, "y": rng.random() < 0.3}
        return {"op": op, "rows": rows, "cols": cols, "type": kind, "dh": rng.random() < 0.6}
    if op == "gemv":
        n, k = spread(rng, 64, 14336), spread(rng, 64, 14336)
        if rng.random() < 0.7:
            k = max(64, k // 64 * 64)
        return {"op": op, "M": rng.choice((1, 1, 2, 3, 4, 5, 7, 8, 11, 16, 23, 32)), "N": n, "K": k,
                "out": rng.choice(("bf16", "fp32"))}
    heads, dim = rng.choice((1, 2, 4, 5, 8, 16)), rng.choice((64, 128, 128, 256))
    page, fmt = rng.choice((16, 32, 48, 64, 128, 256)), rng.choice(("e4m3", "e4m3", "e5m2"))
    if op == "write":
        t = spread(rng, 1, 16384)
        t = max(1, min(t, (1 << 24) // (heads * dim)))
        return {"op": op, "T": t, "Hkv": heads, "D": dim, "page": page,
                "pages": blocks_of(t, page) + rng.randrange(1, 64), "type": rng.choice(("bf16", "fp32")), "fmt": fmt}
    group = rng.choice((1, 2, 3, 4, 7, 8, 16))
    lq = rng.choice((1, 1, 1, 1, rng.randrange(2, 9), spread(rng, 9, 128)))
    length = spread(rng, 1, 16384)
    requests = spread(rng, 1, 32)
    while requests > 1 and (requests * length * heads * dim > (1 << 28) or
                            requests * lq * heads * group * length > (1 << 26)):
        requests = (requests + 1) // 2
    while lq * heads * group * length > (1 << 26):
        lq = (lq + 1) // 2
    return {"op": op, "B": requests, "Lq": lq, "L": length, "Hkv": heads, "G": group, "D": dim, "page": page,
            "fmt": fmt}


def blocks_of(n, size):
    return (n + size - 1) // size


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def to_fp8(v, fmt):
    """MX elements (their bytes) and scale codes of v [.., n] along its last axis, n a multiple of 32:
    X = 2^(floor(log2 max|v|) - emax), elements v / X rounded to nearest even and saturated."""
    kind, emax, top = FP8[fmt]
    v = v.reshape(*v.shape[:-1], -1, BLOCK)
    v = torch.where(v.abs() < 2.0 ** -126, torch.zeros_like(v), v)
    most = v.abs().amax(-1)
    code = (torch.frexp(most)[1] - 1 - emax + 127).clamp_(0, 254)
    code = torch.where(most > 0, code, 0).to(torch.uint8)
    p = (v / code.view(torch.float8_e8m0fnu).float().unsqueeze(-1)).clamp_(-top, top).to(kind)
    return p.view(torch.uint8).flatten(-2), code


def to_fp4(v):
    """The same for E2M1 (largest exponent 2, largest value 6), two elements a byte, even ones low."""
    v = v.reshape(*v.shape[:-1], -1, BLOCK)
    most = v.abs().amax(-1)
    code = (torch.frexp(most)[1] - 1 - 2 + 127).clamp_(0, 254)
    code = torch.where(most > 0, code, 0).to(torch.uint8)
    p = v / code.view(torch.float8_e8m0fnu).float().unsqueeze(-1)
    a = p.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp_(max=6.0)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=v.device)
    c = torch.bucketize(a, edges).to(torch.uint8) | (torch.signbit(p).to(torch.uint8) << 3)
    c = c.flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), code


def padded_rows(rows, cols, kind, g, std=1.0):
    """[rows, cols] of N(0, std), its rows a multiple of 16 bytes apart."""
    per = 16 // torch.empty((), dtype=kind).element_size()
    full = torch.empty((rows, blocks_of(cols, per) * per), dtype=kind, device="cuda").normal_(0.0, std, generator=g)
    return full[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op in ("norm", "norm_grad"):
        rows, cols, kind = case["rows"], case["cols"], TYPES[case["type"]]
        s["w"] = (1.0 + 0.1 * torch.randn(cols, device="cuda", generator=g)).to(kind)
        x = padded_rows(rows, cols, kind, g)
        if op == "norm":
            s["x"] = x
            s["residual"] = padded_rows(rows, cols, kind, g, 3.0) if case["residual"] else None
        else:
            s["h"] = x
            s["rstd"] = 1.0 / torch.sqrt(x.float().square().sum(-1) / cols + EPS)
            s["dy"] = padded_rows(rows, cols, kind, g, 1e-3)
            s["dh"] = padded_rows(rows, cols, kind, g, 1e-3) if case["dh"] else None
    elif op == "gemv":
        n, k = case["N"], case["K"]
        w = torch.zeros((n, blocks(k) * BLOCK), device="cuda")
        w[:, :k].normal_(0.0, 0.02, generator=g)
        s["w_q"], s["w_s"] = to_fp4(w)
        s["x"] = torch.randn((case["M"], k), device="cuda", generator=g).to(torch.bfloat16)
    elif op == "write":
        t, heads, dim, kind = case["T"], case["Hkv"], case["D"], TYPES[case["type"]]
        # keys and values lie in one tensor, as a joint projection leaves them
        both = torch.randn((t, 2, heads, dim), device="cuda", generator=g).to(kind)
        s["k"], s["v"] = both[:, 0], both[:, 1]
        slots = torch.randperm(case["pages"] * case["page"], device="cuda", generator=g)[:t]
        if t >= 8:
            slots[3::8] = -1  # padding tokens of a batch that was rounded up: not written
        s["slots"] = slots
        s["cache"] = empty_cache(case["pages"], heads, case["page"], dim)
    else:
        b, heads, dim, page, length = case["B"], case["Hkv"], case["D"], case["page"], case["L"]
        per = blocks_of(length, page)
        pages = b * per + 3
        s["cache"] = c = {}
        for name in ("k", "v"):
            v = torch.randn((pages, heads, page, dim), device="cuda", generator=g)
            c[name + "_q"], c[name + "_s"] = to_fp8(v, case["fmt"])
            del v
        s["table"] = torch.randperm(pages, device="cuda", generator=g)[:b * per].reshape(b, per).to(torch.int32)
        lens = torch.randint(max(1, length // 4), length + 1, (b,), device="cuda", generator=g)
        lens[0] = length
        if b >= 4:  # a request that has ended, and one that begins
            lens[1], lens[2] = 0, 1
        s["lens"] = lens.to(torch.int32)
        s["q"] = torch.randn((b, case["Lq"], heads * case["G"], dim), device="cuda", generator=g).to(torch.bfloat16)
    return s


def empty_cache(pages, heads, page, dim):
    z = lambda n: torch.zeros((pages, heads, page, n), dtype=torch.uint8, device="cuda")  # noqa: E731
    return {"k_q": z(dim), "k_s": z(dim // BLOCK), "v_q": z(dim), "v_s": z(dim // BLOCK)}


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def as_values(q, s, fmt):
    """What the bytes q and scale codes s stand for, in fp32."""
    v = q.view(FP8[fmt][0]).float().unflatten(-1, (-1, BLOCK))
    return (v * s.view(torch.float8_e8m0fnu).float().unsqueeze(-1)).flatten(-2)


def plain_norm(s):
    case, x, w = s["case"], s["x"], s["w"].float()
    h = x if s["residual"] is None else (x.float() + s["residual"].float()).to(x.dtype)
    hf = h.float()
    rstd = 1.0 / torch.sqrt(hf.square().sum(-1) / case["cols"] + EPS)
    y = hf * rstd.unsqueeze(-1) * w
    pad = blocks(case["cols"]) * BLOCK - case["cols"]
    q, sc = to_fp8(torch.nn.functional.pad(y, (0, pad)), case["fmt"])
    out = {"q": q.view(FP8[case["fmt"]][0]), "s": sc.view(torch.float8_e8m0fnu), "rstd": rstd}
    if s["residual"] is not None:
        out["h"] = h
    if case["y"]:
        out["y"] = y.to(x.dtype)
    return out


def plain_norm_grad(s):
    h, dy = s["h"].float(), s["dy"].float()
    rstd = s["rstd"].unsqueeze(-1)
    xhat = h * rstd
    g = dy * s["w"].float()
    dx = rstd * (g - xhat * ((g * xhat).sum(-1, keepdim=True) / h.shape[1]))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["h"].dtype), "dw": (dy * xhat).sum(0)}


def plain_gemv(s):
    q, k = s["w_q"], s["case"]["K"]
    values = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=q.device)
    codes = torch.stack((q & 15, q >> 4), -1).flatten(-2).unflatten(-1, (-1, BLOCK))
    w = values[codes.int()] * s["w_s"].view(torch.float8_e8m0fnu).float().unsqueeze(-1)
    y = s["x"].float() @ w.flatten(-2)[:, :k].t()
    return y.to(TYPES[s["case"]["out"]])


def plain_write(s):
    case, c = s["case"], s["cache"]
    keep = s["slots"] >= 0
    slots = s["slots"][keep]
    page, at = slots // case["page"], slots % case["page"]
    kq, ks = to_fp8(s["k"][keep].float(), case["fmt"])
    vq, vs = to_fp8(s["v"][keep].float(), case["fmt"])
    c["k_q"][page, :, at], c["k_s"][page, :, at] = kq, ks
    c["v_q"][page, :, at], c["v_s"][page, :, at] = vq, vs
    return seen(c, case["fmt"])


def seen(c, fmt):
    """A cache as the values that it holds."""
    return {n: t.view(FP8[fmt][0] if n.endswith("q") else torch.float8_e8m0fnu) for n, t in c.items()}


def plain_attention(s):
    case, c, table = s["case"], s["cache"], s["table"].long()
    b, lq, heads, g, dim = case["B"], case["Lq"], case["Hkv"], case["G"], case["D"]
    k = as_values(c["k_q"][table], c["k_s"][table], case["fmt"]).transpose(1, 2).flatten(2, 3)  # [B, Hkv, tokens, D]
    v = as_values(c["v_q"][table], c["v_s"][table], case["fmt"]).transpose(1, 2).flatten(2, 3)
    q = s["q"].float().reshape(b, lq, heads, g, dim).permute(0, 2, 1, 3, 4).flatten(2, 3)     # [B, Hkv, Lq G, D]
    scores = torch.matmul(q, k.transpose(2, 3).contiguous()) * dim ** -0.5
    # query i of a request sees its tokens before len - Lq + i + 1
    limit = s["lens"].view(b, 1) - lq + 1 + torch.arange(lq, device=q.device)
    limit = limit.repeat_interleave(g, 1).view(b, 1, lq * g, 1)
    sees = torch.arange(k.shape[2], device=q.device) < limit
    scores = torch.where(sees, scores, -math.inf)
    most = scores.amax(-1, keepdim=True).clamp_(min=-1e30)
    p = torch.exp(scores - most)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    lse = (most + torch.log(total)).squeeze(-1)
    o = o.unflatten(2, (lq, g)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    return {"o": o.to(torch.bfloat16), "lse": lse.unflatten(2, (lq, g)).permute(0, 2, 1, 3).flatten(2, 3)}


PLAIN = {"norm": plain_norm, "norm_grad": plain_norm_grad, "gemv": plain_gemv, "write": plain_write,
         "attention": plain_attention}


# ---------------------------------------------------------------------------
# the framework's operators
# ---------------------------------------------------------------------------
def own_pass(s):
    from microscaling_block_scaled_amd import mx
    case = s["case"]
    op = case["op"]
    if op == "norm":
        o = mx.rmsnorm_quantize(s["x"], s["w"], mx.FORMATS[case["fmt"]], EPS, residual=s["residual"],
                                want_y=case["y"])
        out = {"q": o["q_row"].view(FP8[case["fmt"]][0]), "s": o["s_row"].view(torch.float8_e8m0fnu),
               "rstd": o["rstd"]}
        if s["residual"] is not None:
            out["h"] = o["h"]
        if case["y"]:
            out["y"] = o["y"]
        return out
    if op == "norm_grad":
        return mx.rmsnorm_backward(s["dy"], s["h"], s["w"], s["rstd"], dh=s["dh"])
    if op == "gemv":
        product = mx.gemv if case["out"] == "fp32" else mx.gemv_bf16
        return product(s["x"], s["w_q"], s["w_s"], mx.E2M1, case["M"], case["N"], case["K"])
    if op == "write":
        mx.cache_write(s["k"], s["v"], s["slots"], s["cache"], mx.FORMATS[case["fmt"]])
        return seen(s["cache"], case["fmt"])
    return mx.attention(s["q"], s["cache"], mx.FORMATS[case["fmt"]], s["table"], s["lens"])


def run(state):
    return own_pass(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        n, size = case["rows"] * case["cols"], TYPES[case["type"]].itemsize
        if op == "norm":
            moved = n * size * (1 + 2 * case["residual"] + case["y"]) + case["cols"] * size + 4 * case["rows"]
            return {"bytes": moved + case["rows"] * blocks(case["cols"]) * (BLOCK + 1), "flops": 6 * n}
        return {"bytes": n * size * (3 + case["dh"]) + case["cols"] * (size + 4) + 4 * case["rows"], "flops": 12 * n}
    if op == "gemv":
        m, n, k = case["M"], case["N"], case["K"]
        return {"bytes": n * blocks(k) * 17 + 2 * m * k + m * n * TYPES[case["out"]].itemsize,
                "flops": 2.0 * m * n * k}
    heads, dim = case["Hkv"], case["D"]
    row = heads * (dim + dim // BLOCK)  # one token's keys or values
    if op == "write":
        size = TYPES[case["type"]].itemsize
        return {"bytes": case["T"] * (2 * heads * dim * size + 2 * row + 8), "flops": 8 * case["T"] * heads * dim}
    b, lq, length = case["B"], case["Lq"], case["L"]
    low = max(1, length // 4)
    tokens = length + (b - 1) * (low + length) / 2 if b < 4 else length + 1 + (b - 3) * (low + length) / 2
    q = b * lq * heads * case["G"]
    return {"bytes": tokens * 2 * row + q * (4 * dim + 4) + 4 * tokens / case["page"],
            "flops": 4.0 * lq * heads * case["G"] * dim * tokens}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def decoded(fmt, device):
    """The values of the 256 bytes of an 8-bit format, or of the 16 codes of E2M1, from their fields."""
    bits, man, bias = {"e4m3": (8, 3, 7), "e5m2": (8, 2, 15), "e2m1": (4, 1, 1)}[fmt]
    values = []
    for c in range(1 << bits):
        e, m = (c >> man) & ((1 << (bits - 1 - man)) - 1), c & ((1 << man) - 1)
        v = m * 2.0 ** (1 - bias - man) if e == 0 else (1 + m / (1 << man)) * 2.0 ** (e - bias)
        values.append(-v if c >> (bits - 1) else v)
    return torch.tensor(values, dtype=torch.float64, device=device)


def power(e):
    """2^e in 64 bits, for whole numbers e."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def powers(code):
    """2^(code - 127) in 64 bits."""
    return power(code.int() - 127)


def block_power(v, emax):
    """X of each block of 32 values along the last axis, in 64 bits."""
    most = v.unflatten(-1, (-1, BLOCK)).abs().amax(-1)
    e = ((most.contiguous().view(torch.int64) >> 52) - 1023 - emax).clamp(min=-127)
    return power(torch.where(most > 0, e, -127))


def exact_norm(s):
    case = s["case"]
    h = s["x"].double()
    if s["residual"] is not None:
        h = (h + s["residual"].double()).to(s["x"].dtype).double()
    rstd = (h.pow(2).mean(-1) + EPS).rsqrt()
    y = torch.einsum("rc,r,c->rc", h, rstd, s["w"].double())
    full = torch.zeros((case["rows"], blocks(case["cols"]) * BLOCK), dtype=torch.float64, device=y.device)
    full[:, :case["cols"]] = y
    x = block_power(full, FP8[case["fmt"]][1])
    # The elements are given before their rounding to 8 bits: y is a rounded number itself, and next to the
    # middle of two elements, or its block's largest next to a power of two, either result is right.  So an
    # element's own rounding is part of both sides' distance from it, and the scales have no value here.
    out = {"q": (full.unflatten(-1, (-1, BLOCK)) / x.unsqueeze(-1)).flatten(-2), "s": None, "rstd": rstd}
    if s["residual"] is not None:
        out["h"] = h
    if case["y"]:
        out["y"] = y
    return out


def exact_norm_grad(s):
    h, dy, w, n = s["h"].double(), s["dy"].double(), s["w"].double(), s["h"].shape[1]
    r = s["rstd"].double()
    # dx_j = r w_j dy_j - r^3 h_j (sum_i w_i dy_i h_i) / n
    dot = torch.mv(dy * h, w)
    dx = dy * w * r[:, None] - h * (r.pow(3) * dot / n)[:, None]
    if s["dh"] is not None:
        dx += s["dh"].double()
    return {"dx": dx, "dw": torch.mv((dy * h).t(), r)}


def exact_gemv(s):
    q, k = s["w_q"], s["case"]["K"]
    table = decoded("e2m1", q.device)
    w = torch.empty((q.shape[0], 2 * q.shape[1]), dtype=torch.float64, device=q.device)
    w[:, 0::2], w[:, 1::2] = table[(q & 15).long()], table[(q >> 4).long()]
    w *= powers(s["w_s"]).repeat_interleave(BLOCK, 1)
    return s["x"].double() @ w[:, :k].t()


def exact_write(s):
    case, c = s["case"], s["cache"]
    _, emax, top = FP8[case["fmt"]]
    man, emin = {"e4m3": (3, -6), "e5m2": (2, -14)}[case["fmt"]]
    out = {}
    for name in ("k", "v"):
        v = s[name].double()
        x = block_power(v, emax)
        p = v.unflatten(-1, (-1, BLOCK)) / x.unsqueeze(-1)
        e = torch.frexp(p.abs())[1] - 1
        step = power(e.clamp(min=emin) - man)
        p = (torch.round(p / step) * step).clamp(-top, top).flatten(-2)
        q = decoded(case["fmt"], v.device)[c[name + "_q"].long()]
        sc = powers(c[name + "_s"])
        for t, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                q[slot // case["page"], :, slot % case["page"]] = p[t]
                sc[slot // case["page"], :, slot % case["page"]] = x[t]
        out[name + "_q"], out[name + "_s"] = q, sc
    return out


def exact_attention(s):
    case, c = s["case"], s["cache"]
    lq, heads, g, dim, page = case["Lq"], case["Hkv"], case["G"], case["D"], case["page"]
    table = decoded(case["fmt"], s["q"].device)
    o = torch.zeros((case["B"], lq, heads * g, dim), dtype=torch.float64, device=table.device)
    lse = torch.full(o.shape[:3], -math.inf, dtype=torch.float64, device=table.device)
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        at = s["table"][b, :blocks_of(n, page)].long()
        kv = []
        for name in ("k", "v"):
            v = table[c[name + "_q"][at].long()] * powers(c[name + "_s"][at]).repeat_interleave(BLOCK, -1)
            kv.append(v.permute(1, 0, 2, 3).reshape(heads, -1, dim)[:, :n].contiguous())
        for i in range(lq):
            end = n - lq + 1 + i
            if end <= 0:
                continue
            q = s["q"][b, i].double().view(heads, g, dim)
            a = torch.bmm(q, kv[0][:, :end].transpose(1, 2).contiguous()) / math.sqrt(dim)
            z = torch.logsumexp(a, -1, keepdim=True)
            o[b, i] = torch.bmm(torch.exp(a - z), kv[1][:, :end].contiguous()).reshape(heads * g, dim)
            lse[b, i] = z.reshape(heads * g)
    return {"o": o, "lse": lse}


EXACT = {"norm": exact_norm, "norm_grad": exact_norm_grad, "gemv": exact_gemv, "write": exact_write,
         "attention": exact_attention}


def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))
