"""The paged 8-bit MX key/value cache and attention over it, on the GPU.

The write is compared bit for bit with the oracle's quantization of each token's
head.  Attention is compared, over the oracle's dequantized cache, with the 64-bit
softmax of layer_ref and its error bound."""
import numpy as np
import pytest
import torch

import layer_ref as ref
from gpu_util import Guarded, dev, host, say
from microscaling_block_scaled_amd.synth import bf16_bits, bf16_to_f32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    from microscaling_block_scaled_amd import mx as m
    return m


# ---------------------------------------------------------------------------
# write
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("tokens,heads,dim,page", [(1, 1, 64, 16), (7, 3, 128, 48), (40, 8, 128, 16), (5, 17, 256, 64),
                                                   (90, 2, 64, 32), (3, 40, 64, 16)])
def test_write(mx, oracle, tokens, heads, dim, page, kind, fmt):
    rng = np.random.default_rng(tokens * 100 + heads + dim)
    pages = -(-tokens // page) + 2
    k, v = ((rng.standard_normal((tokens, heads, dim)) * np.exp2(rng.integers(-20, 21, (tokens, heads, 1)))).astype(
        np.float32) for _ in range(2))
    if kind == "bf16":
        k, v = bf16_to_f32(bf16_bits(k)), bf16_to_f32(bf16_bits(v))
    k[0, 0, :32] = 0.0
    if tokens > 4:
        k[2, 0, 3], v[3, 1, 40] = np.inf, np.nan
    slots = rng.permutation(pages * page)[:tokens].astype(np.int64)
    if tokens > 4:
        slots[1], slots[4] = -1, pages * page  # outside: not written
    shapes = {"k_q": dim, "k_s": dim // 32, "v_q": dim, "v_s": dim // 32}
    g = {n: Guarded((pages, heads, page, c)) for n, c in shapes.items()}
    for x in g.values():
        x.t.fill_(0x33)
    want = {n: np.full((pages, heads, page, c), 0x33, np.uint8) for n, c in shapes.items()}
    for name, a in (("k", k), ("v", v)):
        o = oracle.quantize(np.ascontiguousarray(a.reshape(tokens * heads, dim)), fmt, oracle.LAYOUT_ROW)
        q, s = o["q_row"].reshape(tokens, heads, dim), o["s_row"].reshape(tokens, heads, dim // 32)
        for t, slot in enumerate(slots):
            if 0 <= slot < pages * page:
                want[name + "_q"][slot // page, :, slot % page] = q[t]
                want[name + "_s"][slot // page, :, slot % page] = s[t]
    # keys and values as two parts of one projection, heads further apart than dim
    both = torch.full((tokens, 2, heads, dim + 16), float("nan"), dtype=torch.bfloat16 if kind == "bf16" else torch.float32,
                      device="cuda")
    both[:, 0, :, :dim] = dev(bf16_bits(k) if kind == "bf16" else k)
    both[:, 1, :, :dim] = dev(bf16_bits(v) if kind == "bf16" else v)
    say("cache write", tokens, heads, dim, page, kind, fmt)
    mx.cache_write(both[:, 0, :, :dim], both[:, 1, :, :dim], dev(slots), {n: x.t for n, x in g.items()}, fmt)
    torch.cuda.synchronize()
    for n, x in g.items():
        x.check(n)
        assert np.array_equal(host(x.t), want[n]), n


def test_write_broadcast(mx):
    """One key head for all heads, by a stride of 0."""
    k = torch.randn((4, 1, 64), device="cuda")
    c, d = mx.kv_cache(2, 3, 16, 64), mx.kv_cache(2, 3, 16, 64)
    slots = torch.arange(4, device="cuda")
    mx.cache_write(k.expand(4, 3, 64), k.expand(4, 3, 64), slots, c, mx.E4M3)
    mx.cache_write(k.repeat(1, 3, 1), k.repeat(1, 3, 1), slots, d, mx.E4M3)
    assert all(torch.equal(c[n], d[n]) for n in c)


def test_write_of_more_tokens_than_a_grid_holds_threads_for(mx):
    """2^24 tokens and some of 32 heads, a workgroup of 256 threads each; all but a few
    have no slot."""
    tokens = 2 ** 24 + 5
    k, v = (torch.randn((1, 32, 64), device="cuda") for _ in range(2))
    slots = torch.full((tokens,), -1, dtype=torch.int64, device="cuda")
    slots[3], slots[-1] = 1, 17
    c, d = mx.kv_cache(2, 32, 16, 64), mx.kv_cache(2, 32, 16, 64)
    for t in (*c.values(), *d.values()):
        t.zero_()
    say("cache write of 2^24 tokens")
    mx.cache_write(k.expand(tokens, 32, 64), v.expand(tokens, 32, 64), slots, c, mx.E4M3)
    mx.cache_write(k.repeat(2, 1, 1), v.repeat(2, 1, 1), torch.tensor([1, 17], device="cuda"), d, mx.E4M3)
    assert all(torch.equal(c[n], d[n]) for n in c)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
class Case:
    """A cache whose every byte outside the requests' tokens is hostile (NaN elements,
    NaN scales), and queries."""

    def __init__(self, oracle, rng, lens, Lq, heads, group, dim, page, fmt, size=1.0, table_extra=1):
        self.lens, self.Lq, self.heads, self.group, self.dim, self.page, self.fmt = lens, Lq, heads, group, dim, page, fmt
        B = len(lens)
        per = -(-max(max(lens), 1) // page) + table_extra
        pages = B * per + 2
        self.cache = {n: np.full((pages, heads, page, c), 0xFF, np.uint8)
                      for n, c in (("k_q", dim), ("k_s", dim // 32), ("v_q", dim), ("v_s", dim // 32))}
        self.cache["k_q"][:], self.cache["v_q"][:] = 0x7F, 0x7F
        self.table = rng.permutation(pages)[:B * per].reshape(B, per).astype(np.int32)
        self.k, self.v = [], []
        for b, n in enumerate(lens):
            kv = []
            for name in ("k", "v"):
                a = (rng.standard_normal((n, heads, dim)) * np.exp2(rng.integers(-2, 3, (n, heads, 1)))).astype(np.float32)
                o = oracle.quantize(np.ascontiguousarray(a.reshape(n * heads, dim)), fmt, oracle.LAYOUT_ROW)
                q, s = o["q_row"].reshape(n, heads, dim), o["s_row"].reshape(n, heads, dim // 32)
                for t in range(n):
                    at = (self.table[b, t // page], slice(None), t % page)
                    self.cache[name + "_q"][at], self.cache[name + "_s"][at] = q[t], s[t]
                kv.append(oracle.dequantize(o["q_row"], o["s_row"], fmt, n * heads, dim).astype(np.float64)
                          .reshape(n, heads, dim) if n else np.zeros((0, heads, dim)))
            self.k.append(kv[0])
            self.v.append(kv[1])
        self.q = bf16_to_f32(bf16_bits((rng.standard_normal((B, Lq, heads * group, dim)) * size).astype(np.float32)))

    def device(self):
        self.dcache = {n: dev(a) for n, a in self.cache.items()}
        self.dtable, self.dlens = dev(self.table), dev(np.array(self.lens, np.int32))
        return dev(bf16_bits(self.q)).view(self.q.shape)

    def reference(self, scale, limits=None):
        B, Lq, hq, dim = self.q.shape
        o, lse = np.zeros(self.q.shape), np.zeros((B, Lq, hq))
        bo, bl = np.zeros_like(o), np.zeros_like(lse)
        for b in range(B):
            lim = [self.lens[b] - Lq + 1 + i for i in range(Lq)] if limits is None else limits[b]
            for h in range(hq):
                kv = h // self.group
                o[b, :, h], lse[b, :, h], bo[b, :, h], bl[b, :, h] = ref.attention(
                    self.q[b, :, h].astype(np.float64), self.k[b][:, kv], self.v[b][:, kv], lim, scale)
        return o, lse, bo, bl

    def compare(self, got, scale, limits=None, rows=slice(None)):
        o, lse, bo, bl = self.reference(scale, limits)
        go, gl = host(got["o"].float()).astype(np.float64), host(got["lse"]).astype(np.float64)
        tol = bo + ref.HALF_BF16 * (np.abs(o) + bo) + 2.0 ** -133
        assert (np.abs(go - o) <= tol)[rows].all(), (np.abs(go - o) / tol)[rows].max()
        empty = np.isneginf(lse)
        assert np.array_equal(np.isneginf(gl), empty) and (go[empty] == 0).all()
        assert (np.abs(gl - lse)[~empty] <= bl[~empty]).all()


# lengths of nothing and one, around a step of 32, a wave's and a workgroup's share,
# the end of a page, and the split in pieces
SHAPES = [
    # lens, Lq, heads, group, dim, page, fmt
    ([0, 1, 2, 15, 16, 17], 1, 1, 1, 64, 16, 0),
    ([31, 32, 33, 63, 64, 65], 1, 2, 4, 128, 16, 0),
    ([127, 128, 129, 0, 255, 257], 1, 1, 5, 128, 48, 1),
    ([300, 7, 1000], 1, 2, 16, 64, 32, 1),
    ([1100, 1], 1, 1, 8, 256, 64, 0),
    ([3000, 1500, 0, 2049], 1, 2, 4, 128, 64, 0),
    ([2500, 1025], 1, 3, 2, 64, 16, 0),
    ([700], 1, 1, 24, 128, 16, 0),     # more rows than one tile
    ([500, 90], 1, 1, 40, 64, 16, 0),  # four tiles
    ([40, 3, 0, 1], 4, 2, 2, 128, 16, 0),  # some queries see nothing
    ([200, 33, 5], 7, 1, 7, 64, 16, 1),
    ([1300, 64, 31], 33, 2, 2, 128, 32, 0),
    ([90, 1200], 20, 1, 4, 64, 16, 0),
    ([150, 40], 9, 1, 3, 256, 16, 1),
    ([20], 20, 2, 1, 128, 16, 0),      # a whole prompt
    ([129], 129, 1, 4, 64, 16, 0),
]


@pytest.mark.parametrize("lens,Lq,heads,group,dim,page,fmt", SHAPES)
def test_attention(mx, oracle, lens, Lq, heads, group, dim, page, fmt):
    rng = np.random.default_rng(sum(lens) + Lq * 1000 + dim)
    c = Case(oracle, rng, lens, Lq, heads, group, dim, page, fmt)
    q = c.device()
    out = {"o": Guarded(q.shape, torch.bfloat16), "lse": Guarded(q.shape[:3], torch.float32)}
    say("attention", lens, Lq, heads, group, dim, page, fmt)
    got = mx.attention(q, c.dcache, fmt, c.dtable, c.dlens, out={n: g.t for n, g in out.items()})
    torch.cuda.synchronize()
    for n, g in out.items():
        g.check(n)
    c.compare(got, dim ** -0.5)
    again = mx.attention(q, c.dcache, fmt, c.dtable, c.dlens)
    assert torch.equal(got["o"], again["o"]) and torch.equal(got["lse"], again["lse"])


def test_sharp_and_flat_scores(mx, oracle):
    """Scores of hundreds (one token takes all, maxima move often), of zero, and a
    negative scale."""
    rng = np.random.default_rng(1)
    c = Case(oracle, rng, [2100, 77], 1, 1, 4, 128, 16, 0, size=8.0)
    q = c.device()
    for scale in (1.0, 0.0, -0.5):
        say("attention scale", scale)
        c.compare(mx.attention(q, c.dcache, 0, c.dtable, c.dlens, scale=scale), scale)


def test_strided_queries_and_bounds_of_lens(mx, oracle):
    """Queries inside a joint projection; lens past max_len and below zero are clamped;
    a workspace of the caller's."""
    rng = np.random.default_rng(2)
    c = Case(oracle, rng, [1500, 1400, 0], 2, 2, 3, 128, 16, 0)
    q = c.device()
    B, Lq, hq, dim = q.shape
    joint = torch.full((B, Lq, hq + 4, dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    joint[:, :, 2:2 + hq] = q
    lens = dev(np.array([1500, 2 ** 30, -5], np.int32))
    c.lens = [1400, 1400, 0]
    c.k, c.v = [a[:1400] for a in c.k], [a[:1400] for a in c.v]
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    say("attention strides")
    c.compare(mx.attention(joint[:, :, 2:2 + hq], c.dcache, 0, c.dtable, lens, max_len=1400, workspace=ws), dim ** -0.5)


def test_pages_that_are_not_there(mx, oracle):
    """Table entries outside the cache hold no tokens: the others are seen as if the
    sequence had no such place."""
    rng = np.random.default_rng(3)
    for lens, page in (([200], 32), ([1500], 48)):
        c = Case(oracle, rng, lens, 1, 1, 4, 128, page, 0)
        c.table[0, 1], c.table[0, 3] = -1, 10 ** 6
        q = c.device()
        keep = np.ones(lens[0], bool)
        keep[page:2 * page] = keep[3 * page:4 * page] = False
        c.k, c.v = [c.k[0][keep]], [c.v[0][keep]]
        say("attention missing pages", lens)
        c.compare(mx.attention(q, c.dcache, 0, c.dtable, c.dlens), 128 ** -0.5, limits=[[keep.sum()]])
    c.table[:] = -7
    c.device()
    got = mx.attention(q, c.dcache, 0, c.dtable, c.dlens)
    assert (got["o"] == 0).all() and torch.isneginf(got["lse"]).all()


@pytest.mark.parametrize("dim,group,Lq", [(64, 1, 40), (128, 2, 24), (256, 1, 20), (128, 1, 5)])
def test_not_finite_values_reach_only_who_sees_them(mx, oracle, dim, group, Lq):
    """A NaN value (and an infinite one, in E5M2) of a late token: queries before it
    are as without it, queries from it on are NaN (or infinite) in its dims."""
    rng = np.random.default_rng(dim + Lq)
    for fmt in (0, 1):
        n = 100
        c = Case(oracle, rng, [n], Lq, 1, group, dim, 16, fmt)
        q = c.device()
        clean = mx.attention(q, c.dcache, fmt, c.dtable, c.dlens)
        tok, d = n - Lq // 2, 37
        page, at = c.table[0, tok // 16], tok % 16
        c.dcache["v_q"][page, 0, at, d] = 0x7F if fmt == 0 else 0x7C
        say("attention NaN", dim, group, Lq, fmt)
        got = mx.attention(q, c.dcache, fmt, c.dtable, c.dlens)
        see = Lq - (n - tok)  # the first query that sees the token
        assert torch.equal(got["lse"], clean["lse"])
        # summed another way where a step holds the value: one bf16 step apart at most
        a, b = got["o"].float()[:, :see], clean["o"].float()[:, :see]
        assert torch.isfinite(a).all() and (a - b).abs().max() <= 2.0 ** -7 * b.abs().max()
        late = got["o"].float()[:, see:]
        assert not torch.isfinite(late[..., d]).any()
        assert torch.isfinite(late[..., :d]).all() and torch.isfinite(late[..., d + 1:]).all()
        # a NaN scale takes its block of 32 dims
        c.dcache["v_q"][page, 0, at, d] = 0
        c.dcache["v_s"][page, 0, at, 1] = 0xFF
        got = mx.attention(q, c.dcache, fmt, c.dtable, c.dlens)["o"].float()
        assert torch.isfinite(got[:, :see]).all()
        assert torch.isnan(got[:, see:, :, 32:64]).all() and torch.isfinite(got[:, see:, :, :32]).all()
        # a NaN key: nothing for those before it, NaN for those that see it
        c.dcache["v_s"][page, 0, at, 1] = 120
        c.dcache["k_s"][page, 0, at, 0] = 0xFF
        got = mx.attention(q, c.dcache, fmt, c.dtable, c.dlens)
        assert torch.isfinite(got["o"].float()[:, :see]).all() and torch.isnan(got["o"].float()[:, see:]).all()


def test_past_4_gib(mx, oracle):
    """Cache offsets past 32 bits: 36000 pages of 8 heads x 128 tokens x 128 (4.7 GB of
    keys, as much of values), a request in the last ones."""
    rng = np.random.default_rng(8)
    c = Case(oracle, rng, [300], 1, 8, 2, 128, 128, 0)
    q = c.device()
    pages, shift = 36000, 36000 - c.cache["k_q"].shape[0]
    big = mx.kv_cache(pages, 8, 128, 128)
    for n, t in c.dcache.items():
        big[n][shift:] = t
    say("attention past 4 GiB")
    c.compare(mx.attention(q, big, 0, c.dtable + shift, c.dlens), 128 ** -0.5)
    k = torch.randn((1, 8, 128), device="cuda")
    mx.cache_write(k, k, torch.tensor([pages * 128 - 1], device="cuda"), big, mx.E4M3)
    want = mx.quantize(k[0], mx.E4M3)
    assert torch.equal(big["k_q"][-1, :, -1], want["q_row"]) and torch.equal(big["v_s"][-1, :, -1], want["s_row"])


@pytest.mark.parametrize("Lq", [1, 20])
@pytest.mark.parametrize("page", [48, 65520])
def test_pages_of_a_long_request(mx, page, Lq):
    """26 million tokens, in pages whose size is no power of two: the page of every
    token is found.  All but the last of a request's pages are one page of the cache; the
    largest key is in the last 16 tokens of another, which the table names last."""
    dim = 64
    n = 400 * 65520 // page
    cache = mx.kv_cache(3, 1, page, dim)
    for t in cache.values():
        t.zero_()
    cache["k_s"].fill_(127)
    cache["v_s"].fill_(127)
    # page 0 holds ones, page 1 a key that every query takes, with fours; 2 is never named
    cache["v_q"][0], cache["v_q"][1], cache["v_q"][2] = 0x38, 0x48, 0x7F
    cache["k_q"][1, 0, page - 3] = 0x48  # 4: its score is 64 * 4 / 8 = 32 more than the others'
    table = torch.zeros((1, n), dtype=torch.int32, device="cuda")
    table[0, n - 1] = 1
    q = torch.ones((1, Lq, 1, dim), dtype=torch.bfloat16, device="cuda")
    lens = torch.tensor([n * page], dtype=torch.int32, device="cuda")
    say("attention over pages of a long request", page, Lq)
    r = mx.attention(q, cache, mx.E4M3, table, lens)
    got, lse = host(r["o"].float()).astype(np.float64), host(r["lse"]).astype(np.float64)
    for i in range(Lq):
        total = n * page - Lq + i + 1  # tokens that the query sees
        fours = total - (n - 1) * page
        top = np.exp(32.0) if total > n * page - 3 else 0.0
        near = fours - (1 if top else 0)
        l = (n - 1) * page + near + top
        o = ((n - 1) * page + 4.0 * (near + top)) / l
        assert np.abs(got[0, i] - o).max() <= 2.0 ** -7 * o, (i, got[0, i].max(), o)
        assert abs(lse[0, i] - np.log(l)).max() <= 1e-4 * np.log(l), (i, lse[0, i], np.log(l))


def test_other_stream_and_graph(mx, oracle):
    """On a stream that is handed over, and replayed from a graph, results are those of
    the eager call on the current stream."""
    rng = np.random.default_rng(9)
    c = Case(oracle, rng, [1500, 900], 1, 2, 4, 128, 16, 0)
    q = c.device()
    want = mx.attention(q, c.dcache, 0, c.dtable, c.dlens)
    x, w = torch.randn((5, 512), device="cuda").to(torch.bfloat16), torch.randn((96, 512), device="cuda")
    p = mx.quantize(w, mx.E2M1)
    y = mx.gemv(x, p["q_row"], p["s_row"], mx.E2M1, 5, 96, 512)
    nw = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    n = mx.rmsnorm_quantize(x, nw, mx.E4M3, residual=x)
    gr = mx.rmsnorm_backward(x, n["h"], nw, n["rstd"])
    torch.cuda.synchronize()

    def run(stream=None):
        a = mx.attention(q, c.dcache, 0, c.dtable, c.dlens, stream=stream)
        b = mx.gemv(x, p["q_row"], p["s_row"], mx.E2M1, 5, 96, 512, stream=stream)
        d = mx.rmsnorm_quantize(x, nw, mx.E4M3, residual=x, stream=stream)
        e = mx.rmsnorm_backward(x, d["h"], nw, d["rstd"], stream=stream)
        return a["o"], a["lse"], b, d["q_row"], d["h"], e["dx"], e["dw"]

    ref_out = (want["o"], want["lse"], y, n["q_row"], n["h"], gr["dx"], gr["dw"])
    s = torch.cuda.Stream()
    say("other stream")
    got = run(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref_out))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for i in range(4):
        for t in held:
            t.zero_()
        say("graph replay", i)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, ref_out)), i
        assert torch.equal(mx.attention(q, c.dcache, 0, c.dtable, c.dlens)["o"], want["o"])


def test_refusals(mx):
    c = mx.kv_cache(4, 2, 16, 64)
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device="cuda")
    i32, i64 = torch.int32, torch.int64
    q, table, lens = z(1, 1, 4, 64), z(1, 2, t=i32), z(1, t=i32)
    ok = lambda **k: mx.attention(k.get("q", q), k.get("c", c), k.get("fmt", mx.E4M3), k.get("table", table),
                                  k.get("lens", lens), max_len=k.get("max_len"), workspace=k.get("ws"))
    ok()
    for bad in (dict(q=z(1, 1, 4, 32)), dict(q=z(1, 1, 4, 64, t=torch.float32)), dict(q=z(1, 1, 4, 128)[..., ::2]),
                dict(table=z(2, 2, t=i32)), dict(table=z(1, 2, t=i64)), dict(lens=z(2, t=i32)),
                dict(c=c | {"v_s": c["v_s"][:, :1]}), dict(ws=z(4, t=torch.float32))):
        with pytest.raises(ValueError):
            ok(**bad)

    def status(call, want):
        with pytest.raises(mx.MXError) as err:
            call()
        assert err.value.status == want

    status(lambda: ok(max_len=33), mx.MX_ERR_SHAPE)             # more than the table holds
    status(lambda: ok(max_len=-1), mx.MX_ERR_ARG)
    status(lambda: ok(q=z(1, 1, 3, 64)), mx.MX_ERR_SHAPE)       # 3 query heads over 2
    status(lambda: ok(fmt=mx.INT8), mx.MX_ERR_UNSUPPORTED)
    status(lambda: ok(c=mx.kv_cache(4, 2, 24, 64)), mx.MX_ERR_UNSUPPORTED)
    status(lambda: ok(c=mx.kv_cache(4, 2, 16, 96), q=z(1, 1, 4, 96)), mx.MX_ERR_UNSUPPORTED)
    long = z(1, 200, t=i32)
    status(lambda: ok(table=long, ws=z(16, t=torch.uint8)), mx.MX_ERR_SHAPE)  # workspace too small
    off = torch.zeros(4 * 64 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(1, 1, 4, 64)
    status(lambda: ok(q=off), mx.MX_ERR_ALIGN)
    k, slots = z(3, 2, 64), z(3, t=i64)
    for bad in (dict(k=z(3, 2, 32)), dict(v=z(3, 2, 64, t=torch.float32)), dict(slots=z(3, t=i32)), dict(slots=z(2, t=i64))):
        a = dict(k=k, v=k, slots=slots) | bad
        with pytest.raises(ValueError):
            mx.cache_write(a["k"], a["v"], a["slots"], c, mx.E4M3)
    status(lambda: mx.cache_write(k, k, slots, c, mx.E2M1), mx.MX_ERR_UNSUPPORTED)
    status(lambda: mx.cache_write(z(3, 2, 68)[..., :64], k, slots, c, mx.E4M3), mx.MX_ERR_ALIGN)


def test_empty(mx):
    c = mx.kv_cache(4, 2, 16, 64)
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device="cuda")
    o = mx.attention(z(0, 1, 4, 64), c, mx.E4M3, z(0, 2, t=torch.int32), z(0, t=torch.int32))
    assert o["o"].shape == (0, 1, 4, 64)
    # a cache or a table of nothing: queries see nothing
    for cc, tab in ((mx.kv_cache(0, 2, 16, 64), z(2, 3, t=torch.int32)), (c, z(2, 0, t=torch.int32))):
        lens = torch.full((2,), 5, dtype=torch.int32, device="cuda")
        o = mx.attention(z(2, 1, 4, 64), cc, mx.E4M3, tab, lens)
        assert (o["o"] == 0).all() and torch.isneginf(o["lse"]).all()
    mx.cache_write(z(0, 2, 64), z(0, 2, 64), z(0, t=torch.int64), c, mx.E4M3)


def test_bound_past_a_table_that_is_a_slice(mx):
    """A table of 2 columns within rows of 8: a bound of 33 tokens in pages of 16 is refused."""
    c = mx.kv_cache(4, 2, 16, 64)
    wide = torch.zeros((2, 8), dtype=torch.int32, device="cuda")
    q = torch.zeros((2, 1, 4, 64), dtype=torch.bfloat16, device="cuda")
    lens = torch.full((2,), 20, dtype=torch.int32, device="cuda")
    a = mx.attention(q, c, mx.E4M3, wide[:, :2], lens, max_len=32)
    b = mx.attention(q, c, mx.E4M3, wide[:, :2].contiguous(), lens)
    assert torch.equal(a["o"], b["o"]) and torch.equal(a["lse"], b["lse"])
    with pytest.raises(mx.MXError) as err:
        mx.attention(q, c, mx.E4M3, wide[:, :2], lens, max_len=33)
    assert err.value.status == mx.MX_ERR_SHAPE


@pytest.mark.parametrize("B,most", [(16, 1100), (32, 2100)])
def test_many_requests_without_pieces(mx, oracle, B, most):
    """Requests and heads that fill the chip: more than 1024 tokens by one workgroup."""
    rng = np.random.default_rng(B)
    lens = [most, 0, 1] + [int(n) for n in rng.integers(1, 80, B - 3)]
    c = Case(oracle, rng, lens, 1, 8, 2, 64, 16, 0)
    say("attention, many requests", B, most)
    c.compare(mx.attention(c.device(), c.dcache, 0, c.dtable, c.dlens), 64 ** -0.5)
