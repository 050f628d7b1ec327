"""Root-mean-square norm with the residual's addition and MX output, and its
gradient, on the GPU.

Forward: h, y and the codes follow from the returned rstd by single fp32
operations, so given it they are compared bit for bit (codes against the oracle's
quantization of that fp32 y); rstd is held to the bound of its sum.  Gradient:
against the 64-bit formula within the bounds of layer_ref, and against central
differences of the 64-bit forward."""
import numpy as np
import pytest
import torch

import layer_ref as ref
from gpu_util import Guarded, dev, host, say
from microscaling_block_scaled_amd.synth import bf16_bits, bf16_to_f32

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module")
def mx():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    from microscaling_block_scaled_amd import mx as m
    return m


def values(rng, shape, kind, std=1.0):
    """fp32 values of the source type."""
    a = (rng.standard_normal(shape) * std).astype(np.float32)
    return bf16_to_f32(bf16_bits(a)) if kind == "bf16" else a


def to_dev(a, kind, pitch=None):
    """On the GPU in the source type, in rows `pitch` elements apart whose gaps hold
    NaN."""
    t = dev(bf16_bits(a) if kind == "bf16" else a)
    if pitch is None:
        return t
    full = torch.full((a.shape[0], pitch), float("nan"), dtype=t.dtype, device="cuda")
    full[:, :a.shape[1]] = t
    return full[:, :a.shape[1]]


def round_to(a, kind):
    return bf16_to_f32(bf16_bits(a)) if kind == "bf16" else a


def pitch_of(cols, kind):
    per = 8 if kind == "bf16" else 4
    return -(-cols // per) * per


SIZES = [(1, 1), (3, 31), (2, 32), (5, 100), (4, 511), (7, 512), (3, 1000), (9, 1024), (2, 2050), (1030, 72),
         (5, 4096), (3, 4100), (2, 8192), (2, 9000), (2, 16384), (2, 16500)]


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_forward(mx, oracle, rows, cols, kind):
    rng = np.random.default_rng(rows * 7919 + cols)
    fmt = (rows + cols) % 6
    for residual in (True, False):
        x = values(rng, (rows, cols), kind)
        r = values(rng, (rows, cols), kind, 3.0)
        w = values(rng, (cols,), kind) + np.float32(0.0)
        if rows > 1:
            x[1] = r[1] = 0.0  # a row whose mean square is eps alone
        h = round_to(x + r, kind) if residual else x
        pitch = pitch_of(cols, kind) + (8 if rows % 2 else 0)
        o = {"q_row": Guarded((rows, mx.packed_bytes(fmt, 1, cols))), "s_row": Guarded((rows, -(-cols // 32))),
             "rstd": Guarded((rows,), torch.float32)}
        say("norm", rows, cols, kind, fmt, residual)
        got = mx.rmsnorm_quantize(to_dev(x, kind, pitch), dev(bf16_bits(w) if kind == "bf16" else w), fmt, EPS,
                                  residual=to_dev(r, kind, pitch) if residual else None, want_y=True,
                                  out={k: g.t for k, g in o.items()})
        torch.cuda.synchronize()
        for k, g in o.items():
            g.check(k)
        rstd = host(got["rstd"])
        want = ref.norm(h.astype(np.float64), w.astype(np.float64), EPS)[0]
        # half the sum's error, then division, addition, root and reciprocal
        assert (np.abs(rstd - want) <= (ref.norm_depth(cols) / 2 + 5) * ref.U * want).all()
        if residual:
            assert np.array_equal(host(got["h"].float()), h)
        y = (h * rstd[:, None]) * w
        assert np.array_equal(host(got["y"].float()), round_to(y, kind))
        q = oracle.quantize(y, fmt, oracle.LAYOUT_ROW)
        assert np.array_equal(host(got["q_row"]), q["q_row"]) and np.array_equal(host(got["s_row"]), q["s_row"])


@pytest.mark.parametrize("fmt", range(6))
def test_forward_formats_and_values(mx, oracle, fmt):
    """Every format; values over 2^-60 .. 2^60 per row and per column, subnormals,
    signed zeros, infinities and NaN (a row with them gives what the formulas give)."""
    rng = np.random.default_rng(fmt)
    rows, cols = 40, 330
    x = values(rng, (rows, cols), "fp32") * np.exp2(rng.integers(-60, 61, (rows, 1))).astype(np.float32)
    w = (values(rng, (cols,), "fp32") * np.exp2(rng.integers(-60, 61, cols))).astype(np.float32)
    w[::17] = 0.0
    x[:, 5] = -0.0
    x[3] = np.float32(1e-41)
    x[4, 7], x[5, 7], x[6, 9] = np.inf, np.nan, -np.inf
    say("norm values", fmt)
    got = mx.rmsnorm_quantize(to_dev(x, "fp32", 332), dev(w), fmt, 0.0, want_y=True,
                              out={"y": torch.empty((rows, 332), device="cuda")[:, :cols]})
    rstd, y = host(got["rstd"]), host(got["y"])
    with np.errstate(all="ignore"):
        want = (x * rstd[:, None]) * w
    assert np.array_equal(y, want, equal_nan=True)
    assert np.isnan(rstd[5]) and rstd[4] == 0 and rstd[6] == 0
    q = oracle.quantize(y, fmt, oracle.LAYOUT_ROW)
    assert np.array_equal(host(got["s_row"]), q["s_row"]) and np.array_equal(host(got["q_row"]), q["q_row"])


def test_forward_in_place(mx, oracle):
    """h may be x or the residual; also where a row takes two passes."""
    rng = np.random.default_rng(11)
    for rows, cols in ((5, 200), (2, 16600)):
        x, r = values(rng, (rows, cols), "bf16"), values(rng, (rows, cols), "bf16")
        w = dev(bf16_bits(values(rng, (cols,), "bf16")))
        a = mx.rmsnorm_quantize(to_dev(x, "bf16"), w, mx.E4M3, EPS, residual=to_dev(r, "bf16"))
        for which in ("x", "residual"):
            tx, tr = to_dev(x, "bf16"), to_dev(r, "bf16")
            b = mx.rmsnorm_quantize(tx, w, mx.E4M3, EPS, residual=tr, out={"h": tx if which == "x" else tr})
            for k in ("q_row", "s_row", "rstd", "h"):
                assert torch.equal(a[k], b[k]), (which, k)


def test_forward_past_4_gib(mx, oracle):
    """Offsets past 32 bits: 640000 x 4096 in bf16, the last rows checked."""
    rows, cols = 640000, 4096
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(12)
    tail = values(rng, (3, cols), "bf16")
    x[-3:] = dev(bf16_bits(tail))
    w = values(rng, (cols,), "bf16")
    say("norm past 4 GiB")
    got = mx.rmsnorm_quantize(x, dev(bf16_bits(w)), mx.E4M3, EPS)
    y = (tail * host(got["rstd"][-3:])[:, None]) * w
    q = oracle.quantize(y, oracle.E4M3, oracle.LAYOUT_ROW)
    assert np.array_equal(host(got["q_row"][-3:]), q["q_row"])
    assert np.array_equal(host(got["s_row"][-3:]), q["s_row"])


def grad_case(rng, rows, cols, kind):
    h, dy, dh = values(rng, (rows, cols), kind), values(rng, (rows, cols), kind, 1e-3), values(rng, (rows, cols), kind, 1e-3)
    w = values(rng, (cols,), kind)
    rstd = ref.norm(h.astype(np.float64), w, EPS)[0].astype(np.float32)
    return h, dy, dh, w, rstd


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (2, 33), (9, 100), (300, 64), (5, 512), (600, 520), (33, 1024), (17, 2050),
                                       (513, 2048), (6, 4096), (3, 4100), (3, 8192), (2, 8200), (2, 16384), (70, 16500)])
def test_gradient(mx, rows, cols, kind):
    rng = np.random.default_rng(rows * 31 + cols)
    h, dy, dh, w, rstd = grad_case(rng, rows, cols, kind)
    for with_dh in (True, False):
        pitch = pitch_of(cols, kind) + 8
        dw = Guarded((cols,), torch.float32)
        say("norm gradient", rows, cols, kind, with_dh)
        got = mx.rmsnorm_backward(to_dev(dy, kind, pitch), to_dev(h, kind, pitch),
                                  dev(bf16_bits(w) if kind == "bf16" else w), dev(rstd),
                                  dh=to_dev(dh, kind, pitch) if with_dh else None, out={"dw": dw.t})
        dw.check("dw")
        d = dh.astype(np.float64) if with_dh else np.zeros((rows, cols))
        dx, want_w, bx, bw = ref.norm_grad(dy.astype(np.float64), h.astype(np.float64), w.astype(np.float64),
                                           rstd.astype(np.float64), d)
        if kind == "bf16":
            bx = bx + ref.HALF_BF16 * (np.abs(dx) + bx) + 2.0 ** -133
        assert (np.abs(host(got["dx"].float()) - dx) <= bx + 2.0 ** -148).all()
        assert (np.abs(host(got["dw"]) - want_w) <= bw + 2.0 ** -148).all()


def test_gradient_against_differences(mx):
    """The GPU's gradient along a direction against a central difference of the
    64-bit forward (step 1e-4: its own error is about 1e-8 of the derivative)."""
    rng = np.random.default_rng(21)
    rows, cols = 6, 300
    x, r, c, d, ux = (rng.standard_normal((rows, cols)).astype(np.float32) for _ in range(5))
    w, uw = ((1 + 0.3 * rng.standard_normal(cols)).astype(np.float32) for _ in range(2))
    f = mx.rmsnorm_quantize(dev(x), dev(w), mx.E4M3, EPS, residual=dev(r))
    g = mx.rmsnorm_backward(dev(c), f["h"], dev(w), f["rstd"], dh=dev(d))
    L = lambda a, b: ref.norm_loss(x + a * ux.astype(np.float64), r.astype(np.float64), w + b * uw.astype(np.float64),
                                   EPS, c.astype(np.float64), d.astype(np.float64))
    t = 1e-4
    dx, dw = host(g["dx"]).astype(np.float64), host(g["dw"]).astype(np.float64)
    # each element of dx carries some 40 u of its parts; the direction sums them
    for num, part, size in (((L(t, 0) - L(-t, 0)) / (2 * t), (dx * ux).sum(), np.abs(dx * ux).sum()),
                            ((L(0, t) - L(0, -t)) / (2 * t), (dw * uw).sum(), np.abs(dw * uw).sum())):
        assert abs(num - part) <= (100 * ref.U + 1e-7) * size


def test_gradient_in_place_and_repeatable(mx):
    rng = np.random.default_rng(22)
    for rows, cols in ((700, 1100), (3, 16600)):
        h, dy, dh, w, rstd = grad_case(rng, rows, cols, "bf16")
        t = lambda a: to_dev(a, "bf16", pitch_of(cols, "bf16"))
        tw, tr = dev(bf16_bits(w)), dev(rstd)
        a = mx.rmsnorm_backward(t(dy), t(h), tw, tr, dh=t(dh))
        for which in ("dy", "dh", "again"):
            b_dy, b_dh = t(dy), t(dh)
            out = {"dx": b_dy} if which == "dy" else {"dx": b_dh} if which == "dh" else None
            b = mx.rmsnorm_backward(b_dy, t(h), tw, tr, dh=b_dh, out=out)
            assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dw"], b["dw"]), which


def test_more_rows_than_a_grid_holds_threads_for(mx):
    """2^26 rows and some: workgroups of four rows, 256 threads each, pass 2^32 threads, and
    offsets 32 bits.  The last rows are those of a call of their own."""
    rows, n = 2 ** 26 + 11, 1003
    x = torch.zeros((rows, 32), dtype=torch.bfloat16, device="cuda")
    x[:n] = torch.randn((n, 32), device="cuda").bfloat16()
    x[-n:] = torch.randn((n, 32), device="cuda").bfloat16()
    w = torch.rand(32, device="cuda").bfloat16()
    say("norm of 2^26 rows")
    a = mx.rmsnorm_quantize(x, w, mx.E4M3)
    for part in (slice(0, n), slice(rows - n, rows)):
        b = mx.rmsnorm_quantize(x[part], w, mx.E4M3)
        for name in ("q_row", "s_row", "rstd"):
            assert torch.equal(a[name][part], b[name]), name


def test_empty(mx):
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")
    o = mx.rmsnorm_quantize(e(0, 64), e(64), mx.E4M3)
    assert o["q_row"].shape == (0, 64)
    g = mx.rmsnorm_backward(e(0, 64), e(0, 64), e(64), torch.empty(0, device="cuda"))
    assert g["dx"].shape == (0, 64) and (g["dw"] == 0).all()


def test_refusals(mx):
    e = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device="cuda")
    x, w = e(4, 64), e(64)
    for bad in (dict(x=e(4, 64, t=torch.float16)), dict(w=e(63)), dict(w=e(64, t=torch.float32)),
                dict(residual=e(3, 64)), dict(residual=e(4, 128)[:, ::2]), dict(fmt=9),
                dict(out={"h": e(4, 65)[:, :64], "q_row": e(2, 64, t=torch.uint8)})):
        a = dict(x=x, w=w, fmt=mx.E4M3) | bad
        with pytest.raises(ValueError):
            mx.rmsnorm_quantize(a["x"], a["w"], a["fmt"], residual=a.get("residual"), out=a.get("out"))
    for bad in (dict(x=e(4, 72)[:, 4:68]), dict(x=e(4, 68)[:, :64])):  # rows off 16 bytes
        with pytest.raises(mx.MXError) as err:
            mx.rmsnorm_quantize(bad["x"], w, mx.E4M3)
        assert err.value.status == mx.MX_ERR_ALIGN
    with pytest.raises(mx.MXError) as err:
        mx.rmsnorm_quantize(x, w, mx.E4M3, eps=-1.0)
    assert err.value.status == mx.MX_ERR_ARG
    with pytest.raises(mx.MXError) as err:
        mx.rmsnorm_backward(e(40, 64), e(40, 64), w, e(40, t=torch.float32), workspace=e(16, t=torch.uint8))
    assert err.value.status == mx.MX_ERR_SHAPE
    with pytest.raises(ValueError):
        mx.rmsnorm_backward(x, x, w, e(3, t=torch.float32))
