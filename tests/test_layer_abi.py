"""The decoder-layer entry points reject bad arguments on the host with the documented
status codes, and the binding refuses tensors that are not where or what it needs (no
GPU: every case returns before anything is launched)."""
import ctypes

import pytest
import torch

FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation fails first
no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="fake-pointer cases run on CPU only")


@pytest.fixture(scope="module")
def mx():
    from microscaling_block_scaled_amd import mx as m
    return m


@no_gpu
def test_rmsnorm_quantize_validation(mx):
    def f(x=FAKE, ld_x=64, r=FAKE, ld_r=64, w=FAKE, rows=4, cols=64, src=1, fmt=0, eps=1e-5, h=FAKE, ld_h=64, y=None,
          ld_y=0, q=FAKE, s=FAKE, rstd=FAKE):
        return mx.lib.mx_rmsnorm_quantize(x, ld_x, r, ld_r, w, rows, cols, src, fmt, eps, h, ld_h, y, ld_y, q, s, rstd,
                                          None)
    for bad in (dict(src=2), dict(fmt=6), dict(fmt=-1), dict(rows=-1), dict(cols=-1), dict(eps=-1e-9),
                dict(eps=float("nan")), dict(x=None), dict(w=None), dict(q=None), dict(s=None)):
        assert f(**bad) == mx.MX_ERR_ARG, bad
    for bad in (dict(ld_x=63), dict(ld_r=56), dict(ld_h=0), dict(y=FAKE, ld_y=32)):
        assert f(**bad) == mx.MX_ERR_SHAPE, bad
    for bad in (dict(x=FAKE + 8), dict(r=FAKE + 2), dict(w=FAKE + 8), dict(h=FAKE + 8), dict(y=FAKE + 8, ld_y=64),
                dict(q=FAKE + 8), dict(rstd=FAKE + 2), dict(ld_x=68), dict(src=0, ld_x=66, ld_r=66, ld_h=66)):
        assert f(**bad) == mx.MX_ERR_ALIGN, bad
    assert f(rows=1 << 31) == mx.MX_ERR_UNSUPPORTED
    big = (1 << 24) + 8
    assert f(cols=big, ld_x=big, ld_r=big, ld_h=big) == mx.MX_ERR_UNSUPPORTED
    assert f(rows=0, x=None) == mx.MX_OK and f(cols=0, ld_x=0, q=None) == mx.MX_OK


@no_gpu
def test_rmsnorm_backward_validation(mx):
    need = mx.lib.mx_rmsnorm_backward_workspace(40, 64, 1)
    assert need > 0 and need % (64 * 4) == 0
    for rows in (0, 1, 8):  # one workgroup needs none
        assert mx.lib.mx_rmsnorm_backward_workspace(rows, 64, 1) == 0
    for bad in ((-1, 64, 1), (4, -1, 1), (4, 64, 2), (1 << 31, 64, 1), (4, 1 << 25, 1)):
        assert mx.lib.mx_rmsnorm_backward_workspace(*bad) == -1

    def f(dy=FAKE, ld_dy=64, h=FAKE, ld_h=64, w=FAKE, rstd=FAKE, dh=FAKE, ld_dh=64, rows=40, cols=64, src=1, dx=FAKE,
          ld_dx=64, dw=FAKE, ws=FAKE, size=need):
        return mx.lib.mx_rmsnorm_backward(dy, ld_dy, h, ld_h, w, rstd, dh, ld_dh, rows, cols, src, dx, ld_dx, dw, ws,
                                          size, None)
    for bad in (dict(src=5), dict(rows=-1), dict(cols=-2), dict(dy=None), dict(h=None), dict(w=None), dict(rstd=None),
                dict(dx=None), dict(dw=None), dict(ws=None)):
        assert f(**bad) == mx.MX_ERR_ARG, bad
    for bad in (dict(ld_dy=8), dict(ld_h=63), dict(ld_dh=0), dict(ld_dx=56), dict(size=need - 1)):
        assert f(**bad) == mx.MX_ERR_SHAPE, bad
    for bad in (dict(dy=FAKE + 8), dict(ld_h=68), dict(dh=FAKE + 4), dict(dx=FAKE + 2), dict(w=FAKE + 8), dict(ws=FAKE + 8),
                dict(dw=FAKE + 2), dict(rstd=FAKE + 1)):
        assert f(**bad) == mx.MX_ERR_ALIGN, bad
    assert f(cols=0, dw=None) == mx.MX_OK


@no_gpu
def test_gemv_validation(mx):
    for call in (mx.lib.mx_gemv, mx.lib.mx_gemv_bf16):
        def f(x=FAKE, ld_x=64, q=FAKE, s=FAKE, fmt=4, M=2, N=8, K=64, y=FAKE, ld_y=8):
            return call(x, ld_x, q, s, fmt, M, N, K, y, ld_y, None)
        for bad in (dict(fmt=6), dict(fmt=-1), dict(M=-1), dict(N=-1), dict(K=-1, ld_x=0), dict(x=None), dict(q=None),
                    dict(s=None), dict(y=None)):
            assert f(**bad) == mx.MX_ERR_ARG, bad
        for fmt in (0, 1, 2, 3, 5):
            assert f(fmt=fmt) == mx.MX_ERR_UNSUPPORTED
        assert f(ld_x=63) == mx.MX_ERR_SHAPE and f(ld_y=7) == mx.MX_ERR_SHAPE
        for bad in (dict(x=FAKE + 1), dict(q=FAKE + 8), dict(y=FAKE + 1)):
            assert f(**bad) == mx.MX_ERR_ALIGN, bad
        assert f(M=32 * 65535 + 1) == mx.MX_ERR_UNSUPPORTED
        assert f(N=1 << 31, ld_y=1 << 31) == mx.MX_ERR_UNSUPPORTED
        assert f(M=0, x=None, y=None) == mx.MX_OK and f(N=0, ld_y=0, q=None) == mx.MX_OK
    assert mx.lib.mx_gemv(FAKE, 64, FAKE, FAKE, 4, 2, 8, 64, FAKE + 2, 8, None) == mx.MX_ERR_ALIGN  # fp32 on 2 bytes


def cache(mx, **k):
    a = dict(k_q=FAKE, k_s=FAKE, v_q=FAKE, v_s=FAKE, pages=4, heads=2, page=16, dim=64, fmt=0) | k
    return ctypes.byref(mx.Cache(*a.values()))


BAD_CACHES = [("MX_ERR_ARG", dict(fmt=7)), ("MX_ERR_ARG", dict(pages=-1)), ("MX_ERR_ARG", dict(heads=-1)),
              ("MX_ERR_ARG", dict(page=0)), ("MX_ERR_ARG", dict(dim=0)), ("MX_ERR_ARG", dict(k_q=None)),
              ("MX_ERR_ARG", dict(v_s=None)), ("MX_ERR_UNSUPPORTED", dict(fmt=4)), ("MX_ERR_UNSUPPORTED", dict(fmt=5)),
              ("MX_ERR_UNSUPPORTED", dict(dim=96)), ("MX_ERR_UNSUPPORTED", dict(page=24)),
              ("MX_ERR_UNSUPPORTED", dict(page=1 << 17)), ("MX_ERR_UNSUPPORTED", dict(heads=1 << 16)),
              ("MX_ERR_ALIGN", dict(k_q=FAKE + 8)), ("MX_ERR_ALIGN", dict(v_s=FAKE + 4))]


@no_gpu
def test_cache_write_validation(mx):
    def f(c=None, k=FAKE, ld_k=128, hs_k=64, v=FAKE, ld_v=128, hs_v=64, src=1, tokens=3, slots=FAKE, **kc):
        return mx.lib.mx_cache_write(c or cache(mx, **kc), k, ld_k, hs_k, v, ld_v, hs_v, src, tokens, slots, None)
    for want, bad in BAD_CACHES:
        assert f(**bad) == getattr(mx, want), bad
    assert mx.lib.mx_cache_write(None, FAKE, 128, 64, FAKE, 128, 64, 1, 3, FAKE, None) == mx.MX_ERR_ARG
    for bad in (dict(k=None), dict(v=None), dict(slots=None), dict(src=3), dict(tokens=-1), dict(ld_k=-8), dict(hs_v=-8)):
        assert f(**bad) == mx.MX_ERR_ARG, bad
    for bad in (dict(k=FAKE + 8), dict(v=FAKE + 2), dict(ld_k=132), dict(hs_v=68), dict(slots=FAKE + 4),
                dict(src=0, ld_v=130)):
        assert f(**bad) == mx.MX_ERR_ALIGN, bad
    assert f(tokens=1 << 31) == mx.MX_ERR_UNSUPPORTED
    assert f(tokens=0, k=None) == mx.MX_OK and f(pages=0, k_q=None) == mx.MX_OK and f(heads=0, k_q=None) == mx.MX_OK


@no_gpu
def test_attention_validation(mx):
    w = mx.lib.mx_attention_workspace
    assert w(1, 1, 4, 2, 64, 32) == 0                    # one piece needs none
    assert w(1, 1, 4, 2, 64, 100000) > 0
    assert w(0, 1, 4, 2, 64, 100000) == 0 and w(1, 0, 4, 2, 64, 100000) == 0 and w(1, 1, 0, 0, 64, 100000) == 0
    for bad in ((-1, 1, 4, 2, 64, 9), (1, -1, 4, 2, 64, 9), (1, 1, 4, 2, 64, -1), (1, 1, 3, 2, 64, 9), (1, 1, 4, 0, 64, 9),
                (1, 1, 4, 2, 80, 9), (40000, 1, 4, 2, 64, 9), (1, 1 << 20, 32, 2, 64, 9), (1, 1, 4, 2, 64, 1 << 31)):
        assert w(*bad) == -1, bad

    def f(q=FAKE, ld_q=256, table=FAKE, ld_table=2, lens=FAKE, B=3, Lq=1, heads_q=4, max_len=32, o=FAKE, ld_o=256,
          lse=FAKE, ws=None, size=0, **kc):
        return mx.lib.mx_attention(cache(mx, **kc), q, ld_q, table, ld_table, lens, B, Lq, heads_q, 0.125, max_len, o, ld_o,
                                   lse, ws, size, None)
    for want, bad in BAD_CACHES:
        assert f(**bad) == getattr(mx, want), bad
    for bad in (dict(q=None), dict(table=None), dict(lens=None), dict(o=None), dict(B=-1), dict(Lq=-1), dict(max_len=-1)):
        assert f(**bad) == mx.MX_ERR_ARG, bad
    for bad in (dict(heads_q=3), dict(ld_q=248), dict(ld_o=255), dict(max_len=33), dict(ld_table=1), dict(ld_table=-1)):
        assert f(**bad) == mx.MX_ERR_SHAPE, bad
    for bad in (dict(q=FAKE + 8), dict(ld_q=260), dict(o=FAKE + 1), dict(lse=FAKE + 2), dict(table=FAKE + 2),
                dict(lens=FAKE + 1)):
        assert f(**bad) == mx.MX_ERR_ALIGN, bad
    for bad in (dict(B=40000), dict(Lq=1 << 20), dict(max_len=1 << 31, ld_table=1 << 30)):
        assert f(**bad) == mx.MX_ERR_UNSUPPORTED, bad
    long = dict(max_len=100000, ld_table=10000)
    need = w(3, 1, 4, 2, 64, 100000)
    assert f(**long, size=need) == mx.MX_ERR_ARG                          # no workspace
    assert f(**long, ws=FAKE, size=need - 1) == mx.MX_ERR_SHAPE
    assert f(**long, ws=FAKE + 8, size=need) == mx.MX_ERR_ALIGN
    assert f(B=0, q=None) == mx.MX_OK and f(Lq=0, o=None) == mx.MX_OK
    assert f(heads_q=0, heads=0, k_q=None) == mx.MX_OK


def test_binding_refuses_cpu_tensors(mx):
    b = torch.zeros((4, 64), dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int64)
    c = mx.kv_cache(2, 1, 16, 64, device="cpu")
    for call in (lambda: mx.rmsnorm_quantize(b, b[0], mx.E4M3), lambda: mx.rmsnorm_backward(b, b, b[0], i.float()),
                 lambda: mx.gemv(b, b, b, mx.E2M1, 4, 4, 64), lambda: mx.gemv_bf16(b, b, b, mx.E2M1, 4, 4, 64),
                 lambda: mx.cache_write(b.view(4, 1, 64), b.view(4, 1, 64), i, c, mx.E4M3),
                 lambda: mx.attention(b.view(4, 1, 1, 64), c, mx.E4M3, i.view(4, 1).int(), i.int())):
        with pytest.raises(ValueError):
            call()
