"""Pins of the layer operators' 64-bit references (CPU only): the gradient formula
against central differences, and attention against a softmax written out."""
import numpy as np
import pytest

import layer_ref as ref


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 5), (7, 40)])
def test_norm_gradient_against_differences(rows, cols):
    rng = np.random.default_rng(rows * 100 + cols)
    x, r, c, d = (rng.standard_normal((rows, cols)) for _ in range(4))
    w = 1 + 0.3 * rng.standard_normal(cols)
    eps, step = 1e-3, 1e-5
    rstd, _ = ref.norm(x + r, w, eps)
    dx, dw, _, _ = ref.norm_grad(c, x + r, w, rstd, d)
    # the third derivatives are of the size of the values over h^3: steps of 1e-5 leave about 1e-9
    for at in [(i, j) for i in range(rows) for j in range(min(cols, 6))]:
        e = np.zeros_like(x)
        e[at] = step
        for a, b in ((e, 0), (0, e)):  # of x and of the residual
            num = (ref.norm_loss(x + a, r + b, w, eps, c, d) - ref.norm_loss(x - a, r - b, w, eps, c, d)) / (2 * step)
            assert abs(num - dx[at]) < 1e-6 * (1 + abs(dx[at]))
    for j in range(min(cols, 6)):
        e = np.zeros(cols)
        e[j] = step
        num = (ref.norm_loss(x, r, w + e, eps, c, d) - ref.norm_loss(x, r, w - e, eps, c, d)) / (2 * step)
        assert abs(num - dw[j]) < 1e-6 * (1 + abs(dw[j]))


def test_attention_reference():
    rng = np.random.default_rng(5)
    q, k, v = rng.standard_normal((3, 4)), rng.standard_normal((6, 4)), rng.standard_normal((6, 2))
    o, lse, bo, bl = ref.attention(q, k, v, [0, 1, 6], 0.5)
    assert (o[0] == 0).all() and lse[0] == -np.inf
    assert np.allclose(o[1], v[0]) and np.isclose(lse[1], 0.5 * q[1] @ k[0])
    e = np.exp([0.5 * q[2] @ k[t] for t in range(6)])
    assert np.allclose(o[2], sum(e[t] * v[t] for t in range(6)) / e.sum())
    assert np.isclose(lse[2], np.log(e.sum()))
    assert (bo[1:] > 0).all() and (bl[1:] > 0).all() and (bo < 0.1).all()
