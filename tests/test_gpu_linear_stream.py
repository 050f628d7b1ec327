"""The linear layer's steps on a stream that is handed over: what they allocate and free on
return is that stream's, so work of the current stream in between does not reach it."""
import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("normed", [False, True])
def test_steps_on_another_stream(normed):
    from microscaling_block_scaled_amd import linear
    T, H, O = 512, 512, 768
    g = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *n: torch.randn(n, device="cuda", generator=g).to(torch.bfloat16)
    x, res, w, wn, dy, dh = rand(T, H), rand(T, H), rand(O, H), rand(H), rand(T, O), rand(T, H)
    r = linear.Recipe(fmt=4, seed=9, hadamard_signs=0x5A5A0F0F)

    def step(stream, between):
        if normed:
            y, h, saved = linear.forward_normed(x, res, wn, w, r, stream=stream)
            between()
            return y, h, *linear.backward_normed(dy, dh, saved, r, stream=stream)
        y, saved = linear.forward(x, w, r, stream=stream)
        between()
        return y, *linear.backward(dy, saved, r, stream=stream)

    want = step(None, lambda: None)
    a = torch.randn((4096, 4096), device="cuda", generator=g)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    held = []

    def scribble():
        """Memory of every size that a step takes, in the current stream, which does not wait."""
        for n in (T * H, O * H, T * O):
            for part in (1, 2, 4, 16, 32, 64):
                held.extend(torch.full((n // part,), 255, dtype=torch.uint8, device="cuda") for _ in range(6))

    with torch.cuda.stream(s):
        for _ in range(6):  # the step's kernels begin when the current stream is through
            a = a @ a * 1e-2
    say("linear step on another stream", normed)
    got = step(s, scribble)
    scribble()
    s.synchronize()
    torch.cuda.synchronize()
    for p, q in zip(got, want):
        assert torch.equal(p, q)
