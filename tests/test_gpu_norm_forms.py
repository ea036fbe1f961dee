"""Forms of the residual RMS norm that a caller may choose: gradient buffers of
its own, and outputs left out through the C ABI. Which buffers a call gets never
changes what it computes, so every form is held to the bits of the full one."""
import pytest
import torch

import mixture_experts_layer_table_amd as mok
from gpu_support import DEV
from test_gpu_dropout import TYPES, randn, rng_state

pytestmark = pytest.mark.gpu
T, H, EPS = 37, 512, 1e-6


def backward_inputs(stream):
    s, dy = randn((T, H), 1, TYPES[stream], 2.0), randn((T, H), 2)
    w = (1.0 + 0.25 * randn((H,), 3).float()).to(torch.bfloat16)
    rstd = torch.rsqrt(s.double().square().mean(1) + EPS).float()
    return dy, s, w, rstd, randn((T, H), 4, TYPES[stream])


@pytest.mark.parametrize("stream,p", [("bf16", 0.0), ("bf16", 0.25), ("fp32", 0.0)])
def test_a_given_dx_is_written(stream, p):
    # a loop with static buffers reads its dx whatever p has become
    dy, s, w, rstd, dsum = backward_inputs(stream)
    rng = rng_state(5, 6) if p > 0 else None
    want = mok.add_rmsnorm_backward(dy, s, w, rstd, dsum=dsum, p=p, rng=rng)
    grads = dict(dresidual=torch.full_like(s, 7.0), dx=torch.full_like(dy, 7.0),
                 dweight=torch.full((H,), 7.0, device=DEV))
    got = mok.add_rmsnorm_backward(dy, s, w, rstd, dsum=dsum, p=p, rng=rng, grads=grads)
    for n in ("dresidual", "dx", "dweight"):
        assert got[n] is grads[n] and torch.equal(grads[n], want[n]), n


def test_the_returned_gradients_serve_as_buffers():
    # bf16 and p == 0: the dict holds one tensor under two names, and may come back as grads
    dy, s, w, rstd, dsum = backward_inputs("bf16")
    first = mok.add_rmsnorm_backward(dy, s, w, rstd, dsum=dsum)
    want = {n: t.clone() for n, t in first.items()}
    for t in first.values():
        t.zero_()
    again = mok.add_rmsnorm_backward(dy, s, w, rstd, dsum=dsum, grads=first)
    assert again["dx"].data_ptr() == again["dresidual"].data_ptr()
    for n in want:
        assert torch.equal(again[n], want[n]), n
