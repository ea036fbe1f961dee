"""What the binding refuses around the routed experts, case by case and for the
reason it states. All tensors are on the CPU: the check of an argument comes
before the one for a GPU, whose message would answer any other call."""
import pytest
import torch

import mixture_experts_layer_table_amd as mok


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _f32(*shape):
    return torch.zeros(shape)


@pytest.mark.parametrize("dx,message", [(_bf(4, 32), r"dx: shape \(4, 32\)"), (_f32(4, 64), "dx: dtype torch.float32"),
                                        (_bf(64, 4).T, "dx: must be contiguous")])
def test_norm_backward_checks_a_given_dx(dx, message):
    # bf16 stream and p == 0, where dx could also be left to dresidual
    grads = dict(dresidual=_bf(4, 64), dweight=_f32(64), dx=dx)
    with pytest.raises(ValueError, match=message):
        mok.add_rmsnorm_backward(_bf(4, 64), _bf(4, 64), _bf(64), _f32(4), grads=grads)
