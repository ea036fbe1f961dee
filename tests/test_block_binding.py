"""What the binding refuses around the routed experts, case by case and for the
reason it states. All tensors are on the CPU: the check of an argument comes
before the one for a GPU, whose message would answer any other call."""
import pytest
import torch

import mixture_experts_layer_table_amd as mok

P, FAR = 1 << 20, 1 << 44     # 16-byte aligned addresses that nothing reads, apart from each other


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


@pytest.mark.parametrize("n", [2 ** 37 - 8191, 2 ** 37, 2 ** 39])
def test_dropout_past_one_grid_is_refused(n):
    # 8,192 elements a workgroup of 256 threads: a grid of 2^32 threads cannot be launched
    a = [P + i * FAR for i in range(4)]
    assert mok.mok_dropout(a[0], a[1], n, 0.5, a[2], mok.MOK_STREAM_BF16, a[3], None) == mok.MOK_ERROR_INVALID_VALUE
    assert mok.mok_dropout_backward(a[0], n, 0.5, a[2], mok.MOK_STREAM_BF16, a[3], None) == \
        mok.MOK_ERROR_INVALID_VALUE
