"""One and two rows of the feed-forward block, whose forward has kernels of its
own: block scales far apart, the loops past their first pass, and the largest
rows that take these kernels."""
import pytest
import torch

import mixture_experts_layer_table_amd as mok
from test_gpu_ffn import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 2, 5, 300])
@pytest.mark.parametrize("shift", [120, -90])
def test_down_scales_far_apart(T, shift):
    # 2^shift taken from the down weights' scales and given to a by way of h_u: the same products. At 2^120 a code
    # times a's scale alone, times a weight's code, passes fp32's range; more rows run on the matrix cores.
    print(f"[ffn few] down scales T={T} shift={shift}", flush=True)
    c = Case(T, 1024, 512, True, 85)
    q = c.keep
    (ge, gs), (ue, us), (de, ds) = q.fwd_gate, q.fwd_up, q.fwd_down
    ds = ds + 8
    for s, by in ((us, shift), (ds, -shift)):
        assert 0 < int(s.min()) + by and int(s.max()) + by < 255
    base, moved = (mok.weights_mxfp8((ge, gs), (ue, us + a), (de, ds + b), "fwd") for a, b in ((0, 0), (shift, -shift)))
    out, h = mok.ffn_forward(c.ws, c.rows, base, addend=c.add)
    out2, h2 = mok.ffn_forward(c.ws, c.rows, moved, addend=c.add)
    assert torch.isfinite(out).all() and torch.equal(h[:, :c.I], h2[:, :c.I])
    assert torch.equal(out, out2)
