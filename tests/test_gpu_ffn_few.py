"""One and two rows of the feed-forward block, whose forward has kernels of its
own: block scales far apart, the loops past their first pass, and the largest
rows that take these kernels."""
import pytest
import torch

import block_reference as R
import mixture_experts_layer_table_amd as mok
from test_gpu_dropout import U, V
from test_gpu_ffn import TOL_MX, Case
from test_gpu_ffn_tiles import operands, rel, rel_rows, within

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


# Passes: more than 2,048 values of a (the second pass of the loops that make it), more than 2,048 rows of W_down, more than
# 1,024 rows of W_gate in one run, more than 7,168 columns in MXFP8. Limits: the widest rows that come here
PASSES_BF16 = [(2, 4096, 2048), (2, 1088, 2112), (1, 128, 4160), (1, 17472, 128)]
PASSES_MX = [(2, 7168, 2048), (2, 1152, 1152), (1, 8320, 128), (2, 7296, 2176)]
LIMITS_BF16 = [(1, 64, 15360), (2, 64, 7680), (1, 32768, 64), (2, 32768, 256)]
LIMITS_MX = [(1, 128, 15360), (2, 128, 7680), (1, 32768, 128), (2, 32768, 384)]


@pytest.mark.parametrize("T,H,I", PASSES_BF16 + LIMITS_BF16)
@pytest.mark.parametrize("addend", [True, False])
def test_bf16_matches_the_reference(T, H, I, addend):
    # a stays in fp32 here: only its evaluation is off (2^-18), and the sums
    print(f"[ffn few] bf16 T={T} H={H} I={I} addend={addend}", flush=True)
    c = Case(T, H, I, False, T + H + I, addend)
    o, add = operands(c), c.add.double() if addend else None
    out, h = c.forward()
    ref, rh, ra = R.forward(**o, addend=add)
    h_err = (H + 40) * V * (o["x"].abs() @ torch.cat([o["wg"].abs(), o["wu"].abs()], 1))
    within(h, rh, h_err + U * rh.abs() * 1.01, "h")
    a_err = 1.1 * h_err[:, :I] * rh[:, I:].abs() + rh[:, :I].abs() * h_err[:, I:] + 2.0 ** -18 * ra.abs()
    tol = (ra.abs() * (I + 40) * V + a_err) @ o["wd"].abs()
    within(out, ref, 1.01 * tol + U * ref.abs() * 1.01 + (2 * V * add.abs() if addend else 0), "out")
    assert torch.equal(mok.ffn_forward(c.ws, c.rows, c.wf, addend=c.add, save_h=False)[0], out)


@pytest.mark.parametrize("T,H,I", PASSES_MX + LIMITS_MX)
@pytest.mark.parametrize("addend", [True, False])
def test_mxfp8_matches_the_reference(T, H, I, addend):
    print(f"[ffn few] mxfp8 T={T} H={H} I={I} addend={addend}", flush=True)
    c = Case(T, H, I, True, T + H + I, addend)
    out, h = c.forward()
    ref, rh, _ = R.forward(**operands(c), addend=c.add.double() if addend else None, fq=R.fake_quant)
    assert rel_rows(out, ref) < 4 * TOL_MX and rel_rows(h, rh) < 4 * TOL_MX
    assert rel(out, ref) < TOL_MX and rel(h, rh) < TOL_MX
    assert torch.equal(mok.ffn_forward(c.ws, c.rows, c.wf, addend=c.add, save_h=False)[0], out)
