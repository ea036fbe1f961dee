"""The residual RMS norm at sizes past 32 bits: more rows than one grid of a wave
each can hold (2^32 threads), and more than 2^31 elements. The rows are
independent and element i of the dropout is a pure function of i, so a stretch of
rows anywhere has the bits of a small call on that stretch (whose results
test_gpu_norm.py holds to the oracle), its counter moved by the stretch's start.
A stretch is longer than the 1,024 rows up to which a wide row takes more threads,
which add its squares in another order."""
import pytest
import torch

import mixture_experts_layer_table_amd as mok
from gpu_support import DEV
from test_gpu_dropout import randn, rng_state

pytestmark = pytest.mark.gpu
EPS, P, SEED, OFF = 1e-6, 0.25, 91, 7
ROWS = 1032     # of a stretch


def fill(shape, seed):   # without the fp32 copy that randn makes
    g = torch.Generator(DEV).manual_seed(seed)
    return torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(generator=g)


def check_stretches(T, H, starts, mxfp8):
    x, res = fill((T, H), 1), fill((T, H), 2)
    w = (1.0 + 0.25 * randn((H,), 3).float()).to(torch.bfloat16)
    r = mok.add_rmsnorm(x, w, EPS, residual=res, p=P, rng=rng_state(SEED, OFF), mxfp8=mxfp8)
    assert bool((r["rstd"] > 0).all())
    for a in starts:
        s = slice(a, a + ROWS)
        want = mok.add_rmsnorm(x[s], w, EPS, residual=res[s], p=P, rng=rng_state(SEED, OFF + a * H // 4), mxfp8=mxfp8)
        for n in want:
            assert torch.equal(r[n][s], want[n]), (n, a)
    del r["y"]
    torch.cuda.empty_cache()
    g = mok.add_rmsnorm_backward(x, r["sum"], w, r["rstd"], dsum=res, p=P, rng=rng_state(SEED, OFF))
    for a in starts:
        s = slice(a, a + ROWS)
        want = mok.add_rmsnorm_backward(x[s], r["sum"][s], w, r["rstd"][s].clone(), dsum=res[s], p=P,
                                        rng=rng_state(SEED, OFF + a * H // 4))
        for n in ("dresidual", "dx"):
            assert torch.equal(g[n][s], want[n]), (n, a)


def test_more_rows_than_a_grid_holds():
    T, H = 2 ** 26 + 5, 8
    print(f"[norm] T={T} H={H}", flush=True)
    check_stretches(T, H, [0, 2 ** 25 - 4, 2 ** 25, 2 ** 26 - 1030, T - ROWS], False)


def test_more_elements_than_31_bits():
    T, H = 300001, 7168
    print(f"[norm] T={T} H={H}", flush=True)
    edge = 2 ** 31 // H
    check_stretches(T, H, [0, edge // 2 - 4, edge - 1028, edge - 700, T - ROWS], True)
