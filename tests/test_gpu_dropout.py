"""Dropout with the residual's addition on the GPU against the fp64 oracle.

Tolerances, counting roundings (U: bf16 half step 2^-8, V: fp32 half step
2^-24, both relative): a kept value is one fused multiply-add of x, the fp32
scale (off by V) and the residual (one rounding, V of the result): at most
V |x scale| + V |result|, doubled to cover the second-order terms, then the
rounding to the output's type."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_table_amd as mok
from gpu_support import DEV, host_f64
from oracle import block as B

pytestmark = pytest.mark.gpu
U, V = 2.0 ** -8, 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def rng_state(seed, offset):
    return torch.from_numpy(np.array([seed % 2 ** 64, offset % 2 ** 64], np.uint64).view(np.int64)).to(DEV)


def randn(shape, seed, dtype=torch.bfloat16, scale=1.0):
    g = torch.Generator(DEV).manual_seed(seed)
    return (torch.randn(shape, device=DEV, generator=g) * scale).to(dtype)


def check(got, ref, magnitude, dtype):
    got = host_f64(got).reshape(-1)
    tol = 2 * V * (magnitude + np.abs(ref)) + (U if dtype == torch.bfloat16 else V) * np.abs(ref)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), int(np.argmax(bad)))


# lengths: below one chunk of 8, odd ones, around one workgroup's 8,192 elements, several workgroups
@pytest.mark.parametrize("n", [1, 3, 7, 8, 9, 4096, 8191, 8192, 8195, 100003])
@pytest.mark.parametrize("stream,residual", [("bf16", False), ("bf16", True), ("fp32", True)])
def test_dropout_matches_the_oracle(n, stream, residual):
    print(f"[dropout] n={n} {stream} residual={residual}", flush=True)
    p, seed, off = 0.3, 0x0123456789ABCDEF + n, 2 ** 33 + 11 * n
    x = randn((n,), n)
    res = randn((n,), n + 1, TYPES[stream], 3.0) if residual else None
    rng = rng_state(seed, off)
    keep = B.keep_mask(seed, off, n, p)
    branch = B.dropout(host_f64(x), keep, p)
    base = host_f64(res) if residual else np.zeros(n)
    out = mok.dropout(x, rng, p, residual=res)
    assert out.dtype == TYPES[stream]
    check(out, base + branch, np.abs(branch) + np.abs(base), out.dtype)
    dy = randn((n,), n + 2, TYPES[stream])
    dx = mok.dropout_backward(dy, rng, p)
    assert dx.dtype == torch.bfloat16
    grad = B.dropout(host_f64(dy), keep, p)
    check(dx, grad, np.abs(grad), torch.bfloat16)


def test_gradient_is_the_difference_quotient():
    # the operator is linear in x: differences of any size give its gradient up to roundings of the fp32 outputs
    n, p = 5000, 0.4
    rng = rng_state(5, 6)
    x, v = randn((n,), 1), randn((n,), 2)
    res = torch.zeros(n, device=DEV)
    hi = mok.dropout((x.float() + v.float()).to(torch.bfloat16), rng, p, residual=res)
    lo = mok.dropout(x, rng, p, residual=res)
    step = host_f64((x.float() + v.float()).to(torch.bfloat16)) - host_f64(x)
    one = mok.dropout_backward(torch.ones(n, device=DEV), rng, p)   # dx/dx per element
    slope = host_f64(one)
    diff = host_f64(hi) - host_f64(lo)
    tol = 4 * V * (np.abs(host_f64(hi)) + np.abs(host_f64(lo))) + U * np.abs(slope * step)
    assert (np.abs(diff - slope * step) <= tol).all()


def test_dropped_values_leave_nothing_behind():
    n, p, seed = 4099, 0.5, 77
    keep = torch.from_numpy(B.keep_mask(seed, 0, n, p)).to(DEV)
    res = randn((n,), 3)
    for poison in (float("nan"), float("inf"), -float("inf")):
        x = torch.where(keep, randn((n,), 4), torch.tensor(poison, dtype=torch.bfloat16, device=DEV))
        out = mok.dropout(x, rng_state(seed, 0), p, residual=res)
        assert torch.equal(out[~keep], res[~keep]) and torch.isfinite(out).all()
        dx = mok.dropout_backward(x, rng_state(seed, 0), p)
        assert (dx[~keep] == 0).all() and torch.isfinite(dx).all()


def test_zero_probability_needs_no_state():
    x, res = randn((1001,), 5), randn((1001,), 6)
    out = mok.dropout(x, None, 0.0, residual=res)
    assert torch.equal(out, (x.float() + res.float()).to(torch.bfloat16))
    assert torch.equal(mok.dropout_backward(x, None, 0.0), x)
    assert mok.dropout(x[:0], None, 0.0).numel() == 0


@pytest.mark.parametrize("offset", [2 ** 32 - 3, 2 ** 64 - 5])
def test_counter_carries_and_wraps(offset):
    n, p, seed = 64, 0.5, 2 ** 64 - 9
    out = mok.dropout(torch.ones(n, dtype=torch.bfloat16, device=DEV), rng_state(seed, offset), p)
    assert np.array_equal(host_f64(out) != 0, B.keep_mask(seed, offset, n, p))


def test_in_place_and_neighbours_untouched():
    n, p = 8197, 0.2
    rng = rng_state(9, 10)
    x, res = randn((n,), 7), randn((n,), 8)
    ref = mok.dropout(x, rng, p, residual=res)
    for over in ("residual", "x"):
        buf = torch.full((n + 64,), 5.0, dtype=torch.bfloat16, device=DEV)
        buf[:n] = res if over == "residual" else x
        a = buf[:n]
        mok.dropout(x if over == "residual" else a, rng, p, residual=a if over == "residual" else res, out=a)
        assert torch.equal(buf[:n], ref) and (buf[n:] == 5.0).all()
    a = res.clone()
    mok.dropout_backward(a, rng, p, dx=a)
    assert torch.equal(a, mok.dropout_backward(res, rng, p))


def test_far_elements_of_a_large_tensor():
    # 2^31 + 24 elements: byte offsets past 2^32; ones keep the mask visible
    n, p, seed, off = 2 ** 31 + 24, 0.25, 31, 7
    print("[dropout] 2^31 + 24 elements", flush=True)
    x = torch.ones(n, dtype=torch.bfloat16, device=DEV)
    out = mok.dropout(x, rng_state(seed, off), p)
    for a in (0, 2 ** 30, 2 ** 31 - 8, n - 4096):
        a -= a % 4
        m = min(4096, n - a)
        assert np.array_equal(host_f64(out[a:a + m]) != 0, B.keep_mask(seed, off + a // 4, m, p)), a


def test_graph_replays_follow_the_state():
    n, p = 10007, 0.3
    x, res = randn((n,), 11), randn((n,), 12)
    rng = rng_state(21, 0)
    out, dx = torch.empty_like(x), torch.empty_like(x)

    def step():
        mok.dropout(x, rng, p, residual=res, out=out)
        mok.dropout_backward(x, rng, p, dx=dx)
        rng[1] += (n + 3) // 4

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rng.copy_(rng_state(21, 100))
    for rep in range(3):
        at = rng_state(21, 100 + rep * ((n + 3) // 4))
        want, want_dx = mok.dropout(x, at, p, residual=res), mok.dropout_backward(x, at, p)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(dx, want_dx), rep


def test_other_stream():
    n, p = 50001, 0.3
    x, rng = randn((n,), 13), rng_state(3, 4)
    want = mok.dropout(x, rng, p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = mok.dropout(x, rng, p)
    s.synchronize()
    assert torch.equal(got, want)
