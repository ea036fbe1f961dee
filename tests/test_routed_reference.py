"""tests/routed_reference.py against element-by-element loops and differences (CPU)."""
import math

import numpy as np
import pytest
import torch

import routed_reference as R


def _g(seed):
    return torch.Generator().manual_seed(seed)


@pytest.mark.parametrize("T,k,E,align", [(0, 2, 3, 4), (1, 1, 1, 1), (7, 3, 5, 1), (9, 2, 4, 8), (30, 4, 6, 16)])
def test_sort_is_a_stable_sort_with_padding(T, k, E, align):
    ids = torch.randint(-1, E + 1, (T, k), generator=_g(T)).int()   # -1 and E: no expert here
    s = R.sort(ids, E, align)
    flat, off, rows = ids.reshape(-1).tolist(), s["offsets"].tolist(), s["row_slots"].tolist()
    assert off[0] == 0 and all(b % align == 0 for b in off) and off == sorted(off) and off[-1] <= len(rows)
    for e in range(E):
        mine = [f for f, v in enumerate(flat) if v == e]
        run = rows[off[e]:off[e + 1]]
        assert run[:len(mine)] == mine and all(r == -1 for r in run[len(mine):]) and len(run) - len(mine) < align
    assert all(r == -1 for r in rows[off[-1]:])
    for f, r in enumerate(s["slots"].reshape(-1).tolist()):
        assert (r == -1) == (not 0 <= flat[f] < E) and (r == -1 or rows[r] == f)


def test_rows_and_back_by_loops():
    ids = torch.tensor([[0, 2], [2, 2], [-1, 0], [9, -5]]).int()
    s = R.sort(ids, 3, 2)
    x = torch.randn(4, 8, generator=_g(1), dtype=torch.float64)
    rows = R.permute(x, s)
    for t in range(4):
        for j in range(2):
            r = int(s["slots"][t, j])
            if r >= 0:
                assert torch.equal(rows[r], x[t])
    assert float(rows.abs().sum()) == pytest.approx(float(sum(x[t].abs().sum() for t in (0, 0, 1, 1, 2))))
    w = torch.rand(4, 2, generator=_g(2), dtype=torch.float64)
    y = torch.randn(rows.shape, generator=_g(3), dtype=torch.float64)
    add = torch.randn(4, 8, generator=_g(4), dtype=torch.float64)
    out, _ = R.unpermute(y, s, w, add)
    for t in range(4):
        want = add[t].clone()
        for j in range(2):
            r = int(s["slots"][t, j])
            want += w[t, j] * y[r] if r >= 0 else 0.0
        assert torch.allclose(out[t], want, rtol=0, atol=1e-14)
    assert torch.equal(out[3], add[3])


def test_gradients_by_differences():
    ids = torch.tensor([[0, 1], [1, 2], [-1, 0]]).int()
    s = R.sort(ids, 3, 4)
    n, H = s["row_slots"].numel(), 6
    y, w = torch.randn(n, H, generator=_g(5)).double(), torch.rand(3, 2, generator=_g(6)).double()
    dout = torch.randn(3, H, generator=_g(7)).double()
    dy, dw, _ = R.unpermute_backward(dout, y, s, w)
    loss = lambda y, w: float((R.unpermute(y, s, w)[0] * dout).sum())   # noqa: E731
    h = 1e-6
    for at in range(y.numel()):
        d = torch.zeros(y.numel(), dtype=torch.float64)
        d[at] = h
        d = d.view(n, H)
        assert (loss(y + d, w) - loss(y - d, w)) / (2 * h) == pytest.approx(float(dy.view(-1)[at]), abs=1e-8)
    for at in range(6):
        d = torch.zeros(6, dtype=torch.float64)
        d[at] = h
        d = d.view(3, 2)
        assert (loss(y, w + d) - loss(y, w - d)) / (2 * h) == pytest.approx(float(dw.view(-1)[at]), abs=1e-8)
    # the sort's gradient is the unweighted sum back
    x = torch.randn(3, H, generator=_g(8)).double()
    dx, _ = R.unpermute(y, s)
    v = torch.randn(3, H, generator=_g(9)).double()
    moved = (R.permute(x + h * v, s) - R.permute(x - h * v, s)) / (2 * h)
    real = s["row_slots"] >= 0
    assert float((moved[real] * y[real]).sum()) == pytest.approx(float((v * dx).sum()), rel=1e-8)
    hh, da = torch.randn(4, 10, generator=_g(10)).double(), torch.randn(4, 5, generator=_g(11)).double()
    dh = R.glu_backward(da, hh)
    for at in range(hh.numel()):
        d = torch.zeros(hh.numel(), dtype=torch.float64)
        d[at] = h
        d = d.view(4, 10)
        num = float(((R.glu(hh + d) - R.glu(hh - d)) * da).sum()) / (2 * h)
        assert num == pytest.approx(float(dh.view(-1)[at]), abs=1e-7)


def test_blocks_by_loops():
    v = torch.randn(2, 131, 272, generator=_g(12)).double()
    v[0, 3] = 0.0
    v[1, 5, :128] *= 1e-30
    for tile in (False, True):
        s, u = R.scales(v, tile)
        assert s.shape == ((2, 2, 3) if tile else (2, 3, 131))
        for b, r, k in ((0, 0, 0), (0, 3, 200), (1, 5, 17), (1, 130, 271), (0, 127, 128)):
            kb = slice(k // 128 * 128, k // 128 * 128 + 128)
            rb = slice(r // 128 * 128, r // 128 * 128 + 128) if tile else slice(r, r + 1)
            m = max(float(v[b, rb, kb].abs().max()), 2.0 ** -52)
            got = float(s[b, r // 128, k // 128] if tile else s[b, k // 128, r])
            assert got == pytest.approx(m / 448, rel=1e-15)
            assert float(u[b, r, k]) == pytest.approx(float(v[b, r, k]) * 448 / m, rel=1e-14, abs=1e-300)


def test_code_values_and_spacing():
    el = torch.arange(256, dtype=torch.uint8)
    got = R.codes(el).numpy()
    for c in range(256):
        e, m, sign = c >> 3 & 15, c & 7, -1.0 if c > 127 else 1.0
        if c & 127 == 127:
            assert math.isnan(got[c])
            continue
        assert got[c] == sign * (m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    pos = np.sort(got[:127])
    mid = torch.tensor((pos[1:] + pos[:-1]) / 2)
    assert np.allclose(R.half_step(mid).numpy() * 2, pos[1:] - pos[:-1], rtol=1e-12)


def test_products_by_loops():
    a, b = torch.randn(7, 20, generator=_g(13)).double(), torch.randn(2, 5, 20, generator=_g(14)).double()
    out, mag = R.matmul(a, b, torch.tensor([1, 4, 6]).int())
    assert torch.isnan(out[0]).all() and torch.isnan(out[6]).all()
    for m, e in ((1, 0), (3, 0), (4, 1), (5, 1)):
        for n in range(5):
            assert float(out[m, n]) == pytest.approx(sum(float(a[m, k] * b[e, n, k]) for k in range(20)))
            assert float(mag[m, n]) == pytest.approx(sum(abs(float(a[m, k] * b[e, n, k])) for k in range(20)))
    d, x = torch.randn(3, 9, generator=_g(15)).double(), torch.randn(4, 9, generator=_g(16)).double()
    add = torch.randn(2, 3, 4, generator=_g(17)).double()
    out, _ = R.wgrad(d, x, torch.tensor([0, 0, 9]).int(), add)
    assert torch.equal(out[0], add[0])
    assert float(out[1, 2, 3]) == pytest.approx(float(add[1, 2, 3] + (d[2] * x[3]).sum()))
