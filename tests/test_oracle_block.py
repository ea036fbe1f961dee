"""Pins of the block oracle (oracle/block.py): published generator outputs,
closed forms, finite differences, and torch's own autograd."""
import numpy as np
import pytest
import torch

from oracle import block as B


def _rel(a, b):
    return float(np.linalg.norm(a - b) / max(np.linalg.norm(b), 1e-300))


# known answers of Philox4x32-10 that the generator's authors publish with it
@pytest.mark.parametrize("counter,key,words", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_philox_known_answers(counter, key, words):
    assert tuple(int(w) for w in B.philox4x32_10(np.array(counter, np.uint32), key)) == words


def test_keep_mask_counts_words_in_order_and_wraps():
    whole = B.keep_mask(7, 100, 64, 0.3)
    assert np.array_equal(B.keep_mask(7, 101, 60, 0.3), whole[4:])       # one block further: 4 elements
    assert np.array_equal(B.keep_mask(7, 100, 13, 0.3), whole[:13])      # a length that is no multiple of 4
    wrapped = B.keep_mask(7, 2 ** 64 - 1, 8, 0.3)
    assert np.array_equal(wrapped[4:], B.keep_mask(7, 0, 4, 0.3))
    n = 1 << 16
    share = B.keep_mask(12345678901234567, 5, n, 0.3).mean()
    assert abs(share - 0.7) < 5 * np.sqrt(0.21 / n)                      # 5 standard deviations
    assert B.keep_mask(1, 2, 999, 0.0).all()


def test_dropout_ignores_what_it_drops():
    keep = np.array([True, False, True, False])
    x = np.array([1.0, np.nan, -2.0, np.inf])
    assert np.array_equal(B.dropout(x, keep, 0.5), [2.0, 0.0, -4.0, 0.0])


def test_rmsnorm_closed_form_and_gradient():
    rng = np.random.default_rng(1)
    s, w, dy = rng.standard_normal((5, 48)), rng.standard_normal(48), rng.standard_normal((5, 48))
    y, r = B.rmsnorm(s, w, 0.0)
    assert np.allclose(np.sqrt(np.mean((y / w) ** 2, axis=1)), 1.0)
    assert np.allclose(r, np.sqrt(48) / np.linalg.norm(s, axis=1))
    ds_in = rng.standard_normal((5, 48))
    y, r = B.rmsnorm(s, w, 1e-3)
    ds, dw = B.rmsnorm_backward(dy, s, w, r, ds_in)
    st, wt = torch.tensor(s, requires_grad=True), torch.tensor(w, requires_grad=True)
    yt = st * torch.rsqrt(st.square().mean(1, keepdim=True) + 1e-3) * wt
    ((yt * torch.tensor(dy)).sum() + (st * torch.tensor(ds_in)).sum()).backward()
    assert _rel(ds, st.grad.numpy()) < 1e-12 and _rel(dw, wt.grad.numpy()) < 1e-12


def test_ffn_gradients_against_differences_and_autograd():
    rng = np.random.default_rng(2)
    T, H, I = 3, 6, 5
    x, dy, add = rng.standard_normal((T, H)), rng.standard_normal((T, H)), rng.standard_normal((T, H))
    wg, wu, wd = rng.standard_normal((H, I)), rng.standard_normal((H, I)), rng.standard_normal((I, H))
    out, h, _ = B.ffn(x, wg, wu, wd, add)
    g = B.ffn_backward(x, wg, wu, wd, h, dy)
    ts = [torch.tensor(v, requires_grad=True) for v in (x, wg, wu, wd)]
    ot = (torch.nn.functional.silu(ts[0] @ ts[1]) * (ts[0] @ ts[2])) @ ts[3]
    assert _rel(out, ot.detach().numpy() + add) < 1e-12
    (ot * torch.tensor(dy)).sum().backward()
    for name, t in zip(("dx", "dw_gate", "dw_up", "dw_down"), ts):
        assert _rel(g[name], t.grad.numpy()) < 1e-12, name
    v = rng.standard_normal(x.shape)
    eps = 1e-6
    f = lambda z: float(np.sum(B.ffn(z, wg, wu, wd)[0] * dy))  # noqa: E731
    assert abs((f(x + eps * v) - f(x - eps * v)) / (2 * eps) - np.sum(g["dx"] * v)) < 1e-7
    assert np.array_equal(B.ffn_backward(x, wg, wu, wd, h, dy, add)["dx"], g["dx"] + add)


def test_ffn_fake_quant_is_lossless_on_representable_values():
    # values E4M3 holds under a block's scale: fake quantization changes nothing
    rng = np.random.default_rng(3)
    T, H, I = 4, 64, 32
    pick = lambda *sh: rng.choice([-1.0, -0.5, 0.5, 1.0], sh)  # noqa: E731
    x, wg, wu = pick(T, H), pick(H, I), pick(H, I)
    assert np.array_equal(B.ffn(x, wg, wu, pick(I, H), fq=B.fake_quant)[1], B.ffn(x, wg, wu, pick(I, H))[1])
