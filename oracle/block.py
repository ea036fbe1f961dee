"""O6 — the operators around the routed experts, step by step in fp64 (test
infrastructure only): dropout from a counter-based generator, the residual's
addition with a root-mean-square norm, and the dense gated feed-forward block.

The pages describe the routed layer alone ("Mixture-of-Kittens (MoK)" project
summary, Functional API); these follow the plainest definitions:

  Philox4x32 with 10 rounds   Salmon et al., "Parallel Random Numbers: As Easy
                              as 1, 2, 3", SC 2011
  root-mean-square norm       y = s / sqrt(mean(s^2) + eps) * weight
  SwiGLU block                (silu(x W_gate) * (x W_up)) W_down
"""
from __future__ import annotations

import numpy as np

from . import mxfp8

_M32 = np.uint64(0xFFFFFFFF)


def philox4x32_10(counter, key):
    """counter: uint32 [..., 4]; key: two uint32. Returns uint32 [..., 4]."""
    c = [np.asarray(counter)[..., i].astype(np.uint64) for i in range(4)]
    k0, k1 = np.uint64(key[0]), np.uint64(key[1])
    for _ in range(10):
        p0, p1 = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ k0, p1 & _M32, (p0 >> np.uint64(32)) ^ c[3] ^ k1, p0 & _M32]
        k0, k1 = (k0 + np.uint64(0x9E3779B9)) & _M32, (k1 + np.uint64(0xBB67AE85)) & _M32
    return np.stack(c, axis=-1).astype(np.uint32)


def keep_mask(seed: int, offset: int, n: int, p: float) -> np.ndarray:
    """True for the kept elements 0..n-1: word i % 4 of block offset + i // 4 is at least floor(p * 2^32)."""
    blocks = (n + 3) // 4
    ctr = (np.arange(blocks, dtype=np.uint64) + np.uint64(offset % 2 ** 64))      # wraps at 2^64
    counter = np.zeros((blocks, 4), np.uint32)
    counter[:, 0], counter[:, 1] = ctr & _M32, ctr >> np.uint64(32)
    words = philox4x32_10(counter, (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF)).reshape(-1)[:n]
    return words.astype(np.int64) >= int(float(np.float32(p)) * 2.0 ** 32)


def dropout(x, keep, p):
    """x / (1 - p) where kept, 0 elsewhere (whatever x holds there)."""
    return np.where(keep, x / (1.0 - float(np.float32(p))), 0.0) if p > 0 else np.asarray(x, np.float64)


def rmsnorm(s, weight, eps):
    """(y, rstd) of rows s [T, H]."""
    rstd = 1.0 / np.sqrt(np.mean(s * s, axis=1) + eps)
    return s * rstd[:, None] * weight, rstd


def rmsnorm_backward(dy, s, weight, rstd, dsum=None):
    """(ds, dweight) for the gradient dy of y and dsum of s."""
    r = rstd[:, None]
    g = dy * weight
    ds = r * (g - s * r * r * np.mean(g * s, axis=1, keepdims=True))
    return ds if dsum is None else ds + dsum, np.sum(dy * s * r, axis=0)


def _sigmoid(z):
    return 1.0 / (1.0 + np.exp(-z))


def ffn(x, wg, wu, wd, addend=None, fq=None):
    """(out, h, a). fq: the fake quantizer of MXFP8 mode, applied along each product's contraction axis."""
    q = fq or (lambda v, axis: v)
    xq = q(x, 1)
    hg, hu = xq @ q(wg, 0), xq @ q(wu, 0)
    a = hg * _sigmoid(hg) * hu
    out = q(a, 1) @ q(wd, 0)
    return out if addend is None else out + addend, np.concatenate([hg, hu], axis=1), a


def ffn_backward(x, wg, wu, wd, h, dy, addend=None, fq=None):
    """dict(dx, dw_gate, dw_up, dw_down, dh, a) from the saved pre-activations h [T, 2I]."""
    q = fq or (lambda v, axis: v)
    I = wg.shape[1]
    hg, hu = h[:, :I], h[:, I:]
    s = _sigmoid(hg)
    a = hg * s * hu
    da = q(dy, 1) @ q(wd, 1).T
    dhg, dhu = da * hu * s * (1.0 + hg * (1.0 - s)), da * hg * s
    dx = q(dhg, 1) @ q(wg, 1).T + q(dhu, 1) @ q(wu, 1).T
    if addend is not None:
        dx = dx + addend
    return dict(dx=dx, dw_gate=x.T @ dhg, dw_up=x.T @ dhu, dw_down=a.T @ dy, dh=np.concatenate([dhg, dhu], 1), a=a)


def fake_quant(v, axis):
    return mxfp8.fake_quant(v, axis)
