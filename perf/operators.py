"""The operators around the routed experts, case by case: dropout of a branch
into the residual stream, the residual's addition with the RMS norm (BF16 and
MXFP8 rows out), and the gated feed-forward block (the shared expert).

``run`` computes a case in its plain form (elementary torch operations in 32
bits, one rounding at the end) or, with ``own`` set, through the library's
entry points. ``exact`` evaluates the definitions in 64 bits.

Sizes are those of the repository's own configurations: hidden sizes 7,168,
4,096 and 128 with expert widths 2,048, 1,024 and 64, 2,048 tokens a GPU and
16,384 received rows, and single tokens as a decoder calls them.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"
M32 = 0xFFFFFFFF


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # the whole received batch of one GPU, the branch dropped into a bf16 residual stream
        dict(name="dropout_16384x7168", op="dropout", T=16384, H=7168, stream="bf16", residual=True, p=0.1),
        # gradient of the same call on an odd batch with the residual stream kept in fp32
        dict(name="dropout_bwd_2047x4096", op="dropout_bwd", T=2047, H=4096, stream="fp32", residual=True, p=0.25),
        # one decoded token: latency of the call
        dict(name="norm_1x7168", op="norm", T=1, H=7168, stream="bf16", residual=True, p=0.0, y=True, mx=False),
        # 2,048 tokens a GPU, fp32 residual stream, rows out in both formats for an MXFP8 layer
        dict(name="norm_2048x7168_mx", op="norm", T=2048, H=7168, stream="fp32", residual=True, p=0.0, y=True, mx=True),
        # the largest training batch with dropout on the branch, both formats
        dict(name="norm_16384x7168_drop_mx", op="norm", T=16384, H=7168, stream="bf16", residual=True, p=0.1, y=True,
             mx=True),
        # a ragged batch's backward, fp32 stream, dropout on the branch
        dict(name="norm_bwd_777x4096_drop", op="norm_bwd", T=777, H=4096, stream="fp32", dsum=True, p=0.1),
        # the largest batch's backward, bf16 stream
        dict(name="norm_bwd_16384x7168", op="norm_bwd", T=16384, H=7168, stream="bf16", dsum=True, p=0.0),
        # one decoded token through the shared expert, added to the routed output
        dict(name="ffn_1x7168x2048", op="ffn", T=1, H=7168, I=2048, mode="bf16", addend=True, save=False),
        # 2,048 tokens a GPU in MXFP8, saving for the backward
        dict(name="ffn_2048x7168x2048_mx", op="ffn", T=2048, H=7168, I=2048, mode="mxfp8", addend=True, save=True),
        # the largest training batch, BF16
        dict(name="ffn_16384x7168x2048", op="ffn", T=16384, H=7168, I=2048, mode="bf16", addend=False, save=True),
        # a ragged batch's backward at the streaming layer's sizes, BF16
        dict(name="ffn_bwd_1001x4096x1024", op="ffn_bwd", T=1001, H=4096, I=1024, mode="bf16", addend=True),
        # the largest backward, MXFP8 (weight gradients in BF16)
        dict(name="ffn_bwd_16384x7168x2048_mx", op="ffn_bwd", T=16384, H=7168, I=2048, mode="mxfp8", addend=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dropout", "dropout_bwd", "norm", "norm_bwd", "ffn", "ffn_bwd"])
    T = _log(rng, 1, 16384)
    stream = rng.choice(["bf16", "fp32"])
    if op in ("dropout", "dropout_bwd"):
        return dict(op=op, T=T, H=_log(rng, 65, 7168), stream=stream, residual=stream == "fp32" or rng.random() < 0.7,
                    p=round(rng.uniform(0.02, 0.6), 3))
    if op == "norm":
        y = rng.random() < 0.8
        return dict(op=op, T=T, H=32 * _log(rng, 2, 224), stream=stream, residual=rng.random() < 0.8,
                    p=rng.choice([0.0, round(rng.uniform(0.02, 0.5), 3)]), y=y, mx=not y or rng.random() < 0.5)
    if op == "norm_bwd":
        return dict(op=op, T=T, H=8 * _log(rng, 8, 896), stream=stream, dsum=rng.random() < 0.8,
                    p=rng.choice([0.0, round(rng.uniform(0.02, 0.5), 3)]))
    mode = rng.choice(["bf16", "mxfp8"])
    q = 64 if mode == "bf16" else 128
    H, I = q * _log(rng, 128 // q, 7168 // q), q * _log(rng, 128 // q, 2048 // q)
    if op == "ffn":
        return dict(op=op, T=T, H=H, I=I, mode=mode, addend=rng.random() < 0.5, save=rng.random() < 0.6)
    return dict(op=op, T=T, H=H, I=I, mode=mode, addend=rng.random() < 0.5)


def _st(case):
    return 4 if case["stream"] == "fp32" else 2


def work(case):
    T, H = case["T"], case["H"]
    n, op = T * H, case["op"]
    if op == "dropout":
        return dict(bytes=2 * n + _st(case) * n * (2 if case["residual"] else 1), flops=2 * n)
    if op == "dropout_bwd":
        return dict(bytes=(_st(case) if case["residual"] else 2) * n + 2 * n, flops=n)
    if op == "norm":
        b = 2 * n + _st(case) * n * (2 if case["residual"] else 1) + 2 * H + 4 * T
        b += (2 * n if case["y"] else 0) + (n + n // 32 if case["mx"] else 0)
        return dict(bytes=b, flops=6 * n)
    if op == "norm_bwd":
        s = _st(case)
        b = s * n + 2 * n + (s * n if case["dsum"] else 0) + s * n + 6 * H + 4 * T
        b += 2 * n if (case["p"] > 0 or s == 4) else 0
        return dict(bytes=b, flops=12 * n)
    I, mx = case["I"], case["mode"] == "mxfp8"
    wb = 3 * H * I * 33 // 32 if mx else 6 * H * I
    if op == "ffn":
        b = wb + (n + n // 32 if mx else 2 * n) + 2 * n + (2 * n if case["addend"] else 0)
        return dict(bytes=b + (4 * T * I if case["save"] else 0), flops=6 * n * I)
    b = wb + 2 * n + 4 * T * I + 2 * n + 2 * n + (2 * n if case["addend"] else 0) + 6 * H * I
    return dict(bytes=b, flops=12 * n * I)


# ----------------------------------------------------------------------------- inputs

def _randn(g, shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(shape, device=DEV, generator=g) * scale).to(dtype)


def _stream(case):
    return torch.float32 if case["stream"] == "fp32" else torch.bfloat16


def prepare(case, seed):
    g = torch.Generator(DEV).manual_seed(1_000_003 * (seed + 1) + 17)
    T, H, op = case["T"], case["H"], case["op"]
    s = dict(case)
    if op in ("dropout", "dropout_bwd", "norm", "norm_bwd"):
        # seed and offset of the generator, as a training loop holds them on the device
        s["rng"] = torch.randint(0, 1 << 62, (2,), device=DEV, generator=g)
    if op == "dropout":
        s["x"] = _randn(g, (T, H))
        s["residual"] = _randn(g, (T, H), _stream(case), 3.0) if case["residual"] else None
    elif op == "dropout_bwd":
        s["dy"] = _randn(g, (T, H), _stream(case) if case["residual"] else torch.bfloat16)
    elif op == "norm":
        s["x"] = _randn(g, (T, H))
        s["residual"] = _randn(g, (T, H), _stream(case), 3.0) if case["residual"] else None
        s["weight"] = (1.0 + 0.2 * torch.randn(H, device=DEV, generator=g)).to(torch.bfloat16)
        s["eps"] = 1e-6
    elif op == "norm_bwd":
        # what the forward left: the stream rows and their 1 / rms
        s["sum"] = _randn(g, (T, H), _stream(case), 3.0)
        s["rstd"] = torch.rsqrt(s["sum"].double().square().mean(1) + 1e-6).float()
        s["weight"] = (1.0 + 0.2 * torch.randn(H, device=DEV, generator=g)).to(torch.bfloat16)
        s["dy"] = _randn(g, (T, H))
        s["dsum"] = _randn(g, (T, H), _stream(case)) if case["dsum"] else None
    else:
        I, mx = case["I"], case["mode"] == "mxfp8"
        wg, wu = _randn(g, (H, I), scale=H ** -0.5), _randn(g, (H, I), scale=H ** -0.5)
        wd = _randn(g, (I, H), scale=I ** -0.5)
        x = _randn(g, (T, H))
        fwd = op == "ffn"
        if mx:   # the weights as an MXFP8 program keeps them: quantized along each product's contraction axis
            w = [_mx_codes(a) for a in ((wg.T, wu.T, wd.T) if fwd else (wg, wu, wd))]
        else:
            w = [wg, wu, wd]
        s["w"] = w
        s["x"] = _mx_codes(x) if mx and fwd else x
        s["addend"] = _randn(g, (T, H)) if case["addend"] else None
        if not fwd:
            s["dy"] = _randn(g, (T, H))
            s["h"] = (x.float() @ torch.cat([wg, wu], 1).float()).to(torch.bfloat16)   # what the forward left
        if own:   # the handles that such a program keeps: the workspace, and the weights' struct
            import mixture_experts_layer_table_amd as mok
            prec = mok.MOK_MXFP8 if mx else mok.MOK_BF16
            s["ws"] = mok.get_ffn_workspace(prec, device="cuda:0", num_tokens=T, hidden_size=H, intermediate_size=I)
            s["weights"] = mok.weights_mxfp8(*w, "fwd" if fwd else "bwd") if mx else mok.weights_bf16(*w)
    return s


# ----------------------------------------------------------------------------- plain forms (32 bits)

def _mx_codes(v):
    """MXFP8 elements and scales of v [rows, K] along K, 32 values a block."""
    v = v.contiguous().float()
    b = v.view(v.shape[0], -1, 32)
    amax = b.abs().amax(2)
    _, ex = torch.frexp(amax)
    e = torch.where(amax == 0, torch.zeros_like(ex), (ex - 9).clamp(-127, 127))
    q = torch.ldexp(b, -e.unsqueeze(2)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(v.shape), (e + 127).to(torch.uint8)


def _mx_typed(elems, scales):
    """The bytes as the values they stand for (views)."""
    return dict(elems=elems.view(torch.float8_e4m3fn), scales=scales.view(torch.float8_e8m0fnu))


def _mx_values(codes):
    elems, scales = codes
    v = elems.view(torch.float8_e4m3fn).float().view(elems.shape[0], -1, 32)
    return torch.ldexp(v, scales.int().unsqueeze(2) - 127).view(elems.shape)


def _keep(rng, n, p):
    """Kept elements 0..n-1: word i % 4 of Philox4x32-10 at counter offset + i // 4, at least floor(p 2^32)."""
    seed, offset = rng[0], rng[1]
    c = offset + torch.arange((n + 3) // 4, device=rng.device)
    x0, x1 = c & M32, (c >> 32) & M32
    x2, x3 = torch.zeros_like(c), torch.zeros_like(c)
    k0, k1 = seed & M32, (seed >> 32) & M32
    for _ in range(10):
        p0, p1 = x0 * 0xD2511F53, x2 * 0xCD9E8D57   # 64-bit products, read as bit patterns
        x0, x1, x2, x3 = ((p1 >> 32) & M32) ^ x1 ^ k0, p1 & M32, ((p0 >> 32) & M32) ^ x3 ^ k1, p0 & M32
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    words = torch.stack([x0, x1, x2, x3], 1).view(-1)[:n]
    return words >= int(float(np.float32(p)) * 2.0 ** 32)


def _drop(x, rng, p):
    if p == 0:
        return x.float()
    scale = 1.0 / (1.0 - float(np.float32(p)))
    return torch.where(_keep(rng, x.numel(), p).view(x.shape), x.float() * scale, 0.0)


def _plain_dropout(s):
    y = _drop(s["x"], s["rng"], s["p"])
    return y.to(torch.bfloat16) if s["residual"] is None else (s["residual"].float() + y).to(s["residual"].dtype)


def _plain_norm(s):
    v = _drop(s["x"], s["rng"], s["p"])
    if s["residual"] is not None:
        v = s["residual"].float() + v
    total = v.to(_stream(s))   # the norm is of the sum before this rounding
    rstd = 1.0 / torch.sqrt((v * v).mean(1) + s["eps"])
    y = v * rstd[:, None] * s["weight"].float()
    out = dict(sum=total, rstd=rstd)
    if s["y"]:
        out["y"] = y.to(torch.bfloat16)
    if s["mx"]:
        out["mx"] = _mx_typed(*_mx_codes(y))
    return out


def _plain_norm_bwd(s):
    v, r, dy = s["sum"].float(), s["rstd"][:, None], s["dy"].float()
    g = dy * s["weight"].float()
    ds = r * (g - v * ((g * v).mean(1, keepdim=True) * r * r))
    if s["dsum"] is not None:
        ds = ds + s["dsum"].float()
    dweight = (dy * v * r).sum(0)
    dresidual = ds.to(s["sum"].dtype)
    return dict(dresidual=dresidual, dx=_drop(ds, s["rng"], s["p"]).to(torch.bfloat16), dweight=dweight)


def _plain_ffn(s):
    mx = s["mode"] == "mxfp8"
    if mx:
        x = _mx_values(s["x"])
        wg, wu, wd = (_mx_values(w).T for w in s["w"])
    else:
        x = s["x"].float()
        wg, wu, wd = (w.float() for w in s["w"])
    hg, hu = x @ wg, x @ wu
    a = hg / (1.0 + torch.exp(-hg)) * hu
    if mx:
        a = _mx_values(_mx_codes(a))
    out = a @ wd
    if s["addend"] is not None:
        out = out + s["addend"].float()
    out = dict(out=out.to(torch.bfloat16))
    if s["save"]:
        out["h"] = torch.cat([hg, hu], 1).to(torch.bfloat16)
    return out


def _plain_ffn_bwd(s):
    mx, I = s["mode"] == "mxfp8", s["I"]
    x, dy = s["x"].float(), s["dy"].float()
    wg, wu, wd = (_mx_values(w) if mx else w.float() for w in s["w"])
    hg, hu = s["h"][:, :I].float(), s["h"][:, I:].float()
    sg = 1.0 / (1.0 + torch.exp(-hg))
    a = hg * sg * hu
    G = (_mx_values(_mx_codes(dy)) if mx else dy) @ wd.T
    dhu = G * hg * sg
    dhg = G * hu * sg * (1.0 + hg * (1.0 - sg))
    qg, qu = (_mx_values(_mx_codes(dhg)), _mx_values(_mx_codes(dhu))) if mx else (dhg, dhu)
    dx = qg @ wg.T + qu @ wu.T
    if s["addend"] is not None:
        dx = dx + s["addend"].float()
    return {k: v.to(torch.bfloat16) for k, v in dict(dx=dx, dw_gate=x.T @ dhg, dw_up=x.T @ dhu, dw_down=a.T @ dy).items()}


_PLAIN = dict(dropout=_plain_dropout, dropout_bwd=lambda s: _drop(s["dy"], s["rng"], s["p"]).to(torch.bfloat16),
              norm=_plain_norm, norm_bwd=_plain_norm_bwd, ffn=_plain_ffn, ffn_bwd=_plain_ffn_bwd)


# ----------------------------------------------------------------------------- the library's calls

def _own(s):
    import mixture_experts_layer_table_amd as mok
    op = s["op"]
    if op == "dropout":
        return mok.dropout(s["x"], s["rng"], s["p"], residual=s["residual"])
    if op == "dropout_bwd":
        return mok.dropout_backward(s["dy"], s["rng"], s["p"])
    if op == "norm":
        r = mok.add_rmsnorm(s["x"], s["weight"], s["eps"], residual=s["residual"], p=s["p"], rng=s["rng"],
                            stream_dtype=_stream(s), y=s["y"], mxfp8=s["mx"])
        out = dict(sum=r["sum"], rstd=r["rstd"])
        if s["y"]:
            out["y"] = r["y"]
        if s["mx"]:
            out["mx"] = _mx_typed(r["y_elems"], r["y_scales"])
        return out
    if op == "norm_bwd":
        return mok.add_rmsnorm_backward(s["dy"], s["sum"], s["weight"], s["rstd"], dsum=s["dsum"], p=s["p"],
                                        rng=s["rng"])
    if op == "ffn":
        out, h = mok.ffn_forward(s["ws"], s["x"], s["weights"], addend=s["addend"], save_h=s["save"])
        return dict(out=out, h=h) if s["save"] else dict(out=out)
    return mok.ffn_backward(s["ws"], s["x"], s["weights"], s["h"], s["dy"], addend=s["addend"])


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ----------------------------------------------------------------------------- the definitions in 64 bits

def _x_words(rng, n):
    """Philox4x32-10 words of elements 0..n-1, its 32-bit products put together from 16-bit halves."""
    seed, off = (int(v) & (2 ** 64 - 1) for v in rng.tolist())
    i = torch.arange((n + 3) // 4, device=DEV)
    lo = i + (off & M32)
    ctr = [lo & M32, ((lo >> 32) + (off >> 32)) & M32, torch.zeros_like(i), torch.zeros_like(i)]
    key = [seed & M32, seed >> 32]

    def mulhilo(a, m):
        al, ah, ml, mh = a & 0xFFFF, a >> 16, m & 0xFFFF, m >> 16
        low = al * ml
        mid = ah * ml + (low >> 16)
        mid2 = al * mh + (mid & 0xFFFF)
        return ah * mh + (mid >> 16) + (mid2 >> 16), ((mid2 & 0xFFFF) << 16) | (low & 0xFFFF)

    for r in range(10):
        if r:
            key = [(key[0] + 0x9E3779B9) & M32, (key[1] + 0xBB67AE85) & M32]
        h0, l0 = mulhilo(ctr[0], 0xD2511F53)
        h1, l1 = mulhilo(ctr[2], 0xCD9E8D57)
        ctr = [h1 ^ ctr[1] ^ key[0], l1, h0 ^ ctr[3] ^ key[1], l0]
    return torch.stack(ctr, 1).reshape(-1)[:n]


def _x_drop(x, s):
    p = float(np.float32(s["p"]))
    if p == 0:
        return x.double()
    keep = _x_words(s["rng"], x.numel()).view(x.shape) >= math.floor(p * 2.0 ** 32)
    return x.double() / (1.0 - p) * keep


def _x_mx(v):
    """MXFP8 along the last axis in 64 bits: element values [rows, blocks, 32] and scale exponents."""
    b = v.reshape(v.shape[0], -1, 32)
    amax = b.abs().amax(2, keepdim=True)
    e = torch.where(amax > 0, (torch.frexp(amax)[1] - 9).clamp(-127, 127), 0)
    u = torch.ldexp(b, -e).clamp(-448, 448)
    step = torch.ldexp(torch.ones_like(u), (torch.frexp(u)[1] - 1).clamp(min=-6) - 3)
    return torch.round(u / step) * step, e


def _x_fq(v):
    q, e = _x_mx(v)
    return torch.ldexp(q, e).reshape(v.shape)


def _x_codes(codes):
    e = codes[0].long()
    ex, m = (e >> 3) & 15, e & 7
    v = torch.where(ex == 0, m * 2.0 ** -9, torch.ldexp(1.0 + m / 8.0, ex - 7)) * torch.where(e > 127, -1.0, 1.0)
    v = v.double().view(e.shape[0], -1, 32)
    return torch.ldexp(v, codes[1].long().unsqueeze(2) - 127).view(e.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "dropout":
        y = _x_drop(s["x"], s)
        return y if s["residual"] is None else y + s["residual"].double()
    if op == "dropout_bwd":
        return _x_drop(s["dy"], s)
    if op == "norm":
        v = _x_drop(s["x"], s)
        if s["residual"] is not None:
            v = v + s["residual"].double()
        r = (v.square().sum(1) / v.shape[1] + s["eps"]).pow(-0.5)
        y = v * r[:, None] * s["weight"].double()
        out = dict(sum=v, rstd=r)
        if s["y"]:
            out["y"] = y
        if s["mx"]:
            q, e = _x_mx(y)
            out["mx"] = dict(elems=q.reshape(y.shape), scales=torch.ldexp(torch.ones_like(r[:, None]), e[..., 0]))
        return out
    if op == "norm_bwd":
        t, r, dy = s["sum"].double(), s["rstd"].double()[:, None], s["dy"].double()
        n = t * r                                   # the normalised rows
        g = dy * s["weight"].double()
        ds = r * (g - n * (g * n).sum(1, keepdim=True) / t.shape[1])
        if s["dsum"] is not None:
            ds = ds + s["dsum"].double()
        return dict(dresidual=ds, dx=_x_drop(ds, s), dweight=(dy * n).sum(0))
    mx, I = s["mode"] == "mxfp8", s["I"]
    val = (lambda w: _x_codes(w)) if mx else (lambda w: w.double())
    if op == "ffn":
        x = val(s["x"])
        w = [val(a).T if mx else val(a) for a in s["w"]]
        hg, hu = x @ w[0], x @ w[1]
        a = hg * torch.sigmoid(hg) * hu
        out = (_x_fq(a) if mx else a) @ w[2]
        if s["addend"] is not None:
            out = out + s["addend"].double()
        return dict(out=out, h=torch.cat([hg, hu], 1)) if s["save"] else dict(out=out)
    w = [val(a) for a in s["w"]]
    x, dy, h = s["x"].double(), s["dy"].double(), s["h"].double()
    hg, hu = h[:, :I], h[:, I:]
    sg = torch.sigmoid(hg)
    G = (_x_fq(dy) if mx else dy) @ w[2].T
    dh = torch.cat([G * hu * (sg + hg * sg * (1.0 - sg)), G * hg * sg], 1)
    q = _x_fq(dh) if mx else dh
    dx = q @ torch.cat([w[0], w[1]], 1).T
    if s["addend"] is not None:
        dx = dx + s["addend"].double()
    dw = x.T @ dh
    return dict(dx=dx, dw_gate=dw[:, :I], dw_up=dw[:, I:], dw_down=(hg * sg * hu).T @ dy)
