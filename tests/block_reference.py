"""The feed-forward block in fp64 with torch, for shapes that the numpy oracle
would take minutes over: the formulas of oracle/block.py, on whatever device the
tensors are. test_block_plan.py holds it to the oracle."""
import torch


def pow2(e):
    """2^e by its bits (torch.ldexp goes through pow, which may be off by a bit and so break ties)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def fake_quant(v, axis):
    """The values that MXFP8 codes of v hold, 32 values a block along axis."""
    b = v.movedim(axis, -1)
    shape = b.shape
    b = b.reshape(-1, 32)
    amax = b.abs().amax(1, keepdim=True)
    e = torch.where(amax > 0, (torch.frexp(amax)[1] - 9).clamp(-127, 127), 0)
    u = (b * pow2(-e)).clamp(-448.0, 448.0)
    quantum = pow2((torch.frexp(u)[1] - 1).clamp(min=-6) - 3)   # 3 bits below the leading one
    return (torch.round(u / quantum) * quantum * pow2(e)).reshape(shape).movedim(-1, axis)


def keep(v, axis):
    return v


def forward(x, wg, wu, wd, addend=None, fq=keep):
    """(out, h, a)."""
    xq = fq(x, 1)
    hg, hu = xq @ fq(wg, 0), xq @ fq(wu, 0)
    a = hg * torch.sigmoid(hg) * hu
    out = fq(a, 1) @ fq(wd, 0)
    return out if addend is None else out + addend, torch.cat([hg, hu], 1), a


def backward(x, wg, wu, wd, h, dy, addend=None, fq=keep):
    """dict(dx, dw_gate, dw_up, dw_down, dh, a) from the saved h."""
    hg, hu = h.chunk(2, 1)
    s = torch.sigmoid(hg)
    a = hg * s * hu
    da = fq(dy, 1) @ fq(wd, 1).T
    dhg, dhu = da * hu * s * (1.0 + hg * (1.0 - s)), da * hg * s
    dx = fq(dhg, 1) @ fq(wg, 1).T + fq(dhu, 1) @ fq(wu, 1).T
    if addend is not None:
        dx = dx + addend
    return dict(dx=dx, dw_gate=x.T @ dhg, dw_up=x.T @ dhu, dw_down=a.T @ dy, dh=torch.cat([dhg, dhu], 1), a=a)
