"""The routed experts taken apart, in fp64 with torch on whatever device the
tensors are: sort of token slots, rows into experts' order and back, blocks of
128 with one scale, and the products on them. test_routed_reference.py holds
these to element-by-element loops and, where they are gradients, to differences."""
import torch

BLK, LEAST = 128, 2.0 ** -52


def sort_rows(n, E, align):
    """Most rows of n slots."""
    return (n + min(E, n) * (align - 1)) // align * align


def sort(ids, E, align):
    """dict(offsets, slots, row_slots), int32 on ids' device."""
    T, k = ids.shape
    runs = [[] for _ in range(E)]
    for f, e in enumerate(ids.reshape(-1).tolist()):
        if 0 <= e < E:
            runs[e].append(f)
    offsets, slots, row_slots = [0], [-1] * (T * k), [-1] * sort_rows(T * k, E, align)
    for run in runs:
        for i, f in enumerate(run):
            slots[f], row_slots[offsets[-1] + i] = offsets[-1] + i, f
        offsets.append(offsets[-1] + -(-len(run) // align) * align)
    t = lambda v: torch.tensor(v, dtype=torch.int32, device=ids.device)   # noqa: E731
    return dict(offsets=t(offsets), slots=t(slots).view(T, k), row_slots=t(row_slots))


def permute(x, s):
    """rows fp64 [rows, H], zeros in padding rows and behind the last run."""
    src = s["row_slots"].long()
    k = s["slots"].shape[1]
    rows = torch.zeros(src.numel(), x.shape[1], dtype=torch.float64, device=x.device)
    at = (src >= 0).nonzero()[:, 0]
    rows[at] = x.double()[src[at] // k]
    return rows


def unpermute(y, s, w=None, addend=None):
    """(out, the sum of magnitudes that its rounding errors are relative to)."""
    slots = s["slots"].long()
    T, k = slots.shape
    out = torch.zeros(T, y.shape[1], dtype=torch.float64, device=y.device)
    mag = torch.zeros_like(out)
    for j in range(k):
        t = ((slots[:, j] >= 0) & (slots[:, j] < y.shape[0])).nonzero()[:, 0]
        v = y.double()[slots[t, j]]
        if w is not None:
            v = v * w.double()[t, j, None]
        out[t] += v
        mag[t] += v.abs()
    if addend is not None:
        out, mag = out + addend.double(), mag + addend.double().abs()
    return out, mag


def unpermute_backward(dout, y, s, w):
    """(dy, dw, the magnitudes of dw's sums)."""
    slots = s["slots"].long()
    dy = torch.zeros(y.shape, dtype=torch.float64, device=y.device)
    dw = torch.zeros(slots.shape, dtype=torch.float64, device=y.device)
    mag = torch.zeros_like(dw)
    for j in range(slots.shape[1]):
        t = (slots[:, j] >= 0).nonzero()[:, 0]
        r = slots[t, j]
        d = dout.double()[t]
        dy[r] = w.double()[t, j, None] * d
        dw[t, j] = (d * y.double()[r]).sum(1)
        mag[t, j] = (d * y.double()[r]).abs().sum(1)
    return dy, dw, mag


def _pad(v, rows, cols):
    out = torch.zeros(v.shape[0], rows, cols, dtype=torch.float64, device=v.device)
    out[:, :v.shape[1], :v.shape[2]] = v
    return out


def scales(v, tile=False):
    """(m / 448 per block, 448 v / m per value) of v [B, rows, K] in fp64; finite values."""
    B, n, K = v.shape
    nk, nr = -(-K // BLK), -(-n // BLK)
    b = _pad(v.double(), nr * BLK, nk * BLK).view(B, nr, BLK, nk, BLK)
    if tile:
        m = b.abs().amax((2, 4)).clamp(min=LEAST)
        full = m[:, :, None, :, None]
        s = m / 448.0
    else:
        m = b.abs().amax(4).clamp(min=LEAST)           # [B, nr, BLK, nk]
        full = m[..., None]
        s = (m / 448.0).reshape(B, nr * BLK, nk)[:, :n].transpose(1, 2)
    return s, (b * 448.0 / full).reshape(B, nr * BLK, nk * BLK)[:, :n, :K]


def half_step(u):
    """Half of E4M3's spacing at u."""
    e = torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6)))
    return torch.pow(2.0, e - 4)


def codes(elems):
    """Values of E4M3FN codes (uint8), fp64."""
    return elems.view(torch.float8_e4m3fn).double()


def row_values(elems, sc):
    """fp64 [rows, K] of codes [rows, K] with scales [K/128, rows]."""
    return codes(elems) * sc.double().t().repeat_interleave(BLK, 1)[:, :elems.shape[1]]


def tile_values(elems, sc):
    """fp64 [.., rows, K] of codes with scales [.., rows/128, K/128]."""
    full = sc.double().repeat_interleave(BLK, -1).repeat_interleave(BLK, -2)
    return codes(elems) * full[..., :elems.shape[-2], :elems.shape[-1]]


def matmul(a, b, offsets=None):
    """(out, magnitudes): a [M, K], b [N, K] or [E, N, K], fp64; rows of no run NaN."""
    if offsets is None:
        return a @ b.t(), a.abs() @ b.abs().t()
    off = offsets.tolist()
    out = torch.full((a.shape[0], b.shape[1]), float("nan"), dtype=torch.float64, device=a.device)
    mag = out.clone()
    for e in range(len(off) - 1):
        r = slice(off[e], off[e + 1])
        out[r] = a[r] @ b[e].t()
        mag[r] = a[r].abs() @ b[e].abs().t()
    return out, mag


def wgrad(dy, x, offsets=None, addend=None):
    """(out, magnitudes): dy [N, R], x [K, R], fp64."""
    if offsets is None:
        out, mag = dy @ x.t(), dy.abs() @ x.abs().t()
    else:
        off = offsets.tolist()
        runs = [slice(off[e], off[e + 1]) for e in range(len(off) - 1)]
        out = torch.stack([dy[:, r] @ x[:, r].t() for r in runs])
        mag = torch.stack([dy[:, r].abs() @ x[:, r].abs().t() for r in runs])
    if addend is not None:
        out, mag = out + addend.double(), mag + addend.double().abs()
    return out, mag


def glu(h):
    g, u = h.double().chunk(2, -1)
    return g * torch.sigmoid(g) * u


def glu_backward(da, h):
    g, u = h.double().chunk(2, -1)
    s = torch.sigmoid(g)
    return torch.cat([da.double() * u * s * (1.0 + g * (1.0 - s)), da.double() * g * s], -1)


# ----------------------------------------------------------------------------- bounds

def half_eps(dtype):
    return torch.finfo(dtype).eps / 2


def product_bound(ref, mag, K, dtype):
    """Per element: a block's 128 additions are each off by at most one unit in the
    last place (2^-23), its scale's product and its addition into the accumulator
    by half of one (2^-24) each, the addend's addition too; then one rounding to the
    output's type. The fp8 matrix cores of bf16 results cut 15 products of a group
    of 16 at 2^-13 of the largest one's binade: 15 * 2^-13 times the groups'
    largest products, which add up to at most mag."""
    nk = -(-K // BLK)
    cut = 15 * 2.0 ** -13 if dtype is torch.bfloat16 else 0.0
    return ((2 * min(K, BLK) + nk + 4) * 2.0 ** -24 + cut) * mag * 1.01 + half_eps(dtype) * ref.abs() * 1.01 + 1e-37


def product_norm_bound(ref, mag, K, dtype):
    """Of the whole, where errors are spread: a rounding is uniform in half a step
    at the worst place of a binade (half_eps / sqrt 3), the cut of a product
    uniform in 2^-13 of its group's largest; the fp32 terms stay at their worst."""
    nk = -(-K // BLK)
    cut = 2.0 ** -13 if dtype is torch.bfloat16 else 0.0
    return ((2 * min(K, BLK) + nk + 4) * 2.0 ** -24 + cut) * mag.norm() + half_eps(dtype) / 3 ** 0.5 * ref.norm() + 1e-37


def product_errors(got, ref, mag, K):
    """None, or what is wrong with a product."""
    bad = ~((got.double() - ref).abs() <= product_bound(ref, mag, K, got.dtype))
    if bad.any():
        return int(bad.sum()), bad.nonzero()[:4].tolist()
    off, most = float((got.double() - ref).norm()), float(product_norm_bound(ref, mag, K, got.dtype))
    # a single value's rounding can be its worst: few values are held to the bound above alone
    return (off, most) if got.numel() >= 256 and not off <= most else None
