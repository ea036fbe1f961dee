"""The routed experts taken apart, case by case: token rows sorted by expert
and back with their gate weights (and both gradients), quantization to 8-bit
floating point with one fp32 scale for each block of 128 values (activation rows
1 x 128 with scales [K / 128, rows], weights 128 x 128 with scales
[rows / 128, K / 128], either orientation, optionally of the gated activation
silu(g) * u, whose gradient goes with it), and the matrix products on such
operands: dense, grouped by expert, and the weight gradients.

``run`` computes a case in its plain form (elementary torch operations in 32
bits, one rounding at the end) or, with ``own`` set, through the library's
entry points. ``exact`` evaluates the definitions in 64 bits.

Sizes are those of the repository's own configurations: hidden sizes 7,168 and
4,096 with expert widths 2,048 and 1,024, 256, 8 and 4 experts, top-8 and top-1
routing, 2,048 tokens a GPU and 16,384 received rows, and single tokens as a
decoder calls them.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
BLK = 128           # values that share a scale
LEAST = 2.0 ** -52  # smallest magnitude that a block's scale is taken from

_DT = dict(bf16=torch.bfloat16, fp32=torch.float32)


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token sent to its 8 of 256 experts: latency of the two calls
        dict(name="permute_1x7168_top8", op="permute", T=1, H=7168, E=256, k=8, align=1, dtype="bf16", fp8=False,
             away=0.0),
        # a training batch of 2,048 tokens a GPU, rows quantized on the way for the experts' products
        dict(name="permute_2048x7168_top8_fp8", op="permute", T=2048, H=7168, E=256, k=8, align=16, dtype="bf16",
             fp8=True, away=0.0),
        # gradient of the sort for a ragged batch, a quarter of whose choices live on other GPUs
        dict(name="permute_bwd_777x4096_top2", op="permute_bwd", T=777, H=4096, E=8, k=2, align=128, dtype="bf16",
             away=0.25),
        # the experts' rows of 2,048 tokens back in token order, weighted, onto the shared expert's output
        dict(name="unpermute_2048x7168_top8", op="unpermute", T=2048, H=7168, E=256, k=8, align=16, dtype="bf16",
             away=0.0, weights=True, addend=True),
        # its gradient for an odd batch with fp32 rows
        dict(name="unpermute_bwd_1001x4096_top2_fp32", op="unpermute_bwd", T=1001, H=4096, E=8, k=2, align=128,
             dtype="fp32", away=0.25),
        # gate | up weights of 4 experts for the forward product, after each optimizer step
        dict(name="quantize_weights_4x4096x7168", op="quantize", B=4, rows=4096, K=7168, turned=True, tile=True,
             glu=False, dtype="bf16"),
        # an odd batch's gated activation as rows for the down product
        dict(name="quantize_glu_2047x2048", op="quantize", B=1, rows=2047, K=2048, turned=False, tile=False, glu=True,
             dtype="bf16"),
        # gradient of the gated activation, the largest batch
        dict(name="glu_bwd_16384x2048", op="glu_bwd", T=16384, I=2048),
        # one decoded token through the gate | up weights of a shared expert
        dict(name="matmul_1x4096x7168", op="matmul", M=1, N=4096, K=7168, E=0, spread=0.0, out="bf16"),
        # a decoder's batch: 16 experts with 8 rows each on average, some with none
        dict(name="matmul_16x128x4096x7168", op="matmul", M=128, N=4096, K=7168, E=16, spread=1.0, out="bf16"),
        # the received rows of one GPU of 64, skewed over its 4 experts: the largest product
        dict(name="matmul_4x16384x4096x7168", op="matmul", M=16384, N=4096, K=7168, E=4, spread=0.6, out="bf16"),
        # gate | up weight gradients of the same rows
        dict(name="wgrad_4x16384x4096x7168", op="wgrad", R=16384, N=4096, K=7168, E=4, spread=0.6, out="bf16",
             addend=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["permute", "permute_bwd", "unpermute", "unpermute_bwd", "quantize", "glu_bwd", "matmul", "matmul",
                     "wgrad", "wgrad"])
    if op in ("permute", "permute_bwd", "unpermute", "unpermute_bwd"):
        E = _log(rng, 1, 256)
        k = rng.randint(1, min(E, 8))
        fp8 = op == "permute" and rng.random() < 0.5
        c = dict(op=op, T=_log(rng, 1, 16384 // k), H=16 * _log(rng, 4, 448), E=E, k=k, align=rng.choice([1, 16, 128]),
                 dtype="bf16" if fp8 else rng.choice(["bf16", "fp32"]), away=rng.choice([0.0, 0.3]))
        c["T"] = min(c["T"], 2048) if c["dtype"] == "fp32" else c["T"]
        if op == "permute":
            c["fp8"] = fp8
        if op == "unpermute":
            c["weights"], c["addend"] = rng.random() < 0.8, rng.random() < 0.5
        return c
    if op == "quantize":
        glu = rng.random() < 0.4
        turned = rng.random() < 0.5
        return dict(op=op, B=1 if glu else rng.randint(1, 4), rows=16 * _log(rng, 1, 256) if turned else _log(rng, 1, 4096),
                    K=16 * _log(rng, 4, 448), turned=turned, tile=not glu and rng.random() < 0.5, glu=glu,
                    dtype="bf16" if glu else rng.choice(["bf16", "fp32"]))
    if op == "glu_bwd":
        return dict(op=op, T=_log(rng, 1, 16384), I=16 * _log(rng, 4, 128))
    E = rng.choice([0, 0, _log(rng, 1, 16)])
    N, K = 16 * _log(rng, 4, 256), 16 * _log(rng, 4, 448)
    c = dict(op=op, N=N, K=K, E=E, spread=rng.choice([0.3, 1.0]) if E else 0.0, out=rng.choice(["bf16", "fp32"]))
    if op == "matmul":
        return dict(c, M=_log(rng, 1, 16384))
    return dict(c, R=128 * _log(rng, 1, 128) if E else 16 * _log(rng, 1, 1024), addend=rng.random() < 0.5)


def _cap(case):
    """Rows that a sort can fill at most: every choice, and each expert's padding."""
    n, a = case["T"] * case["k"], case["align"]
    return (n + min(case["E"], n) * (a - 1)) // a * a


def work(case):
    op = case["op"]
    if op in ("permute", "permute_bwd", "unpermute", "unpermute_bwd"):
        T, H, k, es = case["T"], case["H"], case["k"], 4 if case["dtype"] == "fp32" else 2
        R = T * k * (1.0 - case["away"])
        if op == "permute":
            row = H + 4 * -(-H // BLK) if case["fp8"] else es * H
            return dict(bytes=T * H * es + R * row + 8 * T * k + 4 * _cap(case) + 4 * case["E"], flops=R * H)
        if op == "permute_bwd":
            return dict(bytes=(R + T) * H * es + 4 * T * k, flops=R * H)
        if op == "unpermute":
            return dict(bytes=(R + T * (2 if case["addend"] else 1)) * H * es + 8 * T * k, flops=2 * R * H)
        return dict(bytes=(2 * R + T) * H * es + 12 * T * k, flops=3 * R * H)
    if op == "quantize":
        n, es = case["B"] * case["rows"] * case["K"], 4 if case["dtype"] == "fp32" else 2
        sc = n // BLK // (BLK if case["tile"] else 1)
        return dict(bytes=n * es * (2 if case["glu"] else 1) + n + 4 * sc, flops=3 * n)
    if op == "glu_bwd":
        return dict(bytes=10 * case["T"] * case["I"], flops=8 * case["T"] * case["I"])
    N, K, E, es = case["N"], case["K"], max(case["E"], 1), 4 if case["out"] == "fp32" else 2
    if op == "matmul":
        M = case["M"]
        read = min(E, M)   # an expert without rows need not be read
        return dict(bytes=M * K * 33 // 32 + read * N * K + es * M * N, flops=2 * M * N * K)
    R = case["R"]
    return dict(bytes=R * (N + K) * 33 // 32 + es * E * N * K * (2 if case["addend"] else 1), flops=2 * R * N * K)


# ----------------------------------------------------------------------------- inputs

def _randn(g, shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(shape, device=DEV, generator=g) * scale).to(dtype)


def _route(g, T, E, k, away):
    """k different experts a token, some more popular than others; -1 for choices that live elsewhere."""
    logits = torch.randn(T, E, device=DEV, generator=g) + 0.5 * torch.randn(E, device=DEV, generator=g)
    ids = logits.topk(k, 1).indices.to(torch.int32)
    gone = torch.rand(T, k, device=DEV, generator=g) < away
    w = torch.softmax(logits.gather(1, ids.long()), 1)
    return torch.where(gone, torch.full_like(ids, -1), ids), w


def _segments(g, n, E, spread, unit):
    """int32 [E + 1]: n rows in E runs of whole units, their sizes lognormal with the given spread."""
    share = torch.exp(spread * torch.randn(E, device=DEV, generator=g, dtype=torch.float64)).cumsum(0)
    ends = (share / share[-1] * (n // unit)).round().long() * unit
    ends[-1] = n
    return torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), ends]).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(DEV).manual_seed(1_000_003 * (seed + 1) + 29)
    s, op = dict(case), case["op"]
    if op in ("permute", "permute_bwd", "unpermute", "unpermute_bwd"):
        T, H, E, k, dt = case["T"], case["H"], case["E"], case["k"], _DT[case["dtype"]]
        s["ids"], s["w"] = _route(g, T, E, k, case["away"])
        cap = _cap(case)
        if op == "permute":
            s["x"] = _randn(g, (T, H), dt)
            # the rows' buffers, made once: what lies behind the last expert's rows stays as it is
            if case["fp8"]:
                s["buffers"] = dict(elems=torch.zeros(cap, H, dtype=torch.uint8, device=DEV),
                                    scales=torch.zeros(-(-H // BLK), cap, device=DEV))
            else:
                s["buffers"] = dict(rows=torch.zeros(cap, H, dtype=dt, device=DEV))
            return s
        s["sort"] = _sort(s["ids"], E, case["align"])
        s["y"] = _randn(g, (cap, H), dt)
        if op == "unpermute":
            s["w"] = s["w"] if case["weights"] else None
            s["addend"] = _randn(g, (T, H), dt) if case["addend"] else None
        if op == "unpermute_bwd":
            s["dout"] = _randn(g, (T, H), dt)
            s["buffers"] = dict(dy=torch.zeros(cap, H, dtype=dt, device=DEV), dw=torch.zeros(T, k, device=DEV))
        return s
    if op == "quantize":
        B, rows, K, two = case["B"], case["rows"], case["K"], 2 if case["glu"] else 1
        s["src"] = _randn(g, (B, K, two * rows) if case["turned"] else (B, rows, two * K), _DT[case["dtype"]])
        return s
    if op == "glu_bwd":
        s["h"] = _randn(g, (case["T"], 2 * case["I"]))
        s["da"] = _randn(g, (case["T"], case["I"]))
        return s
    N, K, E = case["N"], case["K"], case["E"]
    lead = (E,) if E else ()
    if op == "matmul":
        M = case["M"]
        s["a"] = _codes_rows(_randn(g, (M, K), torch.float32))
        s["b"] = _codes_tiles(_randn(g, lead + (N, K), torch.float32, K ** -0.5))
        s["offsets"] = _segments(g, M, E, case["spread"], 1) if E else None
        s["out_buffer"] = torch.zeros(M, N, dtype=_DT[case["out"]], device=DEV)
        rows = M
    else:
        R = case["R"]
        s["dy"] = _codes_rows(_randn(g, (N, R), torch.float32, 0.01))
        s["x"] = _codes_rows(_randn(g, (K, R), torch.float32))
        s["offsets"] = _segments(g, R, E, case["spread"], BLK) if E else None
        s["addend"] = _randn(g, lead + (N, K), _DT[case["out"]]) if case["addend"] else None
        rows = R
    s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max()) if E else rows   # rows of the fullest expert
    return s


# ----------------------------------------------------------------------------- plain forms (32 bits)

def _sort(ids, E, align):
    """offsets [E + 1], slots [T, k] (each choice's row, -1 for none), row_slots [cap] (each row's choice, -1 for none)."""
    T, k = ids.shape
    n = T * k
    cap = (n + min(E, n) * (align - 1)) // align * align
    key = torch.where((ids >= 0) & (ids < E), ids, E).view(-1).long()
    counts = torch.zeros(E + 1, dtype=torch.long, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    begin = counts.cumsum(0) - counts                            # in sorted order, without padding
    offsets = torch.zeros(E + 1, dtype=torch.long, device=ids.device)
    offsets[1:] = ((counts[:E] + align - 1) // align * align).cumsum(0)
    order = torch.sort(key, stable=True).indices
    rank = torch.empty_like(order)
    rank[order] = torch.arange(n, device=ids.device) - begin[key[order]]
    there = key < E
    slots = torch.where(there, offsets[key.clamp(max=E - 1)] + rank, -1)
    row_slots = torch.full((cap + 1,), -1, dtype=torch.long, device=ids.device)
    row_slots[torch.where(there, slots, cap)] = torch.arange(n, device=ids.device)
    return dict(offsets=offsets.to(torch.int32), slots=slots.view(T, k).to(torch.int32),
                row_slots=row_slots[:cap].to(torch.int32))


def _scale_of(amax):
    """The scale of a block and the factor to its codes; a block with a NaN or an infinity has scale 1."""
    fine = torch.isfinite(amax)
    m = torch.where(fine, amax.clamp(min=LEAST), torch.full_like(amax, 448.0))
    return m / 448.0, 448.0 / m, fine


def _blocks(v, axis):
    """v with axis cut into blocks of 128 (zeros behind a last, shorter one): [.., blocks, 128, ..]."""
    n = v.shape[axis]
    nb = -(-n // BLK)
    if nb * BLK != n:
        shape = list(v.shape)
        shape[axis] = nb * BLK - n
        v = torch.cat([v, v.new_zeros(shape)], axis)
    return v.unflatten(axis, (nb, BLK))


def _to_codes(v, r, fine):
    return torch.where(fine, (v * r).clamp(-448.0, 448.0), float("nan")).to(torch.float8_e4m3fn)


def _codes_rows(v):
    """E4M3 codes [.., rows, K] (bytes) and scales [.., K/128, rows] of v, 128 values along the last axis a block."""
    b = _blocks(v.float(), -1)
    amax = b.abs().amax(-1)
    sc, r, fine = _scale_of(torch.where(torch.isfinite(b).all(-1), amax, float("nan")))
    q = _to_codes(b, r[..., None], fine[..., None]).view(torch.uint8).flatten(-2)[..., :v.shape[-1]].contiguous()
    return q, sc.mT.contiguous()


def _codes_tiles(v):
    """Codes and scales [.., rows/128, K/128] of 128 x 128 blocks over the last two axes."""
    b = _blocks(_blocks(v.float(), -1), -3)                      # [.., rb, 128, kb, 128]
    amax = b.abs().amax((-3, -1))
    sc, r, fine = _scale_of(torch.where(torch.isfinite(b).all(-1).all(-2), amax, float("nan")))
    q = _to_codes(b, r[..., :, None, :, None], fine[..., :, None, :, None]).view(torch.uint8)
    q = q.flatten(-2).flatten(-3, -2)[..., :v.shape[-2], :v.shape[-1]].contiguous()
    return q, sc


def _values_rows(codes):
    q, sc = codes
    return q.view(torch.float8_e4m3fn).float() * sc.mT.repeat_interleave(BLK, -1)[..., :q.shape[-1]]


def _values_tiles(codes):
    q, sc = codes
    full = sc.repeat_interleave(BLK, -1).repeat_interleave(BLK, -2)
    return q.view(torch.float8_e4m3fn).float() * full[..., :q.shape[-2], :q.shape[-1]]


def _typed(q, sc):
    """The code bytes as the values they stand for (a view)."""
    return dict(elems=q.view(torch.float8_e4m3fn), scales=sc)


def _from_rows(rows, slots, w=None):
    """sum over j of w[t, j] * rows[slots[t, j]], choices without a row left out."""
    T, k = slots.shape
    there = slots >= 0
    v = rows.float()[slots.clamp(min=0).long()] * there[..., None]
    return (v if w is None else v * w[..., None]).sum(1)


def _into_rows(values, slots, cap):
    """[cap, ..] with values [T, k, ..] in their rows and zeros elsewhere."""
    T, k = slots.shape
    out = values.new_zeros((cap + 1,) + values.shape[2:])
    out[torch.where(slots >= 0, slots, cap).view(-1).long()] = values.flatten(0, 1)
    return out[:cap]


def _plain_permute(s):
    sort = _sort(s["ids"], s["E"], s["align"])
    cap, k = sort["row_slots"].shape[0], s["k"]
    out = dict(sort)
    if not s["fp8"]:
        out["rows"] = _into_rows(s["x"].unsqueeze(1).expand(-1, k, -1), sort["slots"], cap)
        return out
    q, sc = _codes_rows(s["x"])
    # a padding row holds zeros, whose scale is the smallest
    pad = (torch.arange(cap, device=q.device) < sort["offsets"][-1]) & (sort["row_slots"] < 0)
    scales = _into_rows(sc.mT.unsqueeze(1).expand(-1, k, -1), sort["slots"], cap)
    scales = torch.where(pad[:, None], LEAST / 448.0, scales).mT.contiguous()
    out.update(_typed(_into_rows(q.unsqueeze(1).expand(-1, k, -1), sort["slots"], cap), scales))
    return out


def _plain_unpermute_bwd(s):
    slots = s["sort"]["slots"]
    cap, dt = s["y"].shape[0], s["y"].dtype
    d = s["dout"].float()
    there = slots >= 0
    yr = s["y"].float()[slots.clamp(min=0).long()] * there[..., None]
    return dict(dy=_into_rows((d[:, None] * s["w"][..., None]).to(dt), slots, cap), dw=(yr * d[:, None]).sum(-1))


def _glu(h, axis=-1):
    hg, hu = h.float().chunk(2, axis)
    return hg / (1.0 + torch.exp(-hg)) * hu


def _plain_quantize(s):
    v = _glu(s["src"]) if s["glu"] else s["src"].float()
    if s["turned"]:
        v = v.transpose(1, 2)
    return _typed(*(_codes_tiles(v) if s["tile"] else _codes_rows(v)))


def _plain_glu_bwd(s):
    hg, hu = s["h"].float().chunk(2, 1)
    da = s["da"].float()
    sg = 1.0 / (1.0 + torch.exp(-hg))
    return torch.cat([da * hu * sg * (1.0 + hg * (1.0 - sg)), da * hg * sg], 1).to(torch.bfloat16)


def _runs(s, rows):
    """[E, most]: each expert's rows, and which of them there are."""
    off = s["offsets"].long()
    at = off[:-1, None] + torch.arange(s["most"], device=off.device)
    there = at < off[1:, None]
    return at.clamp(max=rows - 1), there


def _plain_matmul(s):
    a, b = _values_rows(s["a"]), _values_tiles(s["b"])
    dt = _DT[s["out"]]
    if not s["E"]:
        return (a @ b.T).to(dt)
    at, there = _runs(s, a.shape[0])
    prod = torch.bmm(a[at], b.transpose(1, 2).contiguous())
    out = prod.new_zeros((a.shape[0] + 1, s["N"]))
    out[torch.where(there, at, a.shape[0]).view(-1)] = prod.flatten(0, 1)
    return out[:-1].to(dt)


def _plain_wgrad(s):
    dy, x = _values_rows(s["dy"]), _values_rows(s["x"])
    if not s["E"]:
        out = dy @ x.T
    else:
        at, there = _runs(s, s["R"])
        d = (dy[:, at] * there).transpose(0, 1).contiguous()                # [E, N, most]
        out = torch.bmm(d, x[:, at].permute(1, 2, 0).contiguous())          # [E, N, K]
    if s["addend"] is not None:
        out = out + s["addend"].float()
    return out.to(_DT[s["out"]])


def _plain_unpermute(s):
    out = _from_rows(s["y"], s["sort"]["slots"], s["w"])
    if s["addend"] is not None:
        out = out + s["addend"].float()
    return out.to(s["y"].dtype)


_PLAIN = dict(permute=_plain_permute, permute_bwd=lambda s: _from_rows(s["y"], s["sort"]["slots"]).to(s["y"].dtype),
              unpermute=_plain_unpermute, unpermute_bwd=_plain_unpermute_bwd, quantize=_plain_quantize,
              glu_bwd=_plain_glu_bwd, matmul=_plain_matmul, wgrad=_plain_wgrad)


# ----------------------------------------------------------------------------- the library's calls

def _own(s):
    import mixture_experts_layer_table_amd as mok
    op = s["op"]
    if op == "permute":
        sort = mok.sort_tokens(s["ids"], s["E"], align=s["align"])
        out = mok.permute(s["x"], sort, rows=not s["fp8"], fp8=s["fp8"], outs=s["buffers"])
        return dict(sort, **(_typed(out["elems"], out["scales"]) if s["fp8"] else out))
    if op == "permute_bwd":
        return mok.permute_backward(s["y"], s["sort"])
    if op == "unpermute":
        return mok.unpermute(s["y"], s["sort"], w=s["w"], addend=s["addend"])
    if op == "unpermute_bwd":
        return mok.unpermute_backward(s["dout"], s["y"], s["sort"], s["w"], grads=s["buffers"])
    if op == "quantize":
        return _typed(*mok.fp8_quantize(s["src"], s["turned"], tile=s["tile"], glu=s["glu"]))
    if op == "glu_bwd":
        return mok.glu_backward(s["da"], s["h"])
    if op == "matmul":
        return mok.fp8_matmul(s["a"], s["b"], s["offsets"], out=s["out_buffer"])
    return mok.fp8_wgrad(s["dy"], s["x"], s["offsets"], out_dtype=_DT[s["out"]], addend=s["addend"])


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ----------------------------------------------------------------------------- the definitions in 64 bits

def _x_codes(v, tile):
    """Values that the E4M3 codes of v [B, rows, K] stand for, unscaled, and the scales, in 64 bits."""
    B, n, K = v.shape
    nk, nr = (K + BLK - 1) // BLK, (n + BLK - 1) // BLK
    kb = torch.arange(K, device=v.device) // BLK
    amax = v.new_zeros((B, n, nk)).index_reduce_(2, kb, v.abs(), "amax")
    if tile:
        amax = v.new_zeros((B, nr, nk)).index_reduce_(1, torch.arange(n, device=v.device) // BLK, amax, "amax")
    m = torch.maximum(amax, torch.full_like(amax, LEAST))
    full = m[:, :, kb]
    if tile:
        full = full[:, torch.arange(n, device=v.device) // BLK]
    u = (v * 448.0 / full).clamp(-448.0, 448.0)
    step = torch.ldexp(torch.ones_like(u), (torch.frexp(u)[1] - 1).clamp(min=-6) - 3)   # E4M3's spacing at u
    return torch.round(u / step) * step, m / 448.0 if tile else (m / 448.0).movedim(2, 1)


def _x_e4m3(q):
    e = q.long()
    ex, m = (e >> 3) & 15, e & 7
    v = torch.where(ex == 0, m.double() * 2.0 ** -9, torch.ldexp(1.0 + m.double() / 8.0, ex - 7))
    return torch.where(e > 127, -v, v)


def _x_rows(codes):
    q, sc = codes
    kb = torch.arange(q.shape[-1], device=q.device) // BLK
    return _x_e4m3(q) * sc.double().movedim(-2, -1)[..., kb]


def _x_tiles(codes):
    q, sc = codes
    kb, rb = (torch.arange(n, device=q.device) // BLK for n in (q.shape[-1], q.shape[-2]))
    return _x_e4m3(q) * sc.double()[..., kb][..., rb, :]


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "permute":
        ids, E, align, k = s["ids"].cpu().tolist(), s["E"], s["align"], s["k"]
        where = [[] for _ in range(E)]
        for t, row in enumerate(ids):
            for j, e in enumerate(row):
                if 0 <= e < E:
                    where[e].append(t * k + j)
        cap = _cap(case)
        row_slots, slots, offsets = [-1] * cap, [-1] * (len(ids) * k), [0]
        for run_ in where:
            at = offsets[-1]
            for i, f in enumerate(run_):
                row_slots[at + i], slots[f] = f, at + i
            offsets.append(at + (len(run_) + align - 1) // align * align)
        x = s["x"].double()
        src = torch.tensor(row_slots, device=DEV)
        inside = torch.arange(cap, device=DEV) < offsets[-1]
        out = {n: torch.tensor(v, dtype=torch.int32, device=DEV) for n, v in
               dict(offsets=offsets, slots=slots, row_slots=row_slots).items()}
        out["slots"] = out["slots"].view(-1, k)
        at = torch.where(src >= 0, src, 0) // k
        if not s["fp8"]:
            out["rows"] = torch.where((src >= 0)[:, None], x[at], 0.0)
            return out
        q, sc = _x_codes(x[None], False)
        out["elems"] = torch.where((src >= 0)[:, None], q[0][at], 0.0)
        out["scales"] = torch.where(src >= 0, sc[0][:, at], torch.where(inside, LEAST / 448.0, 0.0))
        return out
    if op in ("permute_bwd", "unpermute"):
        slots, y = s["sort"]["slots"].long(), s["y"].double()
        w = s["w"].double() if op == "unpermute" and s["w"] is not None else torch.ones(slots.shape, device=DEV).double()
        out = torch.zeros(slots.shape[0], y.shape[1], dtype=torch.float64, device=DEV)
        for j in range(slots.shape[1]):
            t = (slots[:, j] >= 0).nonzero()[:, 0]
            out[t] += w[t, j, None] * y[slots[t, j]]
        return out + s["addend"].double() if op == "unpermute" and s["addend"] is not None else out
    if op == "unpermute_bwd":
        slots, y, d = s["sort"]["slots"].long(), s["y"].double(), s["dout"].double()
        dy, dw = torch.zeros_like(y), torch.zeros(slots.shape, dtype=torch.float64, device=DEV)
        for j in range(slots.shape[1]):
            t = (slots[:, j] >= 0).nonzero()[:, 0]
            r = slots[t, j]
            dy[r] = s["w"].double()[t, j, None] * d[t]
            dw[t, j] = torch.linalg.vecdot(d[t], y[r])
        return dict(dy=dy, dw=dw)
    if op == "quantize":
        v = s["src"].double()
        if s["glu"]:
            half = v.shape[-1] // 2
            v = v[..., :half] * torch.sigmoid(v[..., :half]) * v[..., half:]
        q, sc = _x_codes(v.movedim(1, 2) if s["turned"] else v, s["tile"])
        return dict(elems=q, scales=sc)
    if op == "glu_bwd":
        h, da = s["h"].double(), s["da"].double()
        g, u = h[:, :s["I"]], h[:, s["I"]:]
        sg = torch.sigmoid(g)
        return torch.cat([da * u * (sg + g * sg * (1.0 - sg)), da * g * sg], 1)
    off = s["offsets"].tolist() if s["E"] else None
    if op == "matmul":
        a, b = _x_rows(s["a"]), _x_tiles(s["b"])
        if off is None:
            return torch.matmul(a, b.mT)
        out = torch.zeros(s["M"], s["N"], dtype=torch.float64, device=DEV)
        for e in range(s["E"]):
            out[off[e]:off[e + 1]] = torch.matmul(a[off[e]:off[e + 1]], b[e].mT)
        return out
    d, x = _x_rows(s["dy"]), _x_rows(s["x"])
    add = 0.0 if s["addend"] is None else s["addend"].double()
    if off is None:
        return torch.matmul(d, x.mT) + add
    return torch.stack([torch.matmul(d[:, off[e]:off[e + 1]], x[:, off[e]:off[e + 1]].mT) for e in range(s["E"])]) + add
