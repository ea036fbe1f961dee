"""The routed experts put together from their parts, as a user would: route, sort,
permute into 8-bit rows, grouped products with a gated activation between them,
and back in token order; the whole backward; under a captured graph; on other
streams. Against fp64 of the same codes, step by step."""
import pytest
import torch

import mixture_experts_layer_table_amd as mok
import routed_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


class Experts:
    """Weights of E gated experts in both orientations, as a program keeps them."""

    def __init__(self, E, H, I, seed):
        g = torch.Generator().manual_seed(seed)
        w = lambda *s: (torch.randn(s, generator=g) * s[1] ** -0.5).to(BF).to(DEV)   # noqa: E731
        self.gu, self.dn = w(E, H, 2 * I), w(E, I, H)
        self.gu_f = mok.fp8_quantize(self.gu, True, tile=True)     # [E, 2I, H] along H
        self.dn_f = mok.fp8_quantize(self.dn, True, tile=True)     # [E, H, I] along I
        self.gu_b = mok.fp8_quantize(self.gu, tile=True)           # [E, H, 2I] along 2I
        self.dn_b = mok.fp8_quantize(self.dn, tile=True)           # [E, I, H] along H


def forward(x, logits, k, w, align=128, addend=None):
    """The layer and what its backward needs."""
    E = logits.shape[1]
    ids, gate = mok.route(logits, k)
    sort = mok.sort_tokens(ids, E, align)
    n = sort["row_slots"].shape[0]
    # rows behind the last run stay zeros: the transposed operands of the gradients are quantized over all rows
    xr = mok.permute(x, sort, fp8=True, outs=dict(rows=x.new_zeros((n, x.shape[1])),
                                                  elems=x.new_zeros((n, x.shape[1]), dtype=torch.uint8),
                                                  scales=x.new_zeros(((x.shape[1] + 127) // 128, n), dtype=F32)))
    h = mok.fp8_matmul((xr["elems"], xr["scales"]), w.gu_f, sort["offsets"], out=x.new_zeros((n, w.gu.shape[2])))
    a = mok.fp8_quantize(h[None], glu=True)
    y = mok.fp8_matmul(a, w.dn_f, sort["offsets"], out=x.new_zeros((n, x.shape[1])))
    out = mok.unpermute(y, sort, gate, addend)
    return out, dict(ids=ids, gate=gate, sort=sort, rows=xr, h=h, a=a, y=y)


def backward(dout, s, E, w):
    sort, off = s["sort"], s["sort"]["offsets"]
    g = mok.unpermute_backward(dout, s["y"], sort, s["gate"],
                               grads=dict(dy=torch.zeros_like(s["y"]), dw=torch.empty_like(s["gate"])))
    dyq = mok.fp8_quantize(g["dy"][None])
    da = mok.fp8_matmul(dyq, w.dn_b, off, out=torch.zeros_like(s["h"][:, :w.dn.shape[1]]).contiguous())
    dh = mok.glu_backward(da, s["h"])
    drows = mok.fp8_matmul(mok.fp8_quantize(dh[None]), w.gu_b, off, out=torch.zeros_like(s["y"]))
    # [E, H, 2I] and [E, I, H], contracted over each expert's rows
    xt, dht = mok.fp8_quantize(s["rows"]["rows"][None], True), mok.fp8_quantize(dh[None], True)
    at, dyt = mok.fp8_quantize(s["h"][None], True, glu=True), mok.fp8_quantize(g["dy"][None], True)
    dgu, ddn = mok.fp8_wgrad(xt, dht, off), mok.fp8_wgrad(at, dyt, off)
    return dict(dx=mok.permute_backward(drows, sort), dlogits=mok.route_backward(s["ids"], s["gate"], g["dw"], E),
                dgate=g["dw"], dgu=dgu, ddn=ddn, dy=g["dy"], da=da, dh=dh, dyq=dyq, drows=drows, xt=xt, dht=dht, at=at,
                dyt=dyt)


def _inputs(T, H, E, seed=0):
    g = torch.Generator().manual_seed(seed + T)
    return [torch.randn(s, generator=g).to(d).to(DEV) for s, d in (((T, H), BF), ((T, E), F32), ((T, H), BF))]


def _close(got, ref, mag, K):
    assert R.product_errors(got, ref, mag, K) is None, R.product_errors(got, ref, mag, K)


CASES = [(1, 128, 64, 4, 2), (37, 256, 144, 8, 2), (300, 400, 272, 5, 3), (513, 512, 128, 16, 4)]


@pytest.mark.parametrize("T,H,I,E,k", CASES)
def test_layer_and_its_gradients(T, H, I, E, k):
    print(f"[routed] {T} {H} {I} {E} {k}", flush=True)
    x, logits, dout = _inputs(T, H, E)
    w = Experts(E, H, I, T)
    out, s = forward(x, logits, k, w, addend=x)
    sort = R.sort(s["ids"].cpu(), E, 128)
    for n in sort:
        assert torch.equal(s["sort"][n].cpu(), sort[n])
    off = sort["offsets"]
    end = int(off[-1])
    live = slice(0, end)
    val = lambda c: R.row_values(c[0] if c[0].dim() == 2 else c[0][0], c[1] if c[1].dim() == 2 else c[1][0])   # noqa: E731
    ref, mag = R.matmul(val((s["rows"]["elems"], s["rows"]["scales"])), R.tile_values(*w.gu_f), off)
    _close(s["h"][live], ref[live], mag[live], H)
    ref, mag = R.matmul(val(s["a"]), R.tile_values(*w.dn_f), off)
    _close(s["y"][live], ref[live], mag[live], I)
    ref, mag = R.unpermute(s["y"], s["sort"], s["gate"], x)
    assert ((out.double() - ref).abs() <= (k + 2) * 2.0 ** -24 * mag * 1.01 + R.half_eps(BF) * ref.abs() * 1.01).all()

    g = backward(dout, s, E, w)
    ref, mag = R.matmul(val(g["dyq"]), R.tile_values(*w.dn_b), off)
    _close(g["da"][live], ref[live], mag[live], H)
    ref, mag = R.matmul(val(mok.fp8_quantize(g["dh"][None])), R.tile_values(*w.gu_b), off)
    _close(g["drows"][live], ref[live], mag[live], 2 * I)
    most = int((off[1:] - off[:-1]).max())
    _close(g["dgu"], *R.wgrad(val(g["xt"]), val(g["dht"]), off), most)
    _close(g["ddn"], *R.wgrad(val(g["at"]), val(g["dyt"]), off), most)
    ref, mag = R.unpermute(g["drows"], s["sort"])
    assert ((g["dx"].double() - ref).abs() <= (k + 2) * 2.0 ** -24 * mag * 1.01 + R.half_eps(BF) * ref.abs() * 1.01).all()

    # and the whole against the layer in fp64 without any rounding: E4M3 rounds each of a product's operands by up to
    # 2^-4 of a value, about 2^-4 / sqrt(3) in the mean square, and independent errors add as squares along the chain
    gu, dn = w.gu.double(), w.dn.double()
    want = x.double().clone()
    gate, ids = s["gate"].double(), s["ids"].long()
    for j in range(k):
        h = torch.einsum("th,thi->ti", x.double(), gu[ids[:, j]])
        want += gate[:, j, None] * torch.einsum("ti,tih->th", R.glu(h), dn[ids[:, j]])
    rel = float((out.double() - want).norm() / want.norm())
    assert rel <= 4 * 2.0 ** -4 / 3 ** 0.5, rel


def _bits(t):
    return t.contiguous().view(torch.uint8)


def test_graph_replays_give_the_eager_bits():
    T, H, I, E, k = 130, 256, 144, 8, 2
    x, logits, dout = _inputs(T, H, E, 3)
    w = Experts(E, H, I, 9)

    def step():
        out, s = forward(x, logits, k, w)
        return dict(out=out, **{n: v for n, v in backward(dout, s, E, w).items() if n in
                                ("dx", "dlogits", "dgate", "dgu", "ddn")})
    eager = {n: v.clone() for n, v in step().items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for rep in range(3):
        x0 = x.clone()
        if rep == 1:        # other inputs: the replay follows them
            x.copy_(x0.flip(0))
        want = {n: v.clone() for n, v in step().items()}      # eager work between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(_bits(got[n]), _bits(want[n])), (rep, n)
        if rep != 1:
            for n in want:
                assert torch.equal(_bits(want[n]), _bits(eager[n])), (rep, n)
        x.copy_(x0)


def test_two_streams_at_once():
    T, H, I, E, k = 200, 256, 128, 8, 2
    w = Experts(E, H, I, 5)
    ins = [_inputs(T, H, E, 10 + i) for i in range(2)]
    want = [forward(x, lg, k, w)[0].clone() for x, lg, _ in ins]
    streams = [torch.cuda.Stream() for _ in ins]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(forward(ins[i][0], ins[i][1], k, w)[0])
    torch.cuda.synchronize()
    for i in range(2):
        for o in got[i]:
            assert torch.equal(_bits(o), _bits(want[i]))


def test_the_parts_agree_with_the_fused_layer():
    """The same routing and BF16 weights through the fused layer: the parts' 8-bit
    products stay within the rounding of their operands of it."""
    T, H, I, E, k = 96, 256, 128, 4, 2
    x, logits, _ = _inputs(T, H, E, 4)
    w = Experts(E, H, I, 6)
    out, s = forward(x, logits, k, w)
    c = mok.MoKConfig(minibatch_rows=64, ring_bytes=1 << 20)
    ws = mok.get_workspace(c, device=DEV, num_local_tokens=T, hidden_size=H, intermediate_size=I, num_experts=E, topk=k)
    wts = mok.weights_bf16(w.gu[:, :, :I].contiguous(), w.gu[:, :, I:].contiguous(), w.dn)
    fused, _ = mok.forward(ws, mok.build_schedule(ws, s["ids"]), x, s["gate"], wts)
    rel = float((out.double() - fused.double()).norm() / fused.double().norm())
    assert rel <= 4 * 2.0 ** -4 / 3 ** 0.5, rel      # four 8-bit operands on the way, 2^-4 / sqrt(3) each
