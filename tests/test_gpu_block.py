"""The operators together, as a transformer block's expert half runs them: the
attention branch dropped into the residual stream and normed, the router and
the routed experts on the normed rows, the shared expert added to their output,
and that sum dropped into the stream; then the whole backward. Checked against
the fp64 oracles chained the same way, and captured into a graph."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_table_amd as mok
from gpu_support import DEV, host_f64, status_word
from oracle import block as B
from oracle import layer as L
from test_gpu_dropout import randn, rng_state

pytestmark = pytest.mark.gpu


class Block:
    def __init__(self, mx):
        self.mx = mx
        self.T, self.H, self.I, self.E, self.k = 200, 256, 128, 4, 2
        T, H, I, E = self.T, self.H, self.I, self.E
        s = 500 + mx
        self.res, self.branch, self.dres = randn((T, H), s, scale=2.0), randn((T, H), s + 1), randn((T, H), s + 2)
        self.gamma = (1.0 + 0.2 * randn((H,), s + 3).float()).to(torch.bfloat16)
        self.logits = randn((T, E), s + 4, torch.float32)
        sc = H ** -0.5
        self.we = [randn((E, H, I), s + 5, scale=sc), randn((E, H, I), s + 6, scale=sc),
                   randn((E, I, H), s + 7, scale=I ** -0.5)]
        self.wsh = [randn((H, I), s + 8, scale=sc), randn((H, I), s + 9, scale=sc),
                    randn((I, H), s + 10, scale=I ** -0.5)]
        self.p, self.rng = 0.1, (rng_state(71, 5), rng_state(71, 10 ** 6))
        prec = mok.MOK_MXFP8 if mx else mok.MOK_BF16
        self.ws = mok.get_workspace(mok.MoKConfig(minibatch_rows=64, ring_bytes=1 << 20, precision=prec), device=DEV,
                                    num_local_tokens=T, hidden_size=H, intermediate_size=I, num_experts=E, topk=self.k)
        self.fws = mok.get_ffn_workspace(prec, device=DEV, num_tokens=T, hidden_size=H, intermediate_size=I)
        if mx:
            self.qe = mok.MXFP8Weights(*self.we)
            self.qs = mok.MXFP8Weights(*(w[None] for w in self.wsh))
            self.ew, self.sw = (self.qe.fwd, self.qe.bwd), (self.qs.fwd, self.qs.bwd)
        else:
            self.ew = (mok.weights_bf16(*self.we),) * 2
            self.sw = (mok.weights_bf16(*self.wsh),) * 2

    def step(self):
        n = mok.add_rmsnorm(self.branch, self.gamma, 1e-6, residual=self.res, p=self.p, rng=self.rng[0], mxfp8=self.mx)
        ids, w = mok.route(self.logits, self.k)
        sched = mok.build_schedule(self.ws, ids)
        moe, ctx = mok.forward(self.ws, sched, n["y"], w, self.ew[0])
        rows = (n["y_elems"], n["y_scales"]) if self.mx else n["y"]
        ffn, h = mok.ffn_forward(self.fws, rows, self.sw[0], addend=moe, out=moe)     # on top of the routed output
        out = mok.dropout(ffn, self.rng[1], self.p, residual=n["sum"])
        dffn = mok.dropout_backward(self.dres, self.rng[1], self.p)
        ge = mok.backward(self.ws, sched, ctx, n["y"], w, self.ew[1], dffn)
        dy = ge["dx"]
        gs = mok.ffn_backward(self.fws, n["y"], self.sw[1], h, dffn, addend=dy)
        dl = mok.route_backward(ids, w, ge["dtopk_w"], self.E)
        gn = mok.add_rmsnorm_backward(gs["dx"], n["sum"], self.gamma, n["rstd"], dsum=self.dres, p=self.p,
                                      rng=self.rng[0])
        return dict(out=out, sum=n["sum"], ids=ids, w=w, status=sched, dlogits=dl,
                    dres=gn["dresidual"], dbranch=gn["dx"], dgamma=gn["dweight"],
                    dwd=gs["dw_down"], dwg=gs["dw_gate"], dwu=gs["dw_up"], dwe=ge["dw_down"])


@pytest.mark.parametrize("mx", [False, True])
def test_block_matches_the_chained_oracles(mx):
    print(f"[block] mx={mx}", flush=True)
    b = Block(mx)
    r = b.step()
    torch.cuda.synchronize()
    assert status_word(r["status"]) == 0
    f, fq = host_f64, (B.fake_quant if mx else None)
    lfq = (lambda v, axis: B.fake_quant(v, axis)) if mx else None
    keep = [B.keep_mask(71, off, b.T * b.H, b.p).reshape(b.T, b.H) for off in (5, 10 ** 6)]
    s = f(b.res) + B.dropout(f(b.branch), keep[0], b.p)
    y, rstd = B.rmsnorm(s, f(b.gamma), 1e-6)
    ids, w = r["ids"].cpu().numpy(), r["w"].cpu().numpy()
    We, Ws = [f(t) for t in b.we], [f(t) for t in b.wsh]
    moe, _ = L.forward(y, ids, w, *We, lfq)
    ffn, h, _ = B.ffn(y, *Ws, addend=moe, fq=fq)
    out = s + B.dropout(ffn, keep[1], b.p)
    D = f(b.dres)
    dffn = B.dropout(D, keep[1], b.p)
    ge = L.backward(y, ids, w, *We, dffn, lfq)
    gs = B.ffn_backward(y, *Ws, h, dffn, ge["dx"], fq)
    ds, dgamma = B.rmsnorm_backward(gs["dx"], s, f(b.gamma), rstd, D)
    want = dict(out=out, sum=s, dres=ds, dbranch=B.dropout(ds, keep[0], b.p), dgamma=dgamma, dwd=gs["dw_down"],
                dwg=gs["dw_gate"], dwu=gs["dw_up"], dwe=ge["dWd"])
    # every link rounds rows to bf16 (2^-8 at most) a few times; MXFP8 links add the layer's own 6e-2
    tol = 6e-2 if mx else 2e-2
    errs = {n: L.rel_frobenius(f(r[n]), v) for n, v in want.items()}
    assert all(v < tol for v in errs.values()), errs


@pytest.mark.parametrize("mx", [False, True])
def test_block_replays_from_a_graph(mx):
    b = Block(mx)
    ref = {n: t.clone() for n, t in b.step().items() if n != "status"}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = b.step()
    for rep in range(3):
        eager = b.step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert status_word(got["status"]) == 0
        for n, t in ref.items():
            assert torch.equal(got[n], t) and torch.equal(eager[n], t), (rep, n)
