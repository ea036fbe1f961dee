"""Row kernels of more workgroups than one launch takes (2^23) on the GPU: what the
later launches write is held to the same rows in small calls, or to indexing."""
import pytest
import torch

import mixture_experts_layer_table_amd as mok

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16
GROUPS = 1 << 23


@pytest.fixture(autouse=True)
def _give_back():
    yield
    torch.cuda.empty_cache()


def _tokens(T, H, k, E, align):
    g = torch.Generator(DEV).manual_seed(T)
    ids = torch.randint(-1, E, (T, k), generator=g, device=DEV, dtype=torch.int32)
    x = torch.randn(T, H, generator=g, device=DEV).to(BF)
    return x, mok.sort_tokens(ids, E, align)




def test_permute_and_back():
    T, H = GROUPS + 1000, 8
    x, s = _tokens(T, H, 1, 2, 16)
    print("[large] permute", T, flush=True)
    src, end = s["row_slots"].long(), int(s["offsets"][-1])
    want = torch.where(src[:, None] >= 0, x[src.clamp(min=0)], torch.zeros((), dtype=BF, device=DEV))[:end]
    rows = mok.permute(x, s)["rows"]
    assert torch.equal(rows[:end], want)
    # k = 1 without weights: the token's row, or nothing
    here = s["slots"] >= 0
    back = torch.where(here, x, torch.zeros((), dtype=BF, device=DEV))
    assert torch.equal(mok.unpermute(rows, s), back) and torch.equal(mok.permute_backward(rows, s), back)
    w = torch.full((T, 1), 0.5, device=DEV)
    g = mok.unpermute_backward(x, rows, s, w)
    assert torch.equal(g["dy"][:end], (want.float() * 0.5).to(BF))
    dw = (x.float() * x.float()).sum(1, keepdim=True) * here
    assert ((g["dw"] - dw).abs() <= 8 * 2.0 ** -22 * dw).all()     # 8 terms, either order


def test_permute_to_8_bits():
    T, H = GROUPS + 1000, 16
    x, s = _tokens(T, H, 1, 2, 16)
    got = mok.permute(x, s, rows=False, fp8=True)
    src, end = s["row_slots"].long()[:int(s["offsets"][-1])], int(s["offsets"][-1])
    el, sc = mok.fp8_quantize(x[None])
    pad = mok.fp8_quantize(torch.zeros(1, 1, H, dtype=BF, device=DEV))
    hit = src >= 0
    assert torch.equal(got["elems"][:end], torch.where(hit[:, None], el[0][src.clamp(min=0)], pad[0][0]))
    assert torch.equal(got["scales"][0, :end], torch.where(hit, sc[0, 0][src.clamp(min=0)], pad[1][0, 0]))


# a workgroup takes 16 rows, or 128 rows of a tile
@pytest.mark.parametrize("form,rows_each", [("rows", 16), ("tile", 128), ("turned", 128), ("turned tile", 128)])
def test_quantize(form, rows_each):
    K, part = 16, 4096
    times = GROUPS * rows_each // part + 1
    if torch.cuda.mem_get_info()[0] < 5 * times * part * K:
        pytest.skip("not enough memory")
    print("[large] quantize", form, times * part, flush=True)
    v = torch.randn(part, K, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    turned, tile = "turned" in form, "tile" in form
    one = v.t().contiguous() if turned else v
    el, sc = mok.fp8_quantize(one[None], turned, tile=tile)
    src = one.repeat((1, times) if turned else (times, 1))[None]
    big, bsc = mok.fp8_quantize(src, turned, tile=tile)
    del src
    assert (big.view(times, part * K) == el.view(1, part * K)).all()
    assert (bsc.view(times, -1) == sc.view(1, -1)).all()


def test_glu_backward():
    part, I = 4096, 4096
    times = GROUPS * 256 * 8 // (part * I) + 1
    if torch.cuda.mem_get_info()[0] < 8 * times * part * I:
        pytest.skip("not enough memory")
    print("[large] glu", times * part, flush=True)
    g = torch.Generator(DEV).manual_seed(2)
    da, h = (torch.randn(part, n, generator=g, device=DEV).to(BF) for n in (I, 2 * I))
    want = mok.glu_backward(da, h)
    hh = h.repeat(times, 1)
    got = mok.glu_backward(da.repeat(times, 1), hh, dh=hh)
    for i in range(0, times, 64):
        assert (got[i * part:(i + 64) * part].view(-1, part, 2 * I) == want).all(), i
