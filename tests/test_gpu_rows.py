"""Rows into their experts' order and back on the GPU, against fp64."""
import pytest
import torch

import mixture_experts_layer_table_amd as mok
import routed_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32

# T, H, E, k, align, share of slots without an expert: one token, odd widths, more than 8 slots, several strips of
# a row, all slots elsewhere, an expert twice in a token (the ids are drawn with repeats)
CASES = [(1, 64, 1, 1, 1, 0.0), (1, 7168, 256, 8, 1, 0.0), (5, 8, 3, 2, 4, 0.3), (33, 2056, 8, 3, 16, 0.3),
         (77, 4096, 8, 2, 128, 0.25), (130, 7168, 16, 8, 16, 0.0), (40, 136, 20, 11, 1, 0.2), (9, 512, 4, 17, 128, 0.5),
         (20, 256, 4, 2, 8, 1.0), (3, 20480, 2, 1, 1, 0.0)]


def _case(T, H, E, k, align, away, seed=0):
    g = torch.Generator().manual_seed(T * 7 + H + seed)
    ids = torch.randint(0, E, (T, k), generator=g).int()
    ids = torch.where(torch.rand(T, k, generator=g) < away, -1, ids)
    s = R.sort(ids, E, align)
    return g, {n: t.to(DEV) for n, t in s.items()}


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(dtype).to(DEV)


def _bits(t):
    return t.view(torch.int16 if t.dtype == BF else torch.int32)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", CASES)
def test_permute(case, dtype):
    print(f"[permute] {case} {dtype}", flush=True)
    g, s = _case(*case)
    x = _randn(g, case[:2], dtype)
    n, end = s["row_slots"].numel(), int(s["offsets"][-1])
    rows = torch.full((n, case[1]), 7.0, dtype=dtype, device=DEV)
    got = mok.permute(x, s, outs=dict(rows=rows))["rows"]
    want = R.permute(x, s)
    assert torch.equal(got[:end].double(), want[:end])
    assert (got[end:] == 7.0).all()          # behind the last run: as it was


@pytest.mark.parametrize("rows_too", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", [c for c in CASES if c[1] % 16 == 0])
def test_permute_quantized(case, dtype, rows_too):
    g, s = _case(*case)
    x = _randn(g, case[:2], dtype)
    x[0] = 0.0
    n, H, end = s["row_slots"].numel(), case[1], int(s["offsets"][-1])
    outs = dict(rows=torch.full((n, H), 7.0, dtype=dtype, device=DEV),
                elems=torch.full((n, H), 9, dtype=torch.uint8, device=DEV),
                scales=torch.full((-(-H // 128), n), 5.0, device=DEV))
    got = mok.permute(x, s, rows=rows_too, fp8=True, outs=outs)
    # the same codes as quantizing the sorted rows: a padding row is a row of zeros
    el, sc = mok.fp8_quantize(R.permute(x, s).to(dtype)[None])
    assert torch.equal(got["elems"][:end], el[0, :end]) and torch.equal(got["scales"][:, :end], sc[0, :, :end])
    assert (got["elems"][end:] == 9).all() and (got["scales"][:, end:] == 5.0).all()
    if rows_too:
        assert torch.equal(got["rows"][:end].double(), R.permute(x, s)[:end])
    else:
        assert "rows" not in got and (outs["rows"] == 7.0).all()


def _check_sum(got, ref, mag, k, dtype):
    # k products and k additions (and the addend's) in fp32, then one rounding
    bound = (k + 2) * 2.0 ** -24 * mag * 1.01 + R.half_eps(dtype) * ref.abs() * 1.01 + 1e-37
    bad = (got.double() - ref).abs() > bound
    assert not bad.any(), int(bad.sum())


@pytest.mark.parametrize("weights,addend", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", CASES)
def test_unpermute(case, dtype, weights, addend):
    g, s = _case(*case)
    T, H, k = case[0], case[1], case[3]
    y = _randn(g, (s["row_slots"].numel(), H), dtype)
    y[s["row_slots"] < 0] = float("nan")       # rows without a slot are not read
    w = torch.rand(T, k, generator=g).to(DEV)
    w = torch.where(s["slots"] < 0, float("nan"), w) if weights else None   # nor the weights of slots without a row
    add = _randn(g, (T, H), dtype) if addend else None
    got = mok.unpermute(y, s, w, add)
    ref, mag = R.unpermute(y, s, w, add)
    _check_sum(got, ref, mag, k, dtype)
    if addend:
        same = mok.unpermute(y, s, w, add, out=add)
        assert same is add and torch.equal(_bits(same), _bits(got))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", CASES)
def test_permute_backward(case, dtype):
    g, s = _case(*case)
    d = _randn(g, (s["row_slots"].numel(), case[1]), dtype)
    d[s["row_slots"] < 0] = float("inf")
    ref, mag = R.unpermute(d, s)
    _check_sum(mok.permute_backward(d, s), ref, mag, case[3], dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", CASES)
def test_unpermute_backward(case, dtype):
    g, s = _case(*case)
    T, H, E, k = case[:4]
    n, end = s["row_slots"].numel(), int(s["offsets"][-1])
    y, dout, w = _randn(g, (n, H), dtype), _randn(g, (T, H), dtype), torch.rand(T, k, generator=g).to(DEV)
    grads = dict(dy=torch.full((n, H), 7.0, dtype=dtype, device=DEV), dw=torch.full((T, k), 7.0, device=DEV))
    got = mok.unpermute_backward(dout, y, s, w, grads=grads)
    dy, dw, mag = R.unpermute_backward(dout, y, s, w)
    assert ((got["dy"][:end].double() - dy[:end]).abs() <=
            (R.half_eps(dtype) + (2.0 ** -24 if dtype == BF else 0)) * dy[:end].abs() * 1.01 + 1e-37).all()
    assert (got["dy"][end:] == 7.0).all()
    # a thread's products in a chain of 8 for each of its chunks, then 6 steps of lanes and 4 waves
    steps = 8 * -(-H // 2048) + 16
    assert ((got["dw"].double() - dw).abs() <= steps * 2.0 ** -24 * mag * 1.01 + 1e-37).all()
    # in place of y, the same bits
    again = mok.unpermute_backward(dout, y, s, w, grads=dict(dy=y, dw=torch.empty_like(w)))
    assert torch.equal(_bits(again["dy"][:end]), _bits(got["dy"][:end])) and torch.equal(again["dw"], got["dw"])


def test_no_tokens_and_no_rows():
    s = mok.sort_tokens(torch.empty((0, 2), dtype=torch.int32, device=DEV), 4, 16)
    x = torch.empty((0, 64), dtype=BF, device=DEV)
    assert mok.permute(x, s)["rows"].shape == (0, 64)
    assert mok.unpermute(x, s).shape == (0, 64)
    g = mok.unpermute_backward(x, x, s, torch.empty((0, 2), device=DEV))
    assert g["dy"].shape == (0, 64) and g["dw"].shape == (0, 2)


def test_slots_past_the_rows_count_as_none():
    _, s = _case(12, 64, 3, 2, 1, 0.0)
    s["slots"][3, 1] = 10 ** 6
    s["slots"][4, 0] = -7
    y = torch.randn(s["row_slots"].numel(), 64, device=DEV)
    ref, mag = R.unpermute(y, s)
    _check_sum(mok.unpermute(y, s), ref, mag, 2, F32)
    x = torch.randn(12, 64, device=DEV)
    rows = torch.full_like(y, 3.0)
    mok.permute(x, s, outs=dict(rows=rows))
    lost = [int(r) for r in range(rows.shape[0]) if (rows[r] == 3.0).all()]
    assert len(lost) == 2                      # the rows that the two slots named before


def test_sums_that_cancel_keep_fp32():
    # two slots whose rows differ in the last bits of bf16: the fp32 sum keeps the difference
    s = {n: t.to(DEV) for n, t in R.sort(torch.tensor([[0, 1]]).int(), 2, 1).items()}
    y = torch.tensor([[256.0] * 8, [-255.0] * 8], device=DEV).to(BF)
    w = torch.tensor([[1.0, 1.0 + 2.0 ** -20]], device=DEV)
    want = 256.0 - 255.0 * (1.0 + 2.0 ** -20)
    assert (mok.unpermute(y.float(), s, w).double() - want).abs().max() <= 2.0 ** -23 * 511
