"""Where an expert's run of rows may begin and end in a weight gradient on the GPU
(mok_fp8_wgrad), on each of its paths, against fp64 of the same codes."""
import pytest
import torch

import fp8_shapes as S
import mixture_experts_layer_table_amd as mok
import routed_reference as R
from test_gpu_fp8_matmul import rows as row_codes

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32

# the paths of fp8_shapes.py with one run of rows: 256-row tiles, 128-row tiles, runs joined, fp32 results joined
PATHS = ["whole", "tiles_128", "runs", "runs_f32"]


def _case(name):
    N, K, M, f32, _ = S.WGRAD[name]
    return N, K, M, F32 if f32 else BF


def _check(got, ref, mag, longest):
    wrong = R.product_errors(got, ref, mag, longest)
    assert wrong is None, wrong


def _behind(t, end, kind):
    """The codes t [n, M] with those behind `end` as they are, or NaN of either sign."""
    el = t[0].clone()
    if kind != "codes":
        el[:, end:] = 0x7F if kind == "nan" else 0xFF
    return el, t[1]


@pytest.mark.parametrize("kind", ["codes", "nan", "minus nan"])
@pytest.mark.parametrize("end", [1, 15, 17, 100, 130, 255, -1])
@pytest.mark.parametrize("name", PATHS)
def test_a_run_may_end_at_any_row(name, end, kind):
    N, K, M, dtype = _case(name)
    end = end if end > 0 else M + end
    print(f"[runs] end {name} {end} {kind}", flush=True)
    dy, x = _behind(row_codes(N, M, 3), end, kind), _behind(row_codes(K, M, 4), end, kind)
    off = torch.tensor([0, end]).int()
    got = mok.fp8_wgrad(dy, x, off.to(DEV), out_dtype=dtype)
    _check(got, *R.wgrad(R.row_values(*dy), R.row_values(*x), off), end)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("nan_in", ["dy", "x"])
def test_nan_codes_behind_a_run_in_one_operand(nan_in, dtype):
    N, K, M, end = 272, 528, 512, 256 + 77
    dy, x = row_codes(N, M, 5), row_codes(K, M, 6)
    if nan_in == "dy":
        dy = _behind(dy, end, "nan")
    else:
        x = _behind(x, end, "nan")
    off = torch.tensor([0, 128, 128, end]).int()
    add = torch.randn(3, N, K, device=DEV).to(dtype)
    got = mok.fp8_wgrad(dy, x, off.to(DEV), out_dtype=dtype, addend=add)
    _check(got, *R.wgrad(R.row_values(*dy), R.row_values(*x), off, add), end - 128)


def test_a_nan_code_inside_the_last_unit_stays():
    N, K, M, end = 64, 48, 256, 139
    dy, x = row_codes(N, M, 7), row_codes(K, M, 8)
    dy[0][9, end - 1] = 0x7F
    dy[0][10, end] = 0x7F
    nan = torch.isnan(mok.fp8_wgrad(dy, x, torch.tensor([0, end]).int().to(DEV), out_dtype=F32))
    assert nan[0, 9].all() and int(nan.sum()) == K


@pytest.mark.parametrize("addend", [False, True])
@pytest.mark.parametrize("name", PATHS)
def test_an_expert_without_rows_where_another_run_ends(name, addend):
    N, K, M, dtype = _case(name)
    N, K = min(N, 512), min(K, 528)          # several experts' fit the reference; their path may be another
    print(f"[runs] empty {name} {addend}", flush=True)
    dy, x = row_codes(N, M, 9), row_codes(K, M, 10)
    for ends in ([0, 0, 130, 130, 130, 130], [37, 37, 37, 37, 37], [128, 128, 256 + 16, 256 + 16], [M - 16, M - 16]):
        off = torch.tensor(ends).int()
        E = len(ends) - 1
        add = torch.randn(E, N, K, device=DEV).to(dtype) if addend else None
        got = mok.fp8_wgrad(dy, x, off.to(DEV), out_dtype=dtype, addend=add)
        _check(got, *R.wgrad(R.row_values(*dy), R.row_values(*x), off, add), 256)
        for e in range(E):
            if ends[e] == ends[e + 1]:
                assert torch.equal(got[e], add[e]) if addend else (got[e] == 0).all()


@pytest.mark.parametrize("addend", [False, True])
@pytest.mark.parametrize("name", PATHS)
def test_a_run_that_begins_inside_a_block_is_nan(name, addend):
    N, K, M, dtype = _case(name)
    N, K = min(N, 512), min(K, 528)
    print(f"[runs] start {name} {addend}", flush=True)
    dy, x = row_codes(N, M, 11), row_codes(K, M, 12)
    ends = [0, 100, 256, 300, 301, 301, 384]
    off, E = torch.tensor(ends).int(), len(ends) - 1
    add = torch.randn(E, N, K, device=DEV).to(dtype) if addend else None
    got = mok.fp8_wgrad(dy, x, off.to(DEV), out_dtype=dtype, addend=add)
    ref, mag = R.wgrad(R.row_values(*dy), R.row_values(*x), off, add)
    for e in range(E):
        if ends[e] % 128 and ends[e + 1] > ends[e]:
            assert torch.isnan(got[e]).all(), e
        else:
            _check(got[e], ref[e], mag[e], 128)
