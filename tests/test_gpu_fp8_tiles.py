"""Each path of the products on blocks of 128 (fp8_shapes.py) on the GPU, against
fp64 of the same codes."""
import pytest
import torch

import mixture_experts_layer_table_amd as mok
import fp8_shapes as S
import routed_reference as R
from test_gpu_fp8_matmul import rows as row_codes, tiles as tile_codes

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def _check(got, ref, mag, K):
    wrong = R.product_errors(got, ref, mag, K)
    assert wrong is None, wrong


@pytest.mark.parametrize("name", list(S.DENSE))
def test_dense(name):
    M, N, K, f32, _ = S.DENSE[name]
    print(f"[tiles] {name}", flush=True)
    a, b = row_codes(M, K, M), tile_codes((), N, K, N)
    got = mok.fp8_matmul(a, b, out_dtype=F32 if f32 else BF)
    _check(got, *R.matmul(R.row_values(*a), R.tile_values(*b)), K)
    assert torch.equal(got.view(torch.uint8), mok.fp8_matmul(a, b, out_dtype=got.dtype).view(torch.uint8))


@pytest.mark.parametrize("name", list(S.GROUPED))
def test_grouped(name):
    counts, N, K, f32, _ = S.GROUPED[name]
    print(f"[tiles] grouped {name}", flush=True)
    off = torch.tensor([0] + counts).cumsum(0).int()
    M, E = int(off[-1]), len(counts)
    a, b = row_codes(M, K, M), tile_codes((E,), N, K, N)
    got = mok.fp8_matmul(a, b, off.to(DEV), out_dtype=F32 if f32 else BF)
    _check(got, *R.matmul(R.row_values(*a), R.tile_values(*b), off), K)
    # the same rows behind and before rows of no expert, which stay as they were
    ahead = 24
    wide = (torch.cat([a[0][:ahead], a[0], a[0][:8]]), torch.cat([a[1][:, :ahead], a[1], a[1][:, :8]], 1).contiguous())
    out = torch.full((M + ahead + 8, N), 5.0, dtype=got.dtype, device=DEV)
    if M >= ahead:
        mok.fp8_matmul(wide, b, (off + ahead).to(DEV), out=out)
        _check(out[ahead:M + ahead], *R.matmul(R.row_values(*a), R.tile_values(*b), off), K)
        assert (out[:ahead] == 5.0).all() and (out[M + ahead:] == 5.0).all()


@pytest.mark.parametrize("addend", [False, True])
@pytest.mark.parametrize("name", list(S.WGRAD))
def test_wgrad(name, addend):
    N, K, counts, f32, _ = S.WGRAD[name]
    print(f"[tiles] wgrad {name} {addend}", flush=True)
    off = torch.tensor([0] + counts).cumsum(0).int() if isinstance(counts, list) else None
    if off is not None:    # runs start at multiples of 128; the last one ends anywhere
        off = torch.tensor([0] + [-(-c // 128) * 128 for c in counts]).cumsum(0).int()
        off[-1] = off[-2] + counts[-1] // 16 * 16
    M = int(off[-1]) if off is not None else counts
    dy, x = row_codes(N, M, 3), row_codes(K, M, 4)
    dtype = F32 if f32 else BF
    lead = (len(counts),) if off is not None else ()
    add = torch.randn(lead + (N, K), device=DEV).to(dtype) if addend else None
    got = mok.fp8_wgrad(dy, x, None if off is None else off.to(DEV), out_dtype=dtype, addend=add)
    longest = int((off[1:] - off[:-1]).max()) if off is not None else M
    _check(got, *R.wgrad(R.row_values(*dy), R.row_values(*x), off, add), longest)
    if addend:             # in place of the addend: the same bits
        same = mok.fp8_wgrad(dy, x, None if off is None else off.to(DEV), addend=add, out=add)
        assert torch.equal(same.view(torch.uint8), got.view(torch.uint8))
