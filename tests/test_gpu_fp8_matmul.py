"""Products on operands in blocks of 128 on the GPU, against fp64 of the same codes."""
import pytest
import torch

import mixture_experts_layer_table_amd as mok
import routed_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def _codes(shape, seed, scales, spread=2.0):
    """Random finite E4M3 codes and positive scales of very different sizes."""
    g = torch.Generator().manual_seed(seed)
    el = torch.randint(0, 256, shape, generator=g).to(torch.uint8)
    el = torch.where((el & 0x7F) == 0x7F, torch.zeros_like(el), el)
    return el.to(DEV), torch.exp(spread * torch.randn(scales, generator=g)).to(DEV)


def rows(n, K, seed):
    return _codes((n, K), seed, (-(-K // 128), n))


def tiles(lead, n, K, seed):
    return _codes(lead + (n, K), seed, lead + (-(-n // 128), -(-K // 128)))


def check(got, ref, mag, K):
    assert R.product_errors(got, ref, mag, K) is None, R.product_errors(got, ref, mag, K)


# M, N, K: one row to several tiles, ragged rows, N past whole tiles and not a multiple of 128, K with a shorter last
# block and of a single short one
DENSE = [(1, 16, 16), (1, 256, 128), (2, 4096, 512), (7, 272, 144), (16, 1040, 2048), (33, 128, 7168), (64, 512, 400),
         (100, 48, 256), (129, 576, 1040), (256, 256, 256), (257, 784, 128), (300, 2064, 64), (513, 512, 528),
         (1000, 272, 1424)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,N,K", DENSE)
def test_dense(M, N, K, dtype):
    print(f"[matmul] {M} {N} {K} {dtype}", flush=True)
    a, b = rows(M, K, M + K), tiles((), N, K, N)
    got = mok.fp8_matmul(a, b, out_dtype=dtype)
    assert got.dtype == dtype
    check(got, *R.matmul(R.row_values(*a), R.tile_values(*b)), K)
    # the same call again: the same bits
    again = mok.fp8_matmul(a, b, out_dtype=dtype)
    assert torch.equal(got.view(torch.uint8), again.view(torch.uint8))


# rows of each expert: none first, none last, one row, all in one, ragged, many experts (past 64 in one scan)
GROUPED = [([0, 5, 0, 130, 1, 0], 272, 400), ([300], 256, 128), ([0, 0, 0], 64, 64), ([1] * 8, 4096, 1024),
           ([7, 0, 19, 33, 64, 2, 0, 16, 17], 528, 2048), ([257, 1, 600, 0, 255], 512, 272), ([3] * 130, 32, 144),
           ([0] * 70 + [9] + [0] * 60 + [40, 2], 48, 256), ([128, 256, 384], 1040, 528)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("counts,N,K", GROUPED)
def test_grouped(counts, N, K, dtype):
    print(f"[grouped] {len(counts)} {sum(counts)} {N} {K} {dtype}", flush=True)
    first, behind = 3, 5                       # rows of no expert ahead and behind
    off = torch.tensor([0] + counts).cumsum(0).int() + first
    M, E = int(off[-1]) + behind, len(counts)
    a, b = rows(M, K, M), tiles((E,), N, K, N)
    out = torch.full((M, N), 7.0, dtype=dtype, device=DEV)
    got = mok.fp8_matmul(a, b, off.to(DEV), out=out)
    ref, mag = R.matmul(R.row_values(*a), R.tile_values(*b), off)
    inside = slice(first, M - behind)
    check(got[inside], ref[inside], mag[inside], K)
    assert (got[:first] == 7.0).all() and (got[M - behind:] == 7.0).all()


@pytest.mark.parametrize("M,N,K", [(1, 64, 256), (40, 272, 528), (300, 512, 384)])
def test_one_expert_is_the_dense_product(M, N, K):
    a, b = rows(M, K, 1), tiles((1,), N, K, 2)
    off = torch.tensor([0, M]).int().to(DEV)
    one, dense = mok.fp8_matmul(a, b, off, out_dtype=F32), mok.fp8_matmul(a, b, out_dtype=F32)
    ref, mag = R.matmul(R.row_values(*a), R.tile_values(b[0][0], b[1][0]))
    check(one, ref, mag, K)
    check(dense, ref, mag, K)


def test_offsets_outside_the_rows_count_as_the_nearest_inside():
    a, b = rows(40, 128, 3), tiles((3,), 64, 128, 4)
    off = torch.tensor([-9, 10, 35, 2 ** 31 - 1]).int()
    got = mok.fp8_matmul(a, b, off.to(DEV), out_dtype=F32)
    check(got, *R.matmul(R.row_values(*a), R.tile_values(*b), torch.tensor([0, 10, 35, 40])), 128)


# N, K, R: one block, short last blocks, several tiles either way
WGRAD = [(16, 16, 16), (128, 256, 128), (272, 144, 400), (256, 512, 1040), (528, 272, 64), (1040, 528, 2048)]


@pytest.mark.parametrize("addend", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,K,rows_", WGRAD)
def test_wgrad(N, K, rows_, dtype, addend):
    print(f"[wgrad] {N} {K} {rows_} {dtype} {addend}", flush=True)
    dy, x = rows(N, rows_, 5), rows(K, rows_, 6)
    add = torch.randn(N, K, device=DEV).to(dtype) if addend else None
    got = mok.fp8_wgrad(dy, x, out_dtype=dtype, addend=add)
    check(got, *R.wgrad(R.row_values(*dy), R.row_values(*x), addend=add), rows_)
    if addend:
        same = mok.fp8_wgrad(dy, x, out_dtype=dtype, addend=add, out=add)
        assert same is add and torch.equal(same.view(torch.uint8), got.view(torch.uint8))


# blocks of 128 rows of each expert, the last one's run possibly shorter
@pytest.mark.parametrize("dtype,addend", [(BF, False), (F32, True), (BF, True)])
@pytest.mark.parametrize("blocks,short,N,K", [([0, 1, 0, 3], 0, 272, 144), ([2, 5, 1], 64, 256, 528), ([1] * 9, 16, 64, 64),
                                              ([0, 0], 0, 32, 48), ([0] * 66 + [2, 1], 0, 48, 32)])
def test_wgrad_grouped(blocks, short, N, K, dtype, addend):
    off = torch.tensor([0] + blocks).cumsum(0).int() * 128
    if short:
        off[-1] -= 128 - short
    rows_ = max(int(off[-1]), 16) + 16        # codes of no expert behind the last run
    dy, x = rows(N, rows_, 7), rows(K, rows_, 8)
    add = torch.randn(len(blocks), N, K, device=DEV).to(dtype) if addend else None
    got = mok.fp8_wgrad(dy, x, off.to(DEV), out_dtype=dtype, addend=add)
    longest = max(b * 128 for b in blocks + [1])
    check(got, *R.wgrad(R.row_values(*dy), R.row_values(*x), off, add), longest)


def test_nan_codes_reach_their_rows_and_columns_alone():
    a, b = rows(70, 384, 9), tiles((), 80, 384, 10)
    a[0][33, 200] = 0x7F
    b[0][5, 100] = 0xFF
    got = mok.fp8_matmul(a, b, out_dtype=F32)
    nan = torch.isnan(got)
    want = torch.zeros_like(nan)
    want[33] = True
    want[:, 5] = True
    assert torch.equal(nan, want)
    dy, x = rows(48, 256, 11), rows(64, 256, 12)
    dy[0][40, 255] = 0x7F
    nan = torch.isnan(mok.fp8_wgrad(dy, x, out_dtype=F32))
    assert nan[40].all() and int(nan.sum()) == 64


def test_small_scales_do_not_vanish():
    # both scales at their least: 2^-122 / 448^2 is still a normal number
    a, b = rows(4, 128, 13), tiles((), 32, 128, 14)
    a[1].fill_(2.0 ** -52 / 448)
    b[1].fill_(2.0 ** -52 / 448)
    a[0].fill_(0x7E)
    b[0].fill_(0x7E)                            # 448 everywhere
    got = mok.fp8_matmul(a, b, out_dtype=F32)
    assert ((got.double() / (128 * 2.0 ** -104) - 1).abs() <= 2.0 ** -20).all()


def test_no_rows():
    a, b = rows(0, 128, 15), tiles((), 32, 128, 16)
    assert mok.fp8_matmul(a, b).shape == (0, 32)
    dy, x = rows(32, 0, 17), rows(48, 0, 18)
    assert (mok.fp8_wgrad(dy, x) == 0).all()
    add = torch.randn(32, 48, device=DEV).to(BF)
    assert torch.equal(mok.fp8_wgrad(dy, x, addend=add), add)
