"""Sort of token slots by expert on the GPU: equal to the reference, entry by entry."""
import pytest
import torch

import mixture_experts_layer_table_amd as mok
import routed_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# one launch below 65,536 slots and up to 512 experts, else three
CASES = [(1, 1, 1, 1), (1, 8, 256, 1), (3, 2, 4, 128), (64, 1, 7, 16), (65, 3, 8, 1), (1023, 1, 512, 16),
         (2048, 8, 256, 128), (16384, 1, 4, 128), (2049, 8, 256, 16), (5000, 4, 8, 1024), (300, 8, 513, 3),
         (1, 4, 4096, 1), (163840, 1, 8, 128), (20000, 2, 4096, 1),
         (65535, 1, 8, 16), (65536, 1, 8, 16)]


def _ids(T, k, E, kind):
    g = torch.Generator().manual_seed(T * 31 + E)
    if kind == "one":           # a single expert takes all
        return torch.full((T, k), E - 1, dtype=torch.int32)
    if kind == "none":          # no slot has an expert here
        return torch.where(torch.rand(T, k, generator=g) < 0.5, -1, E).int()
    ids = (torch.rand(T, k, generator=g) ** 2 * E).int().clamp(max=E - 1)
    if kind == "away":
        odd = torch.tensor([-1, E, -2 ** 31, 2 ** 31 - 1]).int()
        gone = torch.rand(T, k, generator=g) < 0.4
        ids = torch.where(gone, odd[torch.randint(0, 4, (T, k), generator=g)], ids)
    return ids


@pytest.mark.parametrize("kind", ["all", "away", "one", "none"])
@pytest.mark.parametrize("T,k,E,align", CASES)
def test_sort_equals_the_reference(T, k, E, align, kind):
    ids = _ids(T, k, E, kind)
    print(f"[sort] {T} {k} {E} {align} {kind}", flush=True)
    got = mok.sort_tokens(ids.to(DEV), E, align)
    want = R.sort(ids, E, align)
    assert mok.sort_rows(T, k, E, align) == want["row_slots"].numel()
    for n in want:
        assert torch.equal(got[n].cpu(), want[n]), n


def test_sort_of_no_tokens():
    for E in (3, 700):
        got = mok.sort_tokens(torch.empty((0, 2), dtype=torch.int32, device=DEV), E, 16)
        assert got["offsets"].tolist() == [0] * (E + 1) and got["row_slots"].numel() == 0


def test_sort_writes_every_entry_of_given_buffers():
    ids = _ids(500, 2, 8, "away").to(DEV)
    outs = dict(offsets=torch.full((9,), 77, dtype=torch.int32, device=DEV),
                slots=torch.full((500, 2), 77, dtype=torch.int32, device=DEV),
                row_slots=torch.full((mok.sort_rows(500, 2, 8, 128),), 77, dtype=torch.int32, device=DEV))
    got = mok.sort_tokens(ids, 8, 128, outs=outs)
    want = R.sort(ids.cpu(), 8, 128)
    for n in want:
        assert got[n] is outs[n] and torch.equal(got[n].cpu(), want[n])
