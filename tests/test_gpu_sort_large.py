"""Sort of token slots at the most rows that 32-bit tables hold, on the GPU."""
import pytest
import torch

import mixture_experts_layer_table_amd as mok

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_rounding_up_next_to_the_limit():
    # the expert's rows plus align - 1 pass 2^31, its rows rounded up do not
    T, align, away = 2147483000, 1000, 5
    assert mok.sort_rows(T, 1, 1, align) == T
    print("[sort] limit", T, align, flush=True)
    ids = torch.zeros(T, 1, dtype=torch.int32, device=DEV)
    ids[away] = -1
    got = mok.sort_tokens(ids, 1, align)
    assert got["offsets"].tolist() == [0, T]
    slots, row_slots = got["slots"].view(-1), got["row_slots"]
    for f0 in range(0, T, 1 << 28):
        f = torch.arange(f0, min(f0 + (1 << 28), T), dtype=torch.int32, device=DEV)
        row = f - (f > away).int()
        row[f == away] = -1
        assert torch.equal(slots[f0:f0 + f.numel()], row), f0
        slot = f + (f >= away).int()
        slot[f == T - 1] = -1              # the padding row
        assert torch.equal(row_slots[f0:f0 + f.numel()], slot), f0
