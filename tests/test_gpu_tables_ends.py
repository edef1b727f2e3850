"""The device-built tables of a step for past lengths at the end of what 32 bits hold."""
import pytest
import torch

from fp4_harness import i32, takes_error
from paged_sliding_window_gb300 import binding

pytestmark = pytest.mark.gpu


def call(past, new, width, free, pos, nxt, n_slots=20):
    n = len(past)
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    cu_new, lens = i32([5] * (n + 1)), i32([5] * n)
    slots = torch.full((n_slots,), -9, dtype=torch.int64, device="cuda")
    binding.block_table_extend(table, i32(past), i32(new), free, pos, nxt, cu_new, lens, slots)
    return table.tolist(), cu_new.tolist(), lens.tolist(), slots.tolist()


@pytest.mark.parametrize("past", [2 ** 31 - 17, 2 ** 31 - 16, 2 ** 31 - 15, 2 ** 31 - 2, 2 ** 31 - 1])
@pytest.mark.parametrize("new", [0, 1, 100])
def test_longest_past(past, new):
    """A past far beyond the row: no page, no id taken, both faults flagged; the sequence beside it as always."""
    pos = i32([0])
    table, cu_new, lens, slots = call([past, 3], [new, 14], 2, i32([8, 9]), pos, pos, n_slots=14)
    fits = past + new <= 2 ** 31 - 1 - 16
    takes_error(binding.DEVERR_CAPACITY | (0 if fits else binding.DEVERR_LENGTH) | binding.DEVERR_BLOCK_ID)
    assert not fits or new == 0
    assert table == [[-1, -1], [-1, 8]] and pos.tolist() == [1]
    assert cu_new == [0, 0, 14] and lens == [past, 17] and slots == [-1] * 13 + [8 * 16]
