"""kvq8_paged_tables: what of held and free pages makes a call malformed: more free and given back than there are."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from ._paged import i32  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("count,lens,status", [(6, [32, 48], 0), (8, [32, 48], 0), (8, [16, 48], 2), (7, [16, 48], 0), (6, [0, 48], 0), (7, [0, 48], 2)])
def test_pages_that_stay_held_are_not_counted(lib, count, lens, status):
    from speculative_verify_attention_gb300 import kvq8_paged_tables
    held, table, ring = i32([2, 3]), i32([[0, 1, 9], [2, 3, 4]]), i32(np.arange(8))
    state, starts, out = i32([0, count]), i32([7, 7, 7]), i32([9])
    slots, pos = torch.zeros(2, dtype=torch.int64, device="cuda"), i32([5, 5])
    kvq8_paged_tables(i32(lens), i32([0, 2]), held, table, ring, state, 16, starts, slots, pos, out)
    assert out.item() == status
    if status:
        assert slots.tolist() == [-1, -1] and held.tolist() == [2, 3] and state.tolist() == [0, count]
    else:
        assert slots.tolist() == [4 * 16 + 14, 4 * 16 + 15] and held.tolist() == [lens[0] // 16, 3]
        assert state.tolist() == [0, count + 2 - lens[0] // 16]
