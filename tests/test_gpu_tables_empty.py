"""The device-built tables of a step without sequences."""
import pytest

from fp4_harness import i32, no_error, takes_error
from paged_sliding_window_gb300 import binding
from test_gpu_tables_ends import call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_slots", [0, 20, 5000])
def test_two_cursors_in_turn_over_a_step_without_sequences(n_slots):
    """The second cursor is what the first was, so no page is handed out twice."""
    free, a, b = i32(range(10, 20)), i32([2]), i32([0])
    assert call([0], [17], 3, free, a, b)[0] == [[12, 13, -1]]
    got = call([], [], 3, free, b, a, n_slots)
    no_error()
    assert a.tolist() == b.tolist() == [4] and got == ([], [0], [], [-9] * n_slots)
    assert call([0], [17], 3, free, a, b)[0] == [[14, 15, -1]]
    no_error()
    assert b.tolist() == [6]


def test_a_bad_cursor_over_a_step_without_sequences():
    free, a, b = i32([3, 4]), i32([7]), i32([0])
    call([], [], 3, free, a, b)
    takes_error(binding.DEVERR_LENGTH)
    assert b.tolist() == [2]


def test_one_cursor_over_a_step_without_sequences():
    free, a = i32(range(10)), i32([3])
    call([], [], 3, free, a, a)
    no_error()
    assert a.tolist() == [3]
