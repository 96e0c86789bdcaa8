"""The plain implementation of block tables that tests/test_gpu_block_table.py compares with, by hand (no GPU needed)."""
import block_table_ref as ref


def test_pages_return_to_the_places_that_a_step_empties():
    """Four places, all of them free: one sequence takes the four pages, another ends with four. None is lost."""
    w = ref.extend([[-1] * 4, [8, 9, 10, 11]], [0, 8], [8, -1], [4, 5, 6, 7], [2, 4, 0], 2, 8)
    assert w["table"][0] == [6, 7, 4, 5] and w["seq_lens"] == [8, 0]
    assert w["pool"] == [2, 4, 0] and [w["ring"][(2 + i) % 4] for i in range(4)] == [8, 9, 10, 11]
    assert w["slots"] == [12, 13, 14, 15, 8, 9, 10, 11]


def test_pages_beyond_the_ring_are_dropped_from_the_last():
    w = ref.extend([[-1] * 4, [8, 9, 10, 11]], [0, 8], [2, -1], [4, 5, 6], [0, 3, 0], 2, 2)
    assert w["pool"] == [1, 3, 0] and [w["ring"][(1 + i) % 3] for i in range(3)] == [5, 6, 8]


def test_absent_pages_do_not_return():
    """A window has passed the second and third page of a sequence, which were given back: it ends with the other two."""
    w = ref.extend([[8, -1, -7, 11]], [8], [-1], [3, 4, -1, -1], [0, 2, 0], 2, 1)
    assert w["pool"] == [0, 4, 0] and w["ring"] == [3, 4, 8, 11]
