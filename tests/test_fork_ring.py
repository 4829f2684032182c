"""The oracle of the forks, pinned by hand where the ring is full: pages that a call takes make room
for those that it returns."""
import numpy as np

from oracle import block_oracle as BO


def test_a_full_ring_takes_back_as_many_pages_as_it_gave():
    table = [[3, 4, -1, -1], [0, 1, 2, 5]]             # 20 and 64 tokens, pages of 16
    ring, state = np.array([8, 9, 6, 7]), [2, 4]       # 6, 7, 8, 9 in order
    got = BO.fork([0, 0, 0, 0, 0], [20, 64], 16, 10, ring, state, np.array(table))
    assert got["block_table"].tolist() == [[3, p, -1, -1] for p in (4, 6, 7, 8, 9)]
    assert got["free_state"].tolist() == [2, 4, 0] and got["free_pages"].tolist() == [2, 5, 0, 1]


def test_what_does_not_fit_is_dropped():
    table = [[3, 4, -1, -1], [0, 1, 2, 5]]
    ring, state = np.array([8, 9, 6, 7]), [2, 4]
    got = BO.fork([0, 0, 0], [20, 64], 16, 10, ring, state, np.array(table))     # two taken, four returned
    assert got["free_state"].tolist() == [0, 4, 0] and got["free_pages"].tolist() == [8, 9, 0, 1]
