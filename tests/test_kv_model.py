"""The plain model of the page operators that the GPU tests compare with: its own pins, worked out by
hand, and the counts' consistency over random runs."""
import numpy as np
import pytest
import torch

from tests import kv_model as m


def small():
    # rows 0 and 1: pages 3, 1 (row 1 shares page 3); row 2 empty; 4 tokens a page
    return m.State([[3, 1, -1], [3, 0, -1], [-1, -1, -1]], [7, 5, 0], [1, 1, 0, 2, 0, 0], 4)


def cache(nb, bs=4):
    return [torch.arange(2 * nb * bs, dtype=torch.float32).reshape(2, nb, bs, 1, 1)]


def test_fork_by_hand():
    st = small()
    assert m.fork(st, [0, 0], [2, 1]) == 0
    assert st.table.tolist() == [[3, 1, -1], [3, 1, -1], [3, 1, -1]]
    assert st.seq.tolist() == [7, 7, 7] and st.ref.tolist() == [0, 3, 0, 3, 0, 0]


def test_fork_swap_reads_rows_as_at_entry():
    st = small()
    assert m.fork(st, [0, 1], [1, 0]) == 0
    assert st.table[:2].tolist() == [[3, 0, -1], [3, 1, -1]] and st.seq.tolist() == [5, 7, 0]
    assert st.ref.tolist() == [1, 1, 0, 2, 0, 0]


def test_resize_copies_a_shared_page_and_takes_the_lowest_free():
    st = small()
    assert m.fork(st, [0], [2]) == 0                      # rows 0 and 2 share page 1 (3 tokens in it)
    c = cache(6)
    before = c[0].clone()
    errors, pos, slot = m.resize(st, [2, 0, 1], [9, 8, 0], c)
    # row 1 gives back 3 and 0; row 2: copy of page 1 and one more: the lowest free pages 0 and 2;
    # row 0 still sees page 1 held twice (as after step 1): page 4
    assert errors == 0
    assert st.table.tolist() == [[3, 4, -1], [-1, -1, -1], [3, 0, 2]]
    assert st.seq.tolist() == [8, 0, 9] and st.ref.tolist() == [1, 0, 1, 2, 1, 0]
    assert pos.tolist() == [8, 7, -1] and slot.tolist() == [2 * 4 + 0, 4 * 4 + 3, -1]
    assert torch.equal(c[0][:, 0, :3], before[:, 1, :3]) and torch.equal(c[0][:, 0, 3:], before[:, 0, 3:])


def test_resize_refuses_what_does_not_fit():
    st = small()
    errors, pos, slot = m.resize(st, [2, 1], [12, 9], cache(6))   # 3 + 1 pages wanted, 3 free
    assert errors == 1 and st.seq.tolist() == [7, 5, 12] and pos.tolist() == [11, 4]
    assert st.table[2].tolist() == [2, 4, 5] and slot.tolist() == [5 * 4 + 3, 0]


def test_compact_by_hand():
    st = small()
    c = cache(6)
    before = c[0].clone()
    assert m.compact(st, c) == (0, 3)
    assert st.ref.tolist() == [1, 1, 2, 0, 0, 0] and st.table[:2].tolist() == [[2, 1, -1], [2, 0, -1]]
    assert torch.equal(c[0][:, 2], before[:, 3])


@pytest.mark.parametrize("seed", range(8))
def test_counts_stay_the_rows_entries(seed):
    r = np.random.default_rng(seed)
    R, M, NB, bs = 6, 5, 20, 4
    st = m.State(np.full((R, M), -1), np.zeros(R), np.zeros(NB), bs)
    c = cache(NB)
    for _ in range(30):
        k = r.integers(0, 3)
        if k == 0:
            m.fork(st, r.integers(0, R, 3), r.permutation(R)[:3])
        elif k == 1:
            m.resize(st, r.permutation(R)[:4], r.integers(0, M * bs + 1, 4), c)
        else:
            m.compact(st, c)
        assert st.consistent()
