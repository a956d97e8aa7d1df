"""GPU: entries of the page operators that sra.h names one by one: what is padding, what counts as an error, what
a refused entry leaves to the ones behind it. Expected states are written out, not computed by a model."""
import numpy as np
import pytest
import torch

import swiglu_rmsnorm_add_gb300 as sra

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BIG = 2 ** 31 - 1


def i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).to(DEV)


def test_copy_counts_every_pair_out_of_range():
    """Also one whose source and destination are the same index; equal indexes in range are nothing to do."""
    nb = 6
    cache = torch.randn(2, nb, 4, 1, 8, device=DEV)
    want = cache.clone()
    want[:, 3] = want[:, 0]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    sra.copy_kv_pages(cache, i32([nb, 0, BIG, 2, -1, nb + 1]), i32([nb, 3, BIG, 2, -1, -1]), err_count=err)
    assert torch.equal(cache, want)
    assert int(err.item()) == 2


@pytest.mark.parametrize("cols", [4, 8192])     # all entries in one CTA, and a grid of them
def test_a_padding_entry_names_no_child(cols):
    """An entry with a negative index in either array does nothing, also to a later entry for the same child; one
    that is refused for another reason has named its child."""
    table = np.full((8, cols), -1)
    table[0, :2], table[1, :1] = [0, 1], [2]
    seq, ref = [7, 3, 0, 0, 0, 0, 0, 0], [1, 1, 1, 0, 0]
    t, s, r = i32(table), i32(seq), i32(ref)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    #                            padding  done  refused: parent, then its child again  padding  done
    sra.fork_kv_rows(t, s, r, i32([-1, 0, 8, 1, -7, 0]), i32([2, 2, 4, 4, 5, 5]), 4, err_count=err)
    for row in (2, 5):
        table[row, :2] = [0, 1]
    assert t.cpu().tolist() == table.tolist()
    assert s.tolist() == [7, 3, 7, 0, 0, 7, 0, 0] and r.tolist() == [3, 3, 1, 0, 0]
    assert int(err.item()) == 2
    # the same child twice: the first entry is done, the second refused
    sra.fork_kv_rows(t, s, r, i32([1, 0]), i32([6, 6]), 4, err_count=err)
    assert s.tolist() == [7, 3, 7, 0, 0, 7, 3, 0] and int(err.item()) == 3


def test_a_row_that_needs_no_page_is_served_behind_a_refused_one():
    """Three free pages and rows that ask for five, for none (inside a last page of its own), for one, and, last, for none:
    the first and the third are refused, the others grow."""
    table = np.full((4, 8), -1)
    table[0, :1], table[1, :2], table[2, :1], table[3, :1] = [6], [0, 1], [2], [3]
    seq, ref = [4, 5, 4, 2], [1, 1, 1, 1, 0, 0, 1, 0]
    t, s, r = i32(table), i32(seq), i32(ref)
    cache = torch.zeros(2, 8, 4, 1, 8, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pos, slot = sra.resize_kv_rows(t, s, r, i32([0, 1, 2, 3]), i32([24, 6, 5, 4]), cache, err_count=err)
    assert t.cpu().tolist() == table.tolist() and r.tolist() == ref
    assert s.tolist() == [4, 6, 4, 4] and int(err.item()) == 2
    assert pos.tolist() == [3, 5, 3, 3] and slot.tolist() == [6 * 4 + 3, 1 * 4 + 1, 2 * 4 + 3, 3 * 4 + 3]
