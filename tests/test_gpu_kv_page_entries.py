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
