"""GPU: the read back with lengths and starts that point anywhere: every row of the results, the rows around them and the
error count against the definition.

A result row i with cu_lens[0] <= i < cu_lens[rows] belongs to the last table row r with cu_lens[r] <= i and is its token
starts[r] + i - cu_lens[r]; a token outside of the table, or on a page out of range, is zeros. Of lengths that do not fall the
count is one for each bad entry that holds a token asked for and one for each row that asks for tokens outside of its table.
"""
import numpy as np
import pytest
import torch

import swiglu_rmsnorm_add_gb300 as sra
from tests import quant_model as qm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
N_KV, HD, BS, NB, MB, TOTAL = 2, 64, 8, 9, 4, 48
BIG = 2 ** 31 - 1


def i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).to(DEV)


def cache_of(fmt, seed):
    x = np.random.default_rng(seed).standard_normal((2, NB, N_KV, BS, HD)).astype(np.float32)
    return qm.encode(x.astype(np.float64), fmt)


def expected(cache, fmt, table, cu, starts):
    """([2, TOTAL, N_KV, HD] with NaN where nothing is written, errors)."""
    out = np.full((2, TOTAL, N_KV, HD), np.nan)
    bad, outside = set(), set()
    for i in range(max(cu[0], 0), min(cu[-1], TOTAL)):
        r = max(k for k in range(len(cu) - 1) if cu[k] <= i)
        tok = (starts[r] if starts is not None else 0) + i - cu[r]
        out[:, i] = 0
        if not 0 <= tok < MB * BS:
            outside.add(r)
        elif not 0 <= table[r, tok // BS] < NB:
            bad.add((r, tok // BS))
        else:
            out[:, i] = qm.decode(cache[:, table[r, tok // BS], :, tok % BS], fmt, HD)
    return out, len(bad) + len(outside)


def check(fmt, dtype, table, cu, starts, ordered=True):
    cache = cache_of(fmt, 1)
    W, guard = N_KV * HD, 40
    buf = torch.full((2, TOTAL + 2 * guard, W), -9.0, dtype=dtype, device=DEV)
    k, v = (buf[p, guard:guard + TOTAL].unflatten(1, (N_KV, HD)) for p in (0, 1))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    sra.read_kv_quant(torch.tensor(cache).to(DEV), i32(table), i32(cu), TOTAL, HD, starts=None if starts is None else i32(starts),
                      out=(k, v), err_count=err)
    got = buf.double().cpu().numpy()
    assert (got[:, :guard] == -9).all() and (got[:, guard + TOTAL:] == -9).all(), "outside of the results"
    got = got[:, guard:guard + TOTAL].reshape(2, TOTAL, N_KV, HD)
    inside = (np.arange(TOTAL) >= cu[0]) & (np.arange(TOTAL) < cu[-1])
    assert (got[:, ~inside] == -9).all(), "rows of nobody"
    if ordered:
        want, errors = expected(cache, fmt, table, cu, starts)
        want = np.where(np.isnan(want), -9.0, qm.rounded(np.nan_to_num(want), dtype))
        assert np.array_equal(got, want), np.argwhere(got != want)[0].tolist()
        assert int(err.item()) == errors


def random_table(seed, rows, bad=0):
    r = np.random.default_rng(seed)
    table = r.integers(0, NB, (rows, MB))
    table.flat[r.permutation(rows * MB)[:bad]] = r.choice([-1, NB, BIG, -BIG - 1], bad)
    return table


@pytest.mark.parametrize("cu,starts", [
    ([0, 10, 20], [-5, BIG]), ([0, 10, 20], [-5, 3]), ([0, 12, 30, 48], [-9, -1, 27]), ([3, 47], [-4]), ([0, 48], [-8]),
    ([0, 9, 18], [-BIG - 1, 31]), ([0, 9, 18], [32, 33]), ([0, 0, 7, 7, 40], [-3, -3, 5, 1])])
@pytest.mark.parametrize("fmt,dtype", [("e2m1", torch.bfloat16), ("int8", torch.float32)])
@pytest.mark.parametrize("bad", [0, 3])
def test_starts(cu, starts, fmt, dtype, bad):
    check(fmt, dtype, random_table(len(cu), len(cu) - 1, min(bad, len(cu))), cu, starts)


@pytest.mark.parametrize("cu,starts", [
    ([-3, 4, 30], None), ([-13, -2, 40], [0, 0]), ([-20, 100], [0]), ([-5, 31, 48], [-2, 29]), ([-5, 31, 48], [-9, 33]), ([-40, 10, 12], [0, 0]),
    ([-BIG - 1, 12], [BIG]), ([-4, 12], [29])])
@pytest.mark.parametrize("seed", range(3))
def test_lengths_that_begin_before_the_results(cu, starts, seed):
    check("e2m1", torch.float16, random_table(seed, len(cu) - 1, 2), cu, starts)


@pytest.mark.parametrize("cu,starts", [
    ([5, 2, 9], None), ([0, 100, 3], None), ([9, 5, 1], [0, 1]), ([BIG, 0, -BIG - 1], [0, -BIG - 1]), ([7, -BIG - 1, BIG, 30], [BIG, -BIG - 1, 0])])
def test_lengths_that_fall(cu, starts):
    check("int8", torch.float16, random_table(7, len(cu) - 1, 2), cu, starts, ordered=False)
