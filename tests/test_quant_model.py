"""The host model of the cache in 4 or 8 bits against what can be said by hand."""
import numpy as np
import pytest
import torch

from tests import quant_model as qm


def test_scales():
    s = qm.scale_values()
    assert s[0] == 0 and s[1] == 2.0 ** -17 and s[7] == 7 * 2.0 ** -17 and s[8] == 2.0 ** -14 and s[120] == 1.0
    assert s[226] == 10240 and s[192] == 512 and (np.diff(s) > 0).all()
    assert 6 * s[226] <= 65504 < 6 * s[227] and 127 * s[192] <= 65504 < 127 * s[193]


@pytest.mark.parametrize("fmt", ["e2m1", "int8"])
def test_held_values_stay(fmt):
    # whatever a row stands for is held exactly when it is stored again, if its group reaches the largest code
    r = np.random.default_rng(1)
    rows = np.zeros((500, qm.row_bytes(fmt, 64)), dtype=np.uint8)
    n = rows.shape[1] - 4
    rows[:, :n] = r.integers(0, 256, (500, n))
    rows[:, n:] = r.integers(8, 180, (500, 4))
    if fmt == "e2m1":
        rows[:, 0:n:8] = 0x7F
    else:
        rows[:, :n] = np.where(rows[:, :n] == 0x80, 0, rows[:, :n])
        rows[:, 0:n:16] = 127
    x = qm.decode(rows, fmt, 64)
    back = qm.encode(x, fmt)
    assert np.array_equal(qm.decode(back, fmt, 64), x)
    assert np.array_equal(back[:, n:], rows[:, n:])


def test_borders():
    x = np.zeros(64)
    x[:16] = [6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, -6]     # scale 1
    y = qm.decode(qm.encode(x, "e2m1"), "e2m1", 64)
    assert y[:16].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, 0, -1, -1, -2, -2, -4, -4, -6]
    x[:16] = [127, .5, 1.5, 2.5, -.5, -1.5, 126.5, 125.5] + [0] * 8
    assert qm.decode(qm.encode(x, "int8"), "int8", 64)[:8].tolist() == [127, 0, 2, 2, 0, -2, 126, 126]


def test_edges():
    x = np.zeros((4, 64))
    x[0, 3], x[1, 20], x[2, :], x[3, 0] = np.inf, np.nan, 1e30, 6 * 2.0 ** -18
    for fmt, top in (("e2m1", 61440.0), ("int8", 65024.0)):
        y = qm.decode(qm.encode(x, fmt), fmt, 64)
        assert np.isnan(y[0, :16]).all() and (y[0, 16:] == 0).all() and np.isnan(y[1, 16:32]).all() and (y[2] == top).all()
        assert (y[3, 0] == 0) == (fmt == "e2m1")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rounding(dtype):
    x = np.concatenate([np.random.default_rng(2).standard_normal(2000) * 3, [65519.99, 65520.0, 1e-7, 2 ** -14 * 0.7]])
    want = torch.tensor(x.astype(np.float32)).to(dtype).double().numpy()
    assert np.array_equal(qm.rounded(x.astype(np.float32).astype(np.float64), dtype), want)
