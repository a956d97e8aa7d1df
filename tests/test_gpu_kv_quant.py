"""GPU: the store that quantises and the read back, against the host model in 64 bits.

The cache's bytes are compared for equality: the definition says which byte every input gives. Q is compared bit for bit
with rope_kv_store's. Values read back are compared for equality with the one rounding of what the bytes stand for.
"""
import numpy as np
import pytest
import torch

import swiglu_rmsnorm_add_gb300 as sra
from tests import quant_model as qm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).to(DEV)


def i64(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int64).to(DEV)


def f64(t):
    return t.detach().double().cpu().numpy()


def tables(hd, max_pos, seed):
    a = np.random.default_rng(seed).uniform(-np.pi, np.pi, (max_pos, hd // 2))
    return torch.tensor(np.cos(a), dtype=F32), torch.tensor(np.sin(a), dtype=F32)


def filled(nb, n_kv, bs, hd, fmt, device=DEV):
    """A cache whose bytes all differ from what a store leaves by chance: 0xA5."""
    c = sra.quant_kv_cache(nb, bs, n_kv, hd, fmt, device=device)
    return c.fill_(0xA5)


def want_store(before, k, v, cos, sin, pos, slot, fmt, style, dtype, norm=None, clip=(-1, 1)):
    """The cache's bytes after the call; before: its bytes at entry."""
    out = before.copy()
    _, nb, n_kv, bs, _ = out.shape
    kk = f64(k)
    if norm is not None:
        a, g = (p.cpu().numpy().astype(np.float32) for p in norm)
        y = np.minimum(np.maximum(kk.astype(np.float32) * a, np.float32(clip[0])), np.float32(clip[1])) * g
        kk = qm.rounded(y.astype(np.float64), dtype)
    P = cos.shape[0]
    ok = (pos >= 0) & (pos < P)
    p = np.where(ok, pos, 0)
    kk = qm.held_k(kk, cos.double().numpy()[p], sin.double().numpy()[p], style, dtype)
    rows = qm.encode(kk, fmt), qm.encode(f64(v), fmt)
    for t in range(len(pos)):
        if ok[t] and 0 <= slot[t] < nb * bs:
            for plane in (0, 1):
                out[plane, slot[t] // bs, :, slot[t] % bs] = rows[plane][t]
    return out


def check_store(T, n_head, n_kv, hd, bs, fmt, dtype, style="neox", seed=0, spread=1.0, fused=False, shift=0, norm=False,
                bad=False, nb=None):
    r, g = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
    nb = nb or -(-T // bs) + 2
    cos, sin = tables(hd, 50, seed)
    W = (n_head + 2 * n_kv) * hd
    buf = torch.randn(T * (W + 8) + shift, generator=g) * torch.exp2(spread * torch.randn(T * (W + 8) + shift, generator=g))
    buf = buf.to(dtype).to(DEV)
    if fused:     # q, k, v as views of one buffer with padded rows, off by `shift` elements
        rows = buf[shift:].view(T, W + 8)
        q, k, v = (rows[:, a * hd:b * hd].unflatten(1, (b - a, hd)) for a, b in
                   ((0, n_head), (n_head, n_head + n_kv), (n_head + n_kv, n_head + 2 * n_kv)))
    else:
        q, k, v = (buf[shift:][a:a + T * n * hd].view(T, n, hd) for a, n in
                   ((0, n_head), (T * n_head * hd, n_kv), (T * (n_head + n_kv) * hd, n_kv)))
    pos, slot = r.integers(0, 50, T), r.permutation(nb * bs)[:T]
    errors = 0
    if bad:
        pos[::5], slot[1::7], slot[2::11] = np.where(r.integers(0, 2, len(pos[::5])), 50, -1), -1, nb * bs
        errors = int(((pos < 0) | (pos >= 50)).sum() + (slot >= nb * bs).sum())
    params = tuple((1 + 0.2 * torch.randn(hd, generator=g)).to(DEV) for _ in range(4)) if norm else None
    cache = filled(nb, n_kv, bs, hd, fmt)
    before, q_before, rest = cache.cpu().numpy(), q.clone(), buf.clone()
    want = want_store(before, k, v, cos, sin, pos, slot, fmt, style, dtype, params[2:] if norm else None, (-1.5, 2.0))
    # q from the store in full precision, over a copy
    q2, plain = q.clone(), torch.zeros(2, nb, bs, n_kv, hd, dtype=dtype, device=DEV)
    kw = dict(style=style, qk_uclip=params, clip=(-1.5, 2.0))
    sra.rope_kv_store(q2, k.clone(), v.clone(), cos.to(DEV), sin.to(DEV), i64(pos), i64(slot), plain, **kw)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    sra.rope_kv_store_quant(q, k, v, cos.to(DEV), sin.to(DEV), i64(pos), i64(slot), cache, err_count=err, **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == errors
    got = cache.cpu().numpy()
    diff = np.argwhere(got != want)
    assert not len(diff), (len(diff), diff[0].tolist(), got[tuple(diff[0])], want[tuple(diff[0])])
    assert torch.equal(q.view(torch.int32 if dtype == F32 else torch.int16), q2.view(torch.int32 if dtype == F32 else torch.int16))
    if T:
        q.copy_(q_before)
        assert torch.equal(buf.view(torch.uint8), rest.view(torch.uint8)), "k, v or the padding changed"


@pytest.mark.parametrize("fmt", ["e2m1", "int8"])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("style", ["neox", "interleaved"])
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_store(fmt, dtype, style, hd):
    check_store(77, 12, 2, hd, 16, fmt, dtype, style, seed=hd + len(fmt), bad=True)


@pytest.mark.parametrize("T,n_head,n_kv,hd,bs", [(1, 1, 1, 64, 8), (1, 32, 4, 128, 16), (3, 3, 3, 256, 7), (300, 8, 1, 64, 32),
                                                (33, 64, 8, 128, 16), (1000, 14, 2, 64, 1), (5, 40, 40, 64, 16)])
@pytest.mark.parametrize("fmt", ["e2m1", "int8"])
def test_store_sizes(T, n_head, n_kv, hd, bs, fmt):
    check_store(T, n_head, n_kv, hd, bs, fmt, BF, seed=T)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("fused,shift", [(True, 0), (True, 1), (False, 3), (True, 8)])
@pytest.mark.parametrize("norm", [False, True])
def test_store_views_and_norms(dtype, fused, shift, norm):
    check_store(41, 6, 2, 128, 16, "e2m1", dtype, "neox", seed=shift, fused=fused, shift=shift, norm=norm)
    check_store(41, 6, 2, 64, 16, "int8", dtype, "interleaved", seed=shift, fused=fused, shift=shift, norm=norm)


@pytest.mark.parametrize("fmt", ["e2m1", "int8"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_store_any_magnitude(fmt, dtype):
    # spreads of 2^+-20 and more within a group: saturation, groups that round to zero, small values beside large ones
    check_store(200, 2, 2, 128, 16, fmt, dtype, seed=9, spread=9.0)
    check_store(200, 2, 2, 128, 16, fmt, dtype, "interleaved", seed=10, spread=16.0)


@pytest.mark.parametrize("fmt", ["e2m1", "int8"])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_store_borders(fmt, dtype):
    """Values on the borders between codes and between scales, and (fp32) the numbers next to them, through V."""
    s = qm.scale_values()
    r = np.random.default_rng(5)
    top = 226 if fmt == "e2m1" else 192
    scale = s[r.integers(1 if dtype != HF else 9, top - 1, 4000)]
    if fmt == "e2m1":
        x = r.choice([.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 0, 4, 6], (4000, 64)) * scale[:, None]
        amax = 6 * scale
    else:
        x = (r.integers(0, 127, (4000, 64)) + 0.5) * scale[:, None]
        amax = 127 * scale
    # every other row's groups have their largest value between two scales, or at one
    nxt = s[np.searchsorted(s, scale) + 1]
    amax[::2] = ((6 if fmt == "e2m1" else 127) * (scale + nxt) / 2)[::2]
    x[:, ::16] = amax[:, None]
    x = np.where(r.integers(0, 2, x.shape), x, -x).astype(np.float32)
    if dtype == F32:
        x = np.where(r.integers(0, 3, x.shape) == 0, x, np.nextafter(x, np.float32(np.inf) * r.choice([-1, 1], x.shape)).astype(np.float32))
    v = torch.tensor(x).to(dtype)[:, None].contiguous().to(DEV)
    T = len(x)
    z = torch.zeros(T, 1, 64, dtype=dtype, device=DEV)
    cache = filled(T // 8, 1, 8, 64, fmt)
    cos, sin = tables(64, 4, 1)
    sra.rope_kv_store_quant(z.clone(), z, v, cos.to(DEV), sin.to(DEV), i64([0] * T), i64(range(T)), cache)
    want = qm.encode(f64(v), fmt)[:, 0]
    got = cache[1].reshape(T, -1).cpu().numpy()
    bad = (got != want).any(-1)
    assert not bad.any(), (int(bad.sum()), x[bad][0], got[bad][0], want[bad][0])
    assert (cache[0] == 0).all()


@pytest.mark.parametrize("fmt", ["e2m1", "int8"])
def test_store_not_finite(fmt):
    T, hd = 16, 128
    k, v = torch.randn(T, 2, hd), torch.randn(T, 2, hd)
    k[0, 0, 3], k[1, 1, 100], v[2, 0, 64], v[3, 1, :] = float("inf"), float("nan"), -float("inf"), float("nan")
    q = torch.zeros(T, 2, hd, dtype=BF, device=DEV)
    cache = filled(2, 2, 8, hd, fmt)
    cos, sin = tables(hd, 4, 1)
    sra.rope_kv_store_quant(q, k.to(BF).to(DEV), v.to(BF).to(DEV), cos.to(DEV), sin.to(DEV), i64([1] * T), i64(range(T)), cache)
    kk, vv = sra.read_kv_quant(cache, i32([[0, 1]]), i32([0, T]), T, hd, F32)
    nan_k, nan_v = torch.zeros(T, 2, hd, dtype=torch.bool), torch.zeros(T, 2, hd, dtype=torch.bool)
    nan_k[0, 0, 0:16] = nan_k[0, 0, 64:80] = True        # the pair of dim 3 is dim 67
    nan_k[1, 1, 96:112] = nan_k[1, 1, 32:48] = True
    nan_v[2, 0, 64:80] = nan_v[3, 1] = True
    assert torch.equal(kk.isnan().cpu(), nan_k) and torch.equal(vv.isnan().cpu(), nan_v)


@pytest.mark.parametrize("fmt", ["e2m1", "int8"])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_read_every_byte(fmt, dtype, hd):
    """All codes under all scales, the NaN one among them."""
    n = qm.row_bytes(fmt, hd) - hd // 16
    rows = np.zeros((256 * 8, n + hd // 16), dtype=np.uint8)
    r = np.random.default_rng(3)
    rows[:, :n] = r.integers(0, 256, (256 * 8, n))
    if fmt == "int8":
        rows[:, :n][rows[:, :n] == 128] = 127
    scales = np.concatenate([np.arange(227 if fmt == "e2m1" else 193), [255]])
    rows[:, n:] = r.choice(scales, (256 * 8, hd // 16))
    cache = torch.tensor(np.stack([rows, rows[::-1]]).reshape(2, 32, 4, 16, -1).copy()).to(DEV)
    order = r.permutation(32)
    k, v = sra.read_kv_quant(cache, i32(order[None]), i32([0, 512]), 512, hd, dtype)
    for plane, got in enumerate((k, v)):
        page = cache[plane].cpu().numpy()[order]                         # [32, 4, 16, R]
        want = qm.decode(page.transpose(0, 2, 1, 3).reshape(512, 4, -1), fmt, hd)
        want = torch.tensor(qm.rounded(np.nan_to_num(want, nan=0.0), dtype)).where(~torch.tensor(want).isnan(), torch.nan)
        assert torch.equal(got.cpu().double().nan_to_num(nan=7e9), want.nan_to_num(nan=7e9))


def random_cache(nb, n_kv, bs, hd, fmt, seed):
    """A cache with every finite value a serving cache may have, on the device."""
    r = np.random.default_rng(seed)
    n = qm.row_bytes(fmt, hd) - hd // 16
    c = r.integers(0, 256, (2, nb, n_kv, bs, n + hd // 16)).astype(np.uint8)
    if fmt == "int8":
        c[..., :n][c[..., :n] == 128] = 0
    c[..., n:] = r.integers(100, 128, c[..., n:].shape)
    return torch.tensor(c).to(DEV)


def dense(cache, fmt, hd, table, row, first, n):
    """[n, n_kv, hd] K and V of a row's tokens from `first` on, in 64 bits."""
    c, bs = cache.cpu().numpy(), cache.shape[3]
    out = np.zeros((2, n, cache.shape[2], hd))
    for i in range(n):
        tok = first + i
        if 0 <= tok < table.shape[1] * bs and 0 <= table[row, tok // bs] < cache.shape[1]:
            out[:, i] = qm.decode(c[:, table[row, tok // bs], :, tok % bs], fmt, hd)
    return out


@pytest.mark.parametrize("fmt,dtype,hd,n_kv,bs", [("e2m1", BF, 128, 2, 16), ("int8", F32, 64, 3, 8), ("e2m1", HF, 256, 1, 5),
                                                 ("int8", BF, 128, 8, 32), ("e2m1", F32, 64, 2, 1)])
def test_read_rows(fmt, dtype, hd, n_kv, bs):
    """Rows of any length, starts, empty rows, bad pages, rows that leave their table, results that are views."""
    r = np.random.default_rng(bs)
    nb, rows, mb = 40, 9, 6
    cache = random_cache(nb, n_kv, bs, hd, fmt, 1)
    table = r.permutation(rows * mb).reshape(rows, mb) % nb
    starts = np.array([0, 3, 0, 2 * bs, 1, 0, 5 * bs, 0, bs])
    lens = np.array([mb * bs, 0, 1, bs + 1, 2 * bs, 3, bs, 0, 2 * bs])
    starts[1] = min(3, mb * bs)
    table[4, 1], table[8, 1] = nb, -1          # row 4 asks for entries 0-2 or 1-2, row 8 for 1-2
    lens[6] += 2                               # past its table
    cu = np.concatenate([[3], 3 + np.cumsum(lens)])
    total = cu[-1] + 4
    buf = torch.full((total, 2 * n_kv * hd + 5), -9.0, dtype=dtype, device=DEV)
    k, v = (buf[:, a:a + n_kv * hd].unflatten(1, (n_kv, hd)) for a in (1, 1 + n_kv * hd))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = sra.read_kv_quant(cache, i32(table), i32(cu), total, hd, starts=i32(starts), out=(k, v), err_count=err)
    assert got[0] is k and got[1] is v
    assert int(err.item()) == 3
    want = torch.full_like(buf, -9.0, device="cpu").double()
    for row in range(rows):
        d = dense(cache, fmt, hd, table, row, starts[row], lens[row])
        for plane in (0, 1):
            want[cu[row]:cu[row + 1], 1 + plane * n_kv * hd:1 + (plane + 1) * n_kv * hd] = torch.tensor(
                qm.rounded(d[plane], dtype).reshape(lens[row], n_kv * hd))
    assert torch.equal(buf.cpu().double(), want)


def test_read_many_rows():
    """More rows than a CTA keeps lengths of, most of them empty."""
    r = np.random.default_rng(1)
    rows, nb, hd = 3001, 64, 64
    cache = random_cache(nb, 1, 8, hd, "e2m1", 2)
    table = r.integers(0, nb, (rows, 2))
    lens = np.where(r.integers(0, 4, rows) == 0, r.integers(0, 17, rows), 0)
    cu = np.concatenate([[0], np.cumsum(lens)])
    k, v = sra.read_kv_quant(cache, i32(table), i32(cu), cu[-1], hd, BF)
    row = np.repeat(np.arange(rows), lens)
    at = np.arange(cu[-1]) - cu[row]
    for plane, got in enumerate((k, v)):
        want = qm.decode(cache[plane].cpu().numpy()[table[row, at // 8], :, at % 8], "e2m1", hd)
        assert np.array_equal(f64(got), want)


def test_read_bad_lengths():
    """Lengths that fall, or lie outside of the results, and starts out of range: nothing out of range happens."""
    cache = random_cache(8, 2, 8, 64, "int8", 3)
    table = i32(np.arange(8).reshape(2, 4))
    for cu, starts in (([5, 2, 9], None), ([-3, 4, 100], None), ([0, 100, 3], None), ([0, 10, 20], [-5, 2 ** 31 - 1]),
                       ([2 ** 31 - 1, 0, -(2 ** 31)], [0, -(2 ** 31)])):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        sra.read_kv_quant(cache, table, i32(cu), 16, 64, BF, starts=None if starts is None else i32(starts), err_count=err)
    k, _ = sra.read_kv_quant(cache, i32(np.zeros((0, 4))), i32([0]), 16, 64, BF)
    torch.cuda.synchronize()
    assert k.shape == (16, 2, 64)
