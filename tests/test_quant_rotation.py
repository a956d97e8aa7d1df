"""The rotated K that is quantised is the rotation's exact value rounded once to fp32 and once to the dtype: inputs at which
one place of fp32 decides the byte, against rational arithmetic.

K = a c - b s is made to come out
* as the rounding residue of two products (the whole group's amax is that residue),
* on a border between codes, or one place of fp32 beside it,
* exactly between such a border and the fp32 number under it, but for a product of 2^-60 of it, of either sign,
* as a zero of either sign, and from products that underflow or overflow fp32.
"""
from fractions import Fraction

import numpy as np
import pytest
import torch

import swiglu_rmsnorm_add_gb300 as sra
from tests import quant_model as qm

DEV = "cuda:0"
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


# --------------------------------------------------------------------------- the model
def nearest32(x: Fraction) -> float:
    """The fp32 number nearest to x, ties to even (x is not 0)."""
    n, d = abs(x.numerator), x.denominator
    e = n.bit_length() - d.bit_length()
    e -= Fraction(n, d) < Fraction(2) ** e              # 2^e <= |x| < 2^(e + 1)
    step = Fraction(2) ** (max(e, -126) - 23)
    y = round(x / step) * step                          # (Fraction's round: ties to even)
    return np.copysign(np.inf if abs(y) >= Fraction(2) ** 128 else float(y), -1.0 if x < 0 else 1.0)


def rotated32(a, c, b, s):
    """a c - b s of fp32 numbers, rounded once; a zero has the sign that IEEE arithmetic gives it."""
    out = np.empty(a.shape, dtype=np.float64)
    for i, v in enumerate(zip(*(x.ravel().tolist() for x in (a, c, b, s)))):
        y = Fraction(v[0]) * Fraction(v[1]) - Fraction(v[2]) * Fraction(v[3])
        out.flat[i] = nearest32(y) if y else v[0] * v[1] - v[2] * v[3]
    return out


def test_nearest32():
    r = np.random.default_rng(0)
    for x in np.concatenate([r.standard_normal(300), r.standard_normal(100) * 2.0 ** -130, [1e-45, 2.0 ** -149, 3e38]]):
        assert nearest32(Fraction(float(x))) == float(np.float32(x))
    one = Fraction(1)
    assert nearest32(one + Fraction(1, 2 ** 24)) == 1.0 and nearest32(one + Fraction(1, 2 ** 24) + Fraction(1, 2 ** 90)) == 1 + 2.0 ** -23
    assert nearest32(one - Fraction(1, 2 ** 25)) == 1.0 and nearest32(one - Fraction(1, 2 ** 25) - Fraction(1, 2 ** 90)) == 1 - 2.0 ** -24
    assert nearest32(-Fraction(2) ** 128) == -np.inf


def test_rotated32_is_the_models():
    # the model of the other tests (64 bits, rounded twice) is the same where nothing lies next to a border
    r = np.random.default_rng(1)
    x, c, s = (r.standard_normal((3, 2, 64)).astype(np.float32), *(r.standard_normal((2, 3, 32)).astype(np.float32)))
    want = qm.rounded(qm.rotated(x.astype(np.float64), c.astype(np.float64), s.astype(np.float64), "neox"), F32)
    got = rotated32(x[..., :32], np.broadcast_to(c[:, None], (3, 2, 32)), x[..., 32:], np.broadcast_to(s[:, None], (3, 2, 32)))
    assert np.array_equal(got, want[..., :32])


# --------------------------------------------------------------------------- the inputs
def f32(x):
    return np.asarray(x, dtype=np.float64).astype(np.float32)


def split(n, limit=1 << 24):
    """n as a product of two factors below limit, or None."""
    for f in range(2, 1 << 14):
        if n % f == 0 and n // f < limit:
            return f, n // f
    return None


class Pairs:
    """T tokens of one head of 64 dims: 32 pairs (a, b), a table row (c, s) for each token."""

    def __init__(self, T):
        self.a, self.b, self.c, self.s = (np.zeros((T, 32), dtype=np.float32) for _ in range(4))

    def rows(self, swap, dtype):
        """a, b, s so that the interesting result a c - b s is the pair's first (or, swapped, second) element."""
        a, b, s = (self.b, self.a, -self.s) if swap else (self.a, self.b, self.s)   # second: b c + a s
        both = torch.tensor(np.stack([a, b])).to(dtype).float().numpy()
        return both[0], both[1], s


def cancelling(T, r):
    """b = a c / s to fp32, and up to two places off: what is left is the products' own rounding."""
    p = Pairs(T)
    angle = r.uniform(0.1, 1.4, (T, 32))
    p.a, p.c, p.s = f32(r.uniform(0.5, 4, (T, 32)) * r.choice([-1, 1], (T, 32))), f32(np.cos(angle)), f32(np.sin(angle))
    p.b = f32(p.a.astype(np.float64) * p.c / p.s)
    for _ in range(2):
        p.b = np.where(r.integers(0, 3, (T, 32)) == 0, np.nextafter(p.b, np.float32(9)), p.b)
    p.b[::4] = f32(p.a[::4].astype(np.float64) * p.c[::4] / p.s[::4])
    return p


BORDERS = {"e2m1": [.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0], "int8": [k + 0.5 for k in (0, 1, 2, 7, 30, 63, 100, 125)]}
TOP = {"e2m1": 6.0, "int8": 127.0}


def at_borders(T, fmt, r):
    """a c - b s on a border of a group with scale 1 or 2^-5, give or take a place of fp32 or two of its products'."""
    p = Pairs(T)
    scale = r.choice([1.0, 2.0 ** -5], (T, 1))
    angle = r.uniform(0.1, 1.4, (T, 32))
    p.c, p.s = f32(np.cos(angle)), f32(np.sin(angle))
    want = r.choice(BORDERS[fmt], (T, 32)) * scale * r.choice([-1, 1], (T, 32))
    p.b = f32(r.standard_normal((T, 32)) * scale)
    p.a = f32((want + p.b.astype(np.float64) * p.s) / p.c)
    p.a = np.where(r.integers(0, 2, (T, 32)) == 0, p.a, np.nextafter(p.a, np.float32(np.inf) * r.choice([-1, 1], (T, 32)).astype(np.float32)))
    # the groups' largest values, as they are: 6 (127) times the scale
    for j in (0, 8, 16, 24):
        p.a[:, j], p.b[:, j], p.c[:, j], p.s[:, j] = TOP[fmt] * scale[:, 0], TOP[fmt] * scale[:, 0], 1, 0
    return p


def at_ties(T, fmt, r):
    """a c exactly half a place under a border, b s = 0 or 2^-60 of it, of either sign: the last decides."""
    p = Pairs(T)
    found = []
    for x in BORDERS[fmt]:
        for k in range(16, 30):      # in units of half a place of the fp32 numbers below the border
            n = x * 2.0 ** k
            if n == int(n) and 1 << 24 < int(n) - 1 < 1 << 25 and split(int(n) - 1):
                found.append((x, k, split(int(n) - 1)))
    assert len(found) > 1
    for t in range(T):
        for j in range(32):
            if j % 8 == 0:
                p.a[t, j] = p.b[t, j] = TOP[fmt]
                p.c[t, j] = 1
            else:
                x, k, (f, g) = found[r.integers(len(found))]
                sign = r.choice([-1.0, 1.0])
                p.a[t, j], p.c[t, j] = sign * f * 2.0 ** -4, g * 2.0 ** (4 - k)
                p.b[t, j], p.s[t, j] = r.choice([-1.0, 0.0, 1.0]) * 2.0 ** -50, x * 2.0 ** -10
    return p


def at_the_ends(T, r):
    """Zeros of either sign; products that underflow fp32, or overflow it and cancel."""
    p = Pairs(T)
    zero = [0.0, -0.0]
    for a in (p.a, p.b):
        a[:] = r.choice(zero, (T, 32))
    p.c, p.s = f32(r.standard_normal((T, 32))), f32(r.standard_normal((T, 32)))
    small = r.integers(0, 2, (T, 32)) == 0
    for a in (p.a, p.b, p.c, p.s):
        a[small] = f32(r.standard_normal((T, 32)) * 2.0 ** -r.integers(40, 75, (T, 32)))[small]
    big = r.integers(0, 4, (T, 32)) == 0        # 2^130, less almost all of it
    p.a[big], p.c[big], p.b[big] = 2.0 ** 120, 1024.0, 2.0 ** 120
    p.s[big] = (1024.0 - f32(2.0 ** -r.integers(110, 125, (T, 32)))).astype(np.float32)[big]
    p.s[big] = np.where(r.integers(0, 2, int(big.sum())) == 0, np.nextafter(np.float32(1024), np.float32(0)), p.s[big])
    for j in range(0, 32, 8):
        p.a[:, j] = p.b[:, j] = 6
        p.c[:, j], p.s[:, j] = 1, 0
    # (the huge differences would be their groups' amax: groups of their own)
    p.a[::2][big[::2]] = 0
    p.c[::2][big[::2]] = 1
    p.b[::2][big[::2]] = 0
    return p


KINDS = {"cancelling": lambda T, fmt, r: cancelling(T, r), "borders": at_borders, "ties": at_ties,
         "ends": lambda T, fmt, r: at_the_ends(T, r)}


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["e2m1", "int8"])
@pytest.mark.parametrize("style", ["neox", "interleaved"])
@pytest.mark.parametrize("swap", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("kind", list(KINDS))
def test_k_is_rounded_once(kind, dtype, swap, style, fmt):
    T, r = 96, np.random.default_rng(list(KINDS).index(kind))
    with np.errstate(over="ignore", under="ignore"):
        p = KINDS[kind](T, fmt, r)
        a, b, s = p.rows(swap, dtype)
        finite = np.isfinite(a).all() and np.isfinite(b).all()
    assert finite or dtype == HF        # (fp16 has no 2^120)
    if not finite:
        a, b = (np.where(np.isfinite(x), x, np.float32(1)) for x in (a, b))
    k = np.zeros((T, 1, 64), dtype=np.float32)
    want = np.zeros((T, 1, 64))
    lo, hi = (slice(0, 32), slice(32, 64)) if style == "neox" else (slice(0, None, 2), slice(1, None, 2))
    k[:, 0, lo], k[:, 0, hi] = a, b
    want[:, 0, lo], want[:, 0, hi] = rotated32(a, p.c, b, s), rotated32(b, p.c, -a, s)
    want = qm.encode(qm.rounded(want, dtype), fmt)[:, 0]
    kt = torch.tensor(k).to(dtype).to(DEV)
    z = torch.zeros(T, 1, 64, dtype=dtype, device=DEV)
    cache = sra.quant_kv_cache(T // 8, 8, 1, 64, fmt, device=DEV)
    at = torch.arange(T, device=DEV)
    sra.rope_kv_store_quant(z.clone(), kt, z, torch.tensor(p.c).to(DEV), torch.tensor(s).to(DEV), at, at, cache, style=style)
    got = cache[0].reshape(T, -1).cpu().numpy()
    bad = (got != want).any(-1)
    t = int(bad.argmax())
    assert not bad.any(), (int(bad.sum()), int((got != want).sum()), t, got[t].tolist(), want[t].tolist())


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["e2m1", "int8"])
@pytest.mark.parametrize("style", ["neox", "interleaved"])
@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("kind", ["borders", "ties", "sparse"])
def test_behind_the_norm_and_out_of_views(kind, shift, dtype, style, fmt):
    """The pairs that are rotated once more take the norm's values, from tensors of any alignment."""
    T, r = 64, np.random.default_rng(7)
    if kind == "sparse":        # two pairs of three are zeros
        p = at_borders(T, fmt, r)
        zero = r.integers(0, 3, (T, 32)) > 0
        p.a[zero], p.b[zero] = -0.0, 0.0
    else:
        p = KINDS[kind](T, fmt, r)
    a, b, s = p.rows(False, dtype)
    lo, hi = (slice(0, 32), slice(32, 64)) if style == "neox" else (slice(0, None, 2), slice(1, None, 2))
    gain = f32(2.0 ** r.integers(-2, 3, 64))
    want, k = np.zeros((T, 1, 64)), np.zeros((T, 1, 64), dtype=np.float32)
    want[:, 0, lo], want[:, 0, hi] = rotated32(a, p.c, b, s), rotated32(b, p.c, -a, s)
    want = qm.encode(qm.rounded(want, dtype), fmt)[:, 0]
    k[:, 0, lo], k[:, 0, hi] = a, b
    k = k / gain                # (the norm's alpha puts it back: powers of two, exact away from fp16's subnormal numbers)
    if dtype == HF:
        k = k * (gain if kind == "ties" else 1)
    alpha = gain if not (dtype == HF and kind == "ties") else np.ones_like(gain)

    def view(x, dt):
        x = torch.tensor(x).to(dt)
        room = torch.zeros(x.numel() + 8, dtype=dt, device=DEV)
        return room[shift:shift + x.numel()].view(x.shape).copy_(x)
    one = view(np.ones(64, dtype=np.float32), F32)
    z = torch.zeros(T, 1, 64, dtype=dtype, device=DEV)
    cache = sra.quant_kv_cache(T // 8, 8, 1, 64, fmt, device=DEV)
    at = torch.arange(T, device=DEV)
    sra.rope_kv_store_quant(z.clone(), view(k, dtype), z, view(p.c, F32), view(s, F32), at, at, cache, style=style,
                            qk_uclip=(one, one, view(alpha, F32), one), clip=(-1e30, 1e30))
    got = cache[0].reshape(T, -1).cpu().numpy()
    diff = np.argwhere(got != want)
    assert not len(diff), (len(diff), diff[0].tolist())
