"""GPU: decode attention over a cache in 4 or 8 bits: rings filled again many times, tables much wider than the requests, and fp32
queries within a bound of their own.

The tolerance of fp32 queries here follows from the scores. With X = the largest sum_i |scale q_i k_i| of a head over its
tokens and e = 2^-23:
* a score is off by (1 + 17 + 17 * HD / 16 + HD / 16) e X at most: q in two fp16 parts (2^-23 of an element), the truncation of a
  product of 16 terms onto a running sum (17 addends, each cut below 2^-23 of the largest; the lower part of q runs over all steps,
  the upper starts anew at each), the additions between steps; and a few roundings of its factor and difference from the
  maximum, 4 e of scores no larger than 1.5 X + 15;
* a probability by that, by 2^-22 of the exponential, 2^-22 of its two parts;
* sums over n tokens: n / 8 + 16 additions (a lane's own, then lanes, warps, CTAs), and for the values 34 truncations a tile.
All of it relative to A = sum_t p_t |V_t|, twice (above and below the division).
"""
import numpy as np
import pytest
import torch

import swiglu_rmsnorm_add_gb300 as sra
from tests import quant_model as qm
from tests.test_gpu_attention_quant import BF, DEV, F32, HF, Case

pytestmark = pytest.mark.gpu


def forced(variant):
    class Force:
        def __enter__(self):
            sra.force_variant("decode_attention_quant", variant)

        def __exit__(self, *_):
            sra.force_variant("decode_attention_quant", -1)
    return Force()


def attend(c, variant, **kw):
    d = c.dev()
    with forced(variant):
        w = sra.decode_attention_quant_workspace(len(c.lens), c.q.shape[1], c.n_kv, c.hd, c.table.shape[1], c.bs, c.fmt, c.dtype, DEV)
        assert (w is not None) == ((variant & 0xff) == 1)
        return [sra.paged_decode_attention_quant(**d, scale=c.scale, workspace=w) for _ in range(kw.get("times", 1))]


FORMS = {"one CTA": 1 << 8, "two": 2 << 8, "stream": 1}


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("fmt,hd,bs,dtype", [("e2m1", 128, 16, BF), ("int8", 64, 32, HF), ("e2m1", 256, 8, F32), ("int8", 256, 16, BF),
                                            ("int8", 128, 8, F32), ("e2m1", 64, 16, BF)])
def test_rings_that_turn_often(form, fmt, hd, bs, dtype):
    """Hundreds of tiles through each warp's ring (where one CTA has a request), the same result every time, that of the formula."""
    c = Case(4, 2, hd, bs, [40000, 3333], fmt, dtype, seed=hd)
    outs = attend(c, FORMS[form], times=20)
    torch.cuda.synchronize()
    c.check(outs[0])
    assert all(torch.equal(outs[0].view(torch.uint8), x.view(torch.uint8)) for x in outs)


@pytest.mark.parametrize("variant", [0, 1])
@pytest.mark.parametrize("auto", [False, True])
@pytest.mark.parametrize("fmt,hd,bs,lens", [("e2m1", 128, 16, [250]), ("int8", 64, 32, [1, 0, 777, 33]), ("e2m1", 256, 8, [40] * 70),
                                           ("int8", 128, 16, [4096] + [3] * 9)])
def test_tables_much_wider_than_the_requests(variant, auto, fmt, hd, bs, lens):
    """Tables for 65536 tokens: what lies behind a request's pages is not looked at."""
    c = Case(8, 2, hd, bs, lens, fmt, BF, seed=len(lens))
    wide = np.full((len(lens), 65536 // bs), 2 ** 31 - 1)
    wide[::2] = -7
    wide[:, :c.table.shape[1] - 1] = c.table[:, :-1]
    c.table = wide
    if not auto:
        (got,) = attend(c, variant)
    else:
        d = c.dev()
        w = sra.decode_attention_quant_workspace(len(lens), 8, 2, hd, wide.shape[1], bs, fmt, BF, DEV) if variant else None
        got = sra.paged_decode_attention_quant(**d, scale=c.scale, workspace=w)
    c.check(got)


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("fmt", ["e2m1", "int8"])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("scale", [0.0, 1e-4, 2e-3, 0.02])
def test_fp32_queries(form, fmt, hd, scale):
    c = Case(6, 2, hd, 16, [300, 1, 33, 77, 150], fmt, F32, seed=hd + 1, scale=scale)
    (got,) = attend(c, FORMS[form])
    o, A, S = c.want()
    q, e, G = c.q.double().numpy(), 2.0 ** -23, 3
    tol = np.zeros_like(o)
    for b, n in enumerate(c.lens):
        k, _ = c.tokens(b)
        for h in range(6):
            X = scale * (np.abs(q[b, h]) * np.abs(k[:, h // G])).sum(-1).max()
            score = (1 + 17 + 17 * hd / 16 + hd / 16) * e * X + 4 * e * (1.5 * X + 15)
            tol[b, h] = e / 2 * np.abs(o[b, h]) + 2 * (score + 2 * 2.0 ** -22 + (n / 8 + 16 + 34 * (n / 32 + 1)) * e / 2) * A[b, h]
    g = got.double().cpu().numpy()
    err = np.abs(g - o) - tol - 2.0 ** -39 * S
    assert (err <= 0).all(), (float(err.max()), float((np.abs(g - o) / np.maximum(tol, 1e-30)).max()))


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("fmt", ["e2m1", "int8"])
@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_whose_steps_are_large(form, fmt, dtype, sign):
    """Scores up to 2^31, whose fp32 neighbours are up to 256 apart: the largest one takes all the weight, and the result is its V."""
    c = Case(4, 2, 128, 16, [26, 9, 1], fmt, dtype, seed=3)
    n = c.cache.shape[-1] - 8
    r = np.random.default_rng(4)
    best = []
    for b, length in enumerate(c.lens):     # K of token t: its scale in every dim, another scale for each token
        step = r.permutation(np.arange(100, 126))[:length]
        for t in range(length):
            row = c.cache[0, c.table[b, t // 16], :, t % 16]
            row[:, :n], row[:, n:] = 0x22 if fmt == "e2m1" else 1, step[t]
        best.append(int(step.argmax() if sign > 0 else step.argmin()))
    c.q = torch.full_like(c.q, 64.0 * sign)
    v = [c.tokens(b)[1] for b in range(3)]
    for e in range(20, 32):
        for m in (1.0, 1.3, 1.9):
            top = max(float(np.abs(64.0 * 128 * qm.decode(c.cache[0, c.table[0, 0], 0, :16], fmt, 128)[:, 0]).max()), 1.0)
            c.scale = m * 2.0 ** e / top / 1.4426950408889634
            (got,) = attend(c, FORMS[form])
            for b in range(3):
                want = np.repeat(qm.rounded(v[b][best[b]], dtype), 2, 0)
                assert np.array_equal(got[b].double().cpu().numpy(), want), (e, m, b)
