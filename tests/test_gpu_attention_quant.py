"""GPU: decode attention over a cache in 4 or 8 bits against the formula in 64 bits.

Tolerance, per output element. With p the exact probabilities, A = sum_t p_t |V_t| and u = eps / 2 of the dtype: the result
is rounded once (u |o|); bf16 and fp16 queries meet probabilities rounded once to fp16 (2^-11 of each, so 2^-11 A), fp32
ones to two fp16 numbers (2^-22 A); K and V are exact. The evaluation in fp32 (a score's dot product of up to 256 terms, the
exponential, sums over the tokens) is allowed 6e-5 A, as in the shared prefix's tests. Where numbers are subnormal, a
rounding is absolute instead: a result is off by up to half of the dtype's smallest number (fp16 2^-25: a result of 1.2e-5 was off
by 2.7e-8, more than 2^-11 of it), and a probability, held at 2^14 times its size relative to the largest, by up to 2^-39 of
that: 2^-39 S, S = sum_t |V_t| (the largest probability is no more than the sum that the result is divided by).

The caches read as NaN wherever a request must not look: pages of nobody, tokens behind a request's last one; the table
entries that are not read are out of range.
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


class Case:
    def __init__(self, n_head, n_kv, hd, bs, lens, fmt, dtype, seed, scale=None, spread=1.0, extra_cols=1):
        r = np.random.default_rng(seed)
        self.lens, self.bs, self.fmt, self.dtype, self.hd, self.n_kv = [int(x) for x in lens], bs, fmt, dtype, hd, n_kv
        self.scale = scale if scale is not None else hd ** -0.5
        pages = [-(-x // bs) for x in self.lens]
        self.nb = sum(pages) + 2
        perm = r.permutation(self.nb)
        self.table = np.full((len(lens), max([0] + pages) + extra_cols), -5)
        self.table[::2] = self.nb + 3
        self.cache = np.full((2, self.nb, n_kv, bs, qm.row_bytes(fmt, hd)), 255, dtype=np.uint8)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = perm[at:at + n]
            x = r.standard_normal((2, n * bs, n_kv, hd)) * np.exp2(r.standard_normal((2, 1, n_kv, hd)) * 0.5) * spread
            rows = qm.encode(x.astype(np.float32).astype(np.float64), fmt)
            rows[:, self.lens[b]:] = 255
            self.cache[:, perm[at:at + n]] = rows.reshape(2, n, bs, n_kv, rows.shape[-1]).transpose(0, 1, 3, 2, 4)
            at += n
        self.q = torch.tensor(r.standard_normal((len(lens), n_head, hd)) * 1.5).to(dtype)

    def dev(self):
        return dict(q=self.q.to(DEV), kv_cache=torch.tensor(self.cache).to(DEV), block_table=i32(self.table),
                    seq_lens=i32(self.lens))

    def tokens(self, b):
        """[2, tokens, n_kv, hd] of the request's tokens in good pages, 64 bits."""
        t = np.arange(min(max(self.lens[b], 0), self.table.shape[1] * self.bs))
        page = self.table[b, t // self.bs] if len(t) else t
        t, page = t[(page >= 0) & (page < self.nb)], page[(page >= 0) & (page < self.nb)]
        return qm.decode(self.cache[:, page, :, t % self.bs].transpose(1, 0, 2, 3), self.fmt, self.hd)

    def want(self):
        q = self.q.double().numpy()
        o, A, S = np.zeros_like(q), np.zeros_like(q), np.zeros_like(q)
        G = q.shape[1] // self.n_kv
        for b in range(len(self.lens)):
            k, v = self.tokens(b)
            for h in range(self.n_kv if k.shape[0] else 0):
                i = slice(h * G, h * G + G)
                s = self.scale * q[b, i] @ k[:, h].T
                p = np.exp(s - s.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                o[b, i], A[b, i], S[b, i] = p @ v[:, h], p @ np.abs(v[:, h]), np.abs(v[:, h]).sum(0)
        return o, A, S

    def check(self, got, what=""):
        o, A, S = self.want()
        u = torch.finfo(self.dtype).eps / 2
        up = 2.0 ** -22 if self.dtype == F32 else 2.0 ** -11
        tol = u * np.abs(o) + (up + 6e-5) * A + 2.0 ** -39 * S + torch.finfo(self.dtype).smallest_normal * u + 1e-30
        g = got.double().cpu().numpy()
        bad = ~((np.abs(g - o) <= tol) | (np.isnan(g) & np.isnan(o)))
        assert not bad.any(), (what, int(bad.sum()), np.nanmax(np.abs(g - o)), np.argwhere(bad)[0].tolist())


FORM = ["auto"]


@pytest.fixture(params=["auto", "cluster", "stream"], autouse=True)
def form(request):
    """The automatic choice, and each of the two forms forced."""
    sra.force_variant("decode_attention_quant", {"auto": -1, "cluster": 0, "stream": 1}[request.param])
    FORM[0] = request.param
    yield request.param
    sra.force_variant("decode_attention_quant", -1)


def workspace(c):
    return sra.decode_attention_quant_workspace(len(c.lens), c.q.shape[1], c.n_kv, c.hd, c.table.shape[1], c.bs, c.fmt, c.dtype, DEV)


def spaces(c):
    """The workspaces to run with: none (the stream form, forced, is refused then), and the one that the form uses."""
    w = workspace(c)
    assert (w is None) if FORM[0] == "cluster" else (w is not None or FORM[0] == "auto")
    return ([] if FORM[0] == "stream" else [None]) + ([] if w is None else [w])


def run(c, what="", errors=0, **kw):
    d = c.dev()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    before = sra.wait_timeouts()
    outs = []
    for w in spaces(c):
        if w is not None:
            w.fill_(255)
        err.zero_()
        got = sra.paged_decode_attention_quant(**d, scale=c.scale, err_count=err, workspace=w, **kw)
        torch.cuda.synchronize()
        assert sra.wait_timeouts() == before
        assert int(err.item()) == errors, (what, int(err.item()))
        c.check(got, (what, w is not None))
        again = sra.paged_decode_attention_quant(**d, scale=c.scale, workspace=w, **kw)
        assert torch.equal(got.view(torch.uint8), again.view(torch.uint8)), "two calls differ"
        outs.append(got)
    return outs


@pytest.mark.parametrize("fmt", ["e2m1", "int8"])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("bs", [8, 16, 32])
def test_values(fmt, dtype, hd, bs):
    run(Case(6, 2, hd, bs, [1, 7, bs, bs + 1, 100, 0, 333], fmt, dtype, seed=hd + bs))


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("n_kv", [1, 3])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_groups(G, n_kv, dtype):
    run(Case(G * n_kv, n_kv, 128, 16, [257, 31, 32, 33], "e2m1", dtype, seed=G))


@pytest.mark.parametrize("fmt,hd,lens", [("e2m1", 128, [5000]), ("int8", 64, [9000, 1, 0]), ("e2m1", 256, [2500] * 3),
                                        ("e2m1", 64, [1] * 70), ("int8", 128, list(range(0, 640, 5))), ("e2m1", 128, [20000, 17]),
                                        ("e2m1", 128, [0, 0, 0]), ("int8", 256, [4097])])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_lengths(fmt, hd, lens, dtype):
    run(Case(12, 2, hd, 16, lens, fmt, dtype, seed=len(lens)))


def test_many_requests():
    r = np.random.default_rng(4)
    run(Case(4, 1, 64, 8, r.integers(0, 90, 1500), "e2m1", BF, seed=4))
    run(Case(4, 2, 128, 16, [0] * 400 + [700] + [0] * 300 + [3], "int8", HF, seed=5))


@pytest.mark.parametrize("scale", [0.0, -0.1, 1.0, 3e-5])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_scales(scale, dtype):
    run(Case(8, 2, 128, 16, [300, 5], "e2m1", dtype, seed=6, scale=scale, spread=0.3))


@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_wide_queries(dtype):
    """Rows of q whose elements differ by many powers of two, far from 1; the scale brings the scores back."""
    for e in (-20, 12) if dtype == HF else (-100, -20, 40, 100):
        c = Case(4, 2, 128, 16, [200, 90], "e2m1", dtype, seed=7)
        g = torch.Generator().manual_seed(1)
        size = torch.exp2(torch.randint(-6 if dtype == HF and e > 0 else 0, 1, c.q.shape, generator=g) * 1.0)
        c.q = (c.q.double() * size * 2.0 ** e / (4 if e == 12 else 1)).to(dtype)
        c.scale = 0.1 * 2.0 ** -e
        if dtype == HF and e < 0:       # fp16's own subnormals
            assert float(c.q.abs().max()) > 0
        run(c, e)


def test_bad_pages_and_lengths():
    c = Case(6, 2, 128, 16, [200, 90, 64], "e2m1", BF, seed=8)
    c.table[0, 3], c.table[0, 12], c.table[2, :4] = c.nb, -1, c.nb + 9      # request 2 has no good page
    run(c, errors=2 + 4)
    c = Case(6, 2, 64, 16, [40, 33, 20], "int8", HF, seed=9, extra_cols=0)
    c.lens = [49, -1, 2 ** 31 - 1]      # past the table, negative: clamped and counted
    c.table[0, 2], c.table[2, 2] = c.nb, -1
    c.cache[c.cache == 255] = 100
    run(c, errors=3 + 1 + 1)


def test_nan_and_infinite_scores():
    c = Case(4, 2, 128, 16, [100, 100, 100, 100], "e2m1", BF, seed=10)
    c.q[0, 0, 5] = float("nan")          # one head of one request
    c.q[1, :] = 0.0
    c.cache[1, c.table[2, 3], 1, 7, 64 + 2] = 255     # V: 16 dims of kv head 1 of request 2
    c.cache[0, c.table[3, 1], 0, 2, 64] = 255         # K: kv head 0 of request 3
    with np.errstate(invalid="ignore"):
        for got in run(c):
            nan = torch.isnan(got).cpu()
            assert nan[0, 0].all() and not nan[0, 1:].any() and not nan[1].any()
            assert nan[2, 2:, 32:48].all() and int(nan[2].sum()) == 2 * 16
            assert nan[3, :2].all() and not nan[3, 2:].any()


def test_no_score_above_minus_infinity():
    c = Case(2, 1, 64, 8, [20, 50], "e2m1", BF, seed=11)
    c.cache[0, :, :, :, :32] = 0x22           # every K value is its group's scale
    c.cache[0, :, :, :, 32:] = 120
    c.q[0] = 0.0
    c.q[0, :, 0] = -float("inf")
    d = c.dev()
    for w in spaces(c):
        got = sra.paged_decode_attention_quant(**d, workspace=w)
        # -inf * 1 + 0 * 1 ... = -inf for every token: nothing weighs
        assert (got[0] == 0).all()
        assert torch.isfinite(got[1]).all()


def test_large_values():
    """Keys and values at the ends of what a group can hold."""
    for fmt, top in (("e2m1", 226), ("int8", 192)):
        c = Case(8, 2, 128, 16, [150, 40], fmt, F32, seed=12, scale=1e-7)
        n = c.cache.shape[-1] - 8
        c.cache[..., n:][c.cache[..., n:] != 255] = top
        run(c)
        c.scale = 0.0
        run(c)


def test_views():
    """q and out as views of wider rows, any alignment."""
    for dtype in (BF, F32):
        for shift in (0, 1, 2, 8):
            c = Case(6, 2, 128, 16, [100, 33, 5], "e2m1", dtype, seed=13)
            d = c.dev()
            W = 6 * 128
            buf = torch.zeros(3 * (W + 24) + shift, dtype=dtype, device=DEV)
            q = buf[shift:].view(3, W + 24)[:, :W].unflatten(1, (6, 128))
            q.copy_(d["q"])
            obuf = torch.full((3 * (W + 9) + shift,), 7.0, dtype=dtype, device=DEV)
            out = obuf[shift:].view(3, W + 9)[:, :W].unflatten(1, (6, 128))
            got = sra.paged_decode_attention_quant(q, d["kv_cache"], d["block_table"], d["seq_lens"], out=out, workspace=spaces(c)[-1])
            assert got is out
            c.check(got)
            out.fill_(7.0)
            assert (obuf == 7.0).all()


def test_against_the_16_bit_cache():
    """The same values in a 16-bit cache give the same attention."""
    c = Case(12, 2, 128, 16, [777, 50, 3], "e2m1", HF, seed=14)
    d = c.dev()
    c.cache[c.cache == 255] = 0
    plain = torch.tensor(qm.decode(c.cache, c.fmt, c.hd)).to(HF).to(DEV).transpose(2, 3).contiguous()
    c.check(sra.paged_decode_attention(d["q"], plain, d["block_table"], d["seq_lens"]))
    run(c)


def test_graph_and_streams():
    c = Case(12, 2, 128, 16, [777, 50, 3, 4000], "e2m1", BF, seed=15)
    d, w = c.dev(), workspace(c)
    want = sra.paged_decode_attention_quant(**d, workspace=w)
    out = torch.empty_like(want)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            sra.paged_decode_attention_quant(**d, out=out, workspace=w)
    for _ in range(3):
        out.zero_()
        if w is not None:
            w.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    got = sra.paged_decode_attention_quant(**d, workspace=w, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_forced_forms(form):
    """Clusters of any size; the stream form without a workspace is refused."""
    c = Case(6, 2, 128, 16, [1500, 0, 33], "e2m1", BF, seed=17)
    d = c.dev()
    for splits in range(1, 17):
        sra.force_variant("decode_attention_quant", splits << 8)
        c.check(sra.paged_decode_attention_quant(**d), splits)
    for variant, w in ((17 << 8, None), (32 << 8, None), (1, None)):
        sra.force_variant("decode_attention_quant", variant)
        with pytest.raises(sra.SRAError) as e:
            sra.paged_decode_attention_quant(**d, workspace=w)
        assert e.value.status == -7
    sra.force_variant("decode_attention_quant", 1)
    w = workspace(c)
    with pytest.raises(sra.SRAError) as e:      # too small
        sra.paged_decode_attention_quant(**d, workspace=w[:-16])
    assert e.value.status == -6
    with pytest.raises(sra.SRAError) as e:      # misaligned
        sra.paged_decode_attention_quant(**d, workspace=torch.empty(w.numel() + 16, dtype=torch.uint8, device=DEV)[8:])
    assert e.value.status == -6


def test_pdl_chain():
    """Calls in a row under programmatic dependent launch, each reading what the one before wrote."""
    c = Case(8, 2, 128, 16, [500, 1200, 64], "e2m1", BF, seed=16)
    d = c.dev()
    w = workspace(c)
    want, q = [], d["q"].clone()
    for _ in range(4):
        q = sra.paged_decode_attention_quant(q, d["kv_cache"], d["block_table"], d["seq_lens"], workspace=w)
        want.append(q)
    torch.cuda.synchronize()
    old = sra.set_pdl(True)
    try:
        for _ in range(20):
            q = d["q"].clone()
            for k in range(4):
                q = sra.paged_decode_attention_quant(q, d["kv_cache"], d["block_table"], d["seq_lens"], workspace=w)
            torch.cuda.synchronize()
            assert torch.equal(q, want[-1])
    finally:
        sra.set_pdl(old)
