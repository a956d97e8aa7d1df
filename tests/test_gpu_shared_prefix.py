"""GPU: attention over a shared prefix against the formula in 64 bits.

Tolerance, per output element. With p the exact probabilities, A = sum_t p_t |V_t| and u = eps / 2 of
the dtype: the result is rounded once (u |o|); the prefix's probabilities are rounded once to the
dtype before they multiply V (u A, taken for every token; fp32 inputs have no such rounding); the
evaluation in fp32 (a score's dot product of up to 256 terms, the exponential, sums over the tokens)
is allowed 6e-5 A: the bound that the decode attention's tests use, 3e-5, once for the numerator and
once for the sum that it is divided by.

The caches hold NaN wherever a request must not look: pages of nobody, tokens behind a request's
last one, and the table entries that are not read are out of range.
"""
import numpy as np
import pytest
import torch

import swiglu_rmsnorm_add_gb300 as sra

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


class Case:
    def __init__(self, B, n_head, n_kv, hd, bs, prefix, lens, dtype, seed, extra_cols=1, scale=None, spread=1.0):
        r = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.B, self.P, self.lens, self.bs, self.dtype = B, prefix, [int(x) for x in lens], bs, dtype
        self.n_kv, self.hd, self.scale = n_kv, hd, scale if scale is not None else hd ** -0.5
        pages = lambda L: -(-L // bs)
        M = pages(max([prefix] + self.lens)) + extra_cols
        own = [max(0, pages(L) - prefix // bs) if L > prefix else 0 for L in self.lens]
        nb = pages(prefix) + sum(own) + 2
        perm = r.permutation(nb)
        self.ptable = np.full(pages(prefix) + 2, nb + 7)      # entries past the prefix are never read
        self.ptable[:pages(prefix)] = perm[:pages(prefix)]
        self.table = np.full((B, M), -5)
        at = pages(prefix)
        cache = torch.full((2, nb, bs, n_kv, hd), float("nan"))
        V = lambda *s: torch.randn(s, generator=g) * spread
        for t in range(prefix):
            cache[:, self.ptable[t // bs], t % bs] = V(2, n_kv, hd)
        for b in range(B):
            first = prefix // bs
            self.table[b, first:first + own[b]] = perm[at:at + own[b]]
            at += own[b]
            for t in range(prefix, self.lens[b]):
                cache[:, self.table[b, t // bs], t % bs] = V(2, n_kv, hd)
        self.q = V(B, n_head, hd).to(dtype)
        self.cache = cache.to(dtype)
        self.nb = nb

    def dev(self):
        i = lambda a: torch.as_tensor(np.asarray(a), dtype=torch.int32).to(DEV)
        return dict(q=self.q.to(DEV), kv_cache=self.cache.to(DEV), prefix_table=i(self.ptable), prefix_len=i([self.P]),
                    block_table=i(self.table), seq_lens=i(self.lens))

    def where(self, b):
        """Flat token index of request b's tokens; None for a token in a bad page."""
        out = []
        for t in range(min(max(self.lens[b], 0), self.table.shape[1] * self.bs)):
            page = int(self.ptable[t // self.bs] if t < self.P else self.table[b, t // self.bs])
            if 0 <= page < self.nb:
                out.append(page * self.bs + t % self.bs)
        return out

    def want(self):
        """(o, A) in 64 bits."""
        o = torch.zeros(self.q.shape, dtype=torch.float64, device=DEV)
        A = torch.zeros_like(o)
        cache, q = self.cache.to(DEV).flatten(1, 2), self.q.to(DEV).double()
        G = q.shape[1] // self.n_kv
        for b in range(self.B):
            w = self.where(b)
            if not w:
                continue
            k, v = cache[:, torch.tensor(w, device=DEV)].double()
            for h in range(self.n_kv):
                s = slice(h * G, h * G + G)
                p = torch.softmax(self.scale * q[b, s] @ k[:, h].T, -1)
                o[b, s], A[b, s] = p @ v[:, h], p @ v[:, h].abs()
        return o, A

    def check(self, got, what=""):
        o, A = self.want()
        u = torch.finfo(self.dtype).eps / 2
        up = 0.0 if self.dtype == torch.float32 else u
        tol = u * o.abs() + (up + 6e-5) * A + 1e-30
        # a request that is clamped to its row's capacity attends to NaN tokens: NaN is the formula's value
        bad = ~(((got.double() - o).abs() <= tol) | (o.isnan() & got.isnan()))
        assert not bool(bad.any()), (what, int(bad.sum()), float((got.double() - o).abs().max()),
                                     [int(x) for x in bad.nonzero()[0]])


def run(c, what="", expect_errors=0, **kw):
    d = c.dev()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    before = sra.wait_timeouts()
    got = sra.shared_prefix_attention(**d, scale=c.scale, err_count=err, **kw)
    torch.cuda.synchronize()
    assert sra.wait_timeouts() == before
    assert int(err.item()) == expect_errors, what
    c.check(got, what)
    return got


@pytest.fixture(params=["auto", "decode", "batched"])
def path(request):
    """The automatic choice, and each of the two paths forced."""
    sra.force_variant("shared_prefix", {"auto": -1, "decode": 0, "batched": 1}[request.param])
    yield request.param
    sra.force_variant("shared_prefix", -1)


def serves(path, dtype, hd, prefix_pages=1):
    return path != "batched" or prefix_pages > 0


def ragged(B, prefix, own, seed):
    r = np.random.default_rng(seed)
    lens = prefix + r.integers(0, own + 1, B)
    if B > 2:
        lens[r.integers(0, B)] = 0
        lens[r.integers(0, B)] = int(r.integers(0, prefix + 1))
    return lens


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("n_head,n_kv", [(8, 8), (12, 2), (21, 3), (8, 1)])
@pytest.mark.parametrize("bs", [8, 16, 32])
def test_shapes_dtypes(dtype, hd, n_head, n_kv, bs, path):
    if not serves(path, dtype, hd):
        pytest.skip("the prefix needs a page")
    B = {8: 5, 16: 19, 32: 40}[bs]
    prefix = {64: 200, 128: 391, 256: 128}[hd]
    run(Case(B, n_head, n_kv, hd, bs, prefix, ragged(B, prefix, 70, hd + bs), dtype, hd + bs + n_head))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 127, 128, 129, 256, 511, 640])
@pytest.mark.parametrize("B", [1, 2, 23, 65])
def test_prefix_lengths(dtype, prefix, B, path):
    if not serves(path, dtype, 128):
        pytest.skip("the prefix needs a page")
    run(Case(B, 12, 2, 128, 16, prefix, ragged(B, prefix, 40, prefix + B), dtype, prefix + B))


@pytest.mark.parametrize("hd,n_head,n_kv", [(128, 12, 2), (64, 32, 4), (128, 4, 4), (256, 8, 2)])
@pytest.mark.parametrize("B", [16, 64, 150])
def test_long_prefixes(hd, n_head, n_kv, B):
    run(Case(B, n_head, n_kv, hd, 16, 6000 + B, ragged(B, 6000 + B, 300, B), torch.bfloat16, B + hd))


@pytest.mark.parametrize("dtype,hd", [(torch.bfloat16, 128), (torch.float32, 64), (torch.float16, 256)])
def test_no_own_tokens_no_prefix_nothing(dtype, hd, path):
    if not serves(path, dtype, hd):
        pytest.skip("the prefix needs a page")
    run(Case(30, 8, 2, hd, 16, 300, [300] * 30, dtype, 1), "only the prefix")
    run(Case(30, 8, 2, hd, 16, 300, [0] * 30, dtype, 2), "no tokens at all")
    run(Case(30, 8, 2, hd, 16, 300, list(range(30)), dtype, 3), "all shorter than the prefix")
    run(Case(30, 8, 2, hd, 16, 0, list(range(30)), dtype, 4), "no prefix")
    c = Case(30, 8, 2, hd, 16, 0, [0] * 30, dtype, 5)
    assert not bool(run(c).any())


@pytest.mark.parametrize("dtype,hd", [(torch.bfloat16, 128), (torch.float16, 64), (torch.float32, 128)])
def test_peaked_scores(dtype, hd, path):
    """Scores of some hundreds: the running maximum moves many times and most weights vanish."""
    if not serves(path, dtype, hd):
        pytest.skip("the prefix needs a page")
    run(Case(40, 12, 2, hd, 16, 1000, ragged(40, 1000, 90, 7), dtype, 7, scale=1.0, spread=2.0))


@pytest.mark.parametrize("B,prefix,own", [(3, 9000, 40), (40, 9000, 40), (3, 64, 9000), (40, 64, 3000)])
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_many_small_probabilities(hd, B, prefix, own):
    """One token has nearly all of the weight and V = 0 (the first of the longer part), all the others 2^-25.5 of
    it each and V = 1. In fp16 the probabilities, at 2^7 relative to the largest, are subnormal here, with a step of 2^-24
    and an error of half of one: 2^-32 of the largest, per token, beside what every fp16 result is allowed (half a step of
    its own, 2^-25 or more, and the evaluation in fp32)."""
    c = Case(B, 12, 2, hd, 16, prefix, [prefix + own] * B, torch.float16, 3, scale=float(np.log(2.0)))
    c.q.zero_()
    c.q[..., 0] = 1
    some = ~c.cache[0].isnan().any(-1)
    for plane, value in ((0, 0.0), (1, 1.0)):
        c.cache[plane][some] = value
    c.cache[0][..., 0][some] = -5.5
    pages = [(c.ptable[0], 0)] if prefix > own else [(c.table[b, prefix // 16], 0) for b in range(B)]
    for page, at in pages:
        c.cache[0, page, at, :, 0], c.cache[1, page, at] = 20, 0
    sra.force_variant("shared_prefix", 1)
    try:
        got = sra.shared_prefix_attention(**c.dev(), scale=c.scale)
    finally:
        sra.force_variant("shared_prefix", -1)
    o, A = c.want()
    assert float(o.min()) > 3000 * 2.0 ** -26
    step = torch.maximum(2.0 ** -11 * o, torch.full_like(o, 2.0 ** -25))
    assert bool(((got.double() - o).abs() <= step + 6e-5 * A + (prefix + own) * 2.0 ** -32).all())


@pytest.mark.parametrize("dtype,hd", [(torch.bfloat16, 128), (torch.float16, 64), (torch.float32, 64),
                                      (torch.bfloat16, 256)])
def test_bad_entries_are_skipped_and_counted(dtype, hd, path):
    if not serves(path, dtype, hd):
        pytest.skip("the prefix needs a page")
    c = Case(33, 8, 2, hd, 16, 417, [600] * 33, dtype, 11)
    c.ptable[3], c.ptable[9] = -1, c.nb
    c.table[4, 30] = 2 ** 31 - 1
    c.table[5, 26] = -9        # the page in which the prefix ends, behind it
    c.lens[6] = -3
    c.lens[7] = c.table.shape[1] * c.bs + 1
    c.lens[8] = 100            # inside the prefix
    bad_of_7 = c.table.shape[1] - 38   # its row's entries behind its pages
    run(c, expect_errors=2 + 1 + 1 + 1 + 1 + bad_of_7)


def test_prefix_length_is_clamped(path):
    c = Case(20, 8, 2, 128, 16, 64, [64] * 20, torch.bfloat16, 12)
    d = c.dev()
    d["prefix_table"] = d["prefix_table"][:4].contiguous()
    for n, P in ((99999, 64), (-1, 0)):
        d["prefix_len"].fill_(n)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        if P == 0:
            d["block_table"][:, :4] = d["prefix_table"]
        got = sra.shared_prefix_attention(**d, scale=c.scale, err_count=err)
        assert int(err.item()) == 1
        c.check(got)


@pytest.mark.parametrize("dtype,hd", [(torch.bfloat16, 128), (torch.float32, 64)])
def test_strided_queries_and_outputs(dtype, hd, path):
    """q as a view of a fused QKV buffer, out as a view of a wider one whose other columns stay."""
    if not serves(path, dtype, hd):
        pytest.skip("the prefix needs a page")
    c = Case(50, 8, 2, hd, 16, 500, ragged(50, 500, 50, 3), dtype, 3)
    d = c.dev()
    qkv = torch.randn(50, 12, hd, device=DEV).to(dtype)
    qkv[:, :8] = d["q"]
    d["q"] = qkv[:, :8]
    wide = torch.full((50, 11, hd), 7.0, device=DEV, dtype=dtype)
    got = sra.shared_prefix_attention(**d, scale=c.scale, out=wide[:, 2:10])
    c.check(got)
    assert bool((wide[:, :2] == 7).all()) and bool((wide[:, 10:] == 7).all())


def test_queries_at_an_odd_element(path):
    c = Case(50, 8, 2, 128, 16, 500, ragged(50, 500, 50, 4), torch.bfloat16, 4)
    d = c.dev()
    flat = torch.empty(c.q.numel() + 1, device=DEV, dtype=torch.bfloat16)[1:]
    d["q"] = flat.copy_(d["q"].reshape(-1)).view(c.q.shape)
    out = torch.empty(c.q.numel() + 1, device=DEV, dtype=torch.bfloat16)[1:].view(c.q.shape)
    if path == "batched":   # wants query rows aligned to 4 bytes
        with pytest.raises(sra.SRAError) as e:
            sra.shared_prefix_attention(**d, scale=c.scale, out=out)
        assert e.value.status == -7
        return
    c.check(sra.shared_prefix_attention(**d, scale=c.scale, out=out))


@pytest.mark.parametrize("off", [2, 4])
def test_queries_at_4_and_8_bytes(off, path):
    c = Case(50, 8, 2, 128, 16, 500, ragged(50, 500, 50, 4), torch.bfloat16, 4)
    d = c.dev()
    flat = torch.empty(c.q.numel() + off, device=DEV, dtype=torch.bfloat16)[off:]
    d["q"] = flat.copy_(d["q"].reshape(-1)).view(c.q.shape)
    c.check(sra.shared_prefix_attention(**d, scale=c.scale))


def test_negative_and_zero_scale(path):
    for scale in (-0.09, 0.0):
        run(Case(30, 8, 2, 64, 16, 300, ragged(30, 300, 50, 8), torch.float16, 8, scale=scale))


def test_equals_decode_attention_on_forked_rows(path):
    """Rows that hold the prefix's pages themselves: the same call, the same answer within both tolerances."""
    c = Case(24, 12, 2, 128, 16, 1024, 1024 + np.arange(24) * 5, torch.bfloat16, 6)
    c.table[:, :64] = c.ptable[:64]
    d = c.dev()
    a = sra.shared_prefix_attention(**d)
    b = sra.paged_decode_attention(d["q"], d["kv_cache"], d["block_table"], d["seq_lens"])
    c.check(a)
    c.check(b)
    d["prefix_table"] = d["block_table"][3].contiguous()   # a row of the table as the prefix's table
    c.check(sra.shared_prefix_attention(**d))   # (its length sets the splits, so the sums' order may differ)


@pytest.mark.parametrize("pdl", [False, True])
def test_graph_replay_with_new_lengths(pdl, path):
    """One captured call: prefix, lengths, tables and queries change between replays; two graphs with a
    workspace each do not disturb one another."""
    a = Case(70, 12, 2, 128, 16, 800, ragged(70, 800, 100, 1), torch.bfloat16, 1, extra_cols=40)
    d = a.dev()
    prev = sra.set_pdl(pdl)
    try:
        graphs = []
        for _ in range(2):
            ws = sra.shared_prefix_workspace(70, 12, 2, 128, d["prefix_table"].numel(), a.table.shape[1], 16,
                                             torch.bfloat16, DEV)
            out = torch.empty_like(d["q"])
            sra.shared_prefix_attention(**d, scale=a.scale, out=out, workspace=ws)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                sra.shared_prefix_attention(**d, scale=a.scale, out=out, workspace=ws)
            graphs.append((g, out, ws))
    finally:
        sra.set_pdl(prev)
    for g, out, _ in graphs:
        out.zero_()
        g.replay()
        a.check(out)
    d["seq_lens"].copy_(torch.tensor(ragged(70, 400, 0, 9), dtype=torch.int32))
    d["prefix_len"].fill_(400)
    a.lens, a.P = d["seq_lens"].cpu().tolist(), 400
    d["q"].copy_(torch.randn(d["q"].shape, device=DEV))
    a.q = d["q"].cpu()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs[0][0].replay()
    with torch.cuda.stream(s):
        graphs[1][0].replay()
    torch.cuda.synchronize()
    for _, out, _ in graphs:
        a.check(out)


def test_same_result_every_time_and_on_another_stream(path):
    c = Case(64, 12, 2, 128, 16, 3000, ragged(64, 3000, 200, 5), torch.bfloat16, 5)
    d = c.dev()
    first = sra.shared_prefix_attention(**d, scale=c.scale)
    c.check(first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (None, s, s.cuda_stream):
        out = torch.empty_like(first)
        sra.shared_prefix_attention(**d, scale=c.scale, out=out, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out, first)


@pytest.mark.parametrize("dtype,hd,B", [(torch.bfloat16, 128, 64), (torch.float16, 64, 21), (torch.bfloat16, 128, 43),
                                        (torch.bfloat16, 256, 21)])
def test_calls_in_a_row_on_cold_caches(dtype, hd, B):
    """Calls that nothing waits between, on caches in turn that do not fit the L2 together and on workspaces that
    hold NaN: copies of K and V arrive late and out of order, whatever is taken too early shows. The rows
    are an odd number of tiles (the last has both streams on tiles of its own), several laps of the ring long."""
    cases = [Case(B, 48, 8, hd, 16, 2900 + 16 * k, ragged(B, 2900, 60, k), dtype, k) for k in range(2)]
    d = [c.dev() for c in cases]
    far = [torch.empty(2, 6 * c.nb, 16, 8, hd, dtype=dtype, device=DEV) for c in cases for _ in range(3)]
    for k, f in enumerate(far):     # the same pages, six times as far apart
        f.fill_(float("nan"))
        f[:, ::6] = d[k // 3]["kv_cache"]
    six = lambda t: torch.where((t >= 0) & (t < 1 << 20), t * 6, t)
    calls = []
    for k, f in enumerate(far):
        x = dict(d[k // 3], kv_cache=f)
        x["prefix_table"], x["block_table"] = six(x["prefix_table"]), six(x["block_table"])
        calls.append(x)
    want = [sra.shared_prefix_attention(**d[i], scale=cases[i].scale) for i in range(2)]
    for c, w in zip(cases, want):
        c.check(w)
    ws = [sra.shared_prefix_workspace(B, 48, 8, hd, x["prefix_table"].numel(), x["block_table"].shape[1], 16, dtype, DEV)
          for x in calls]
    before = sra.wait_timeouts()
    for _ in range(20):
        for w in ws:
            w.view(torch.uint8).fill_(255)
        got = [sra.shared_prefix_attention(**x, scale=cases[0].scale, workspace=w) for x, w in zip(calls, ws)]
        again = [sra.shared_prefix_attention(**x, scale=cases[0].scale, workspace=w) for x, w in zip(calls, ws)]
        torch.cuda.synchronize()
        for k in range(len(calls)):
            assert torch.equal(got[k], want[k // 3]) and torch.equal(again[k], want[k // 3]), k
    assert sra.wait_timeouts() == before


@pytest.mark.parametrize("pdl", [False, True])
def test_calls_at_once_beside_other_tensor_memory_users(pdl):
    """Calls on two streams, each with a workspace of its own, beside projections on a third: all of them
    allocate tensor memory on the SMs that they share, and each gives what it gives alone."""
    cs = [Case(64, 12, 2, 128, 16, 3000, ragged(64, 3000, 200, 5), torch.bfloat16, 5),
          Case(30, 32, 4, 64, 32, 2500, ragged(30, 2500, 100, 6), torch.float16, 6)]
    x = torch.randn(64, 1536, device=DEV).to(torch.bfloat16)
    w, W = torch.ones(1536, device=DEV, dtype=torch.bfloat16), torch.randn(2048, 1536, device=DEV).to(torch.bfloat16)
    lw = sra.linear_workspace(64, 1536, torch.bfloat16, DEV, N=2048)
    prev = sra.set_pdl(pdl)
    try:
        calls = []
        for c in cs:
            d = c.dev()
            ws = sra.shared_prefix_workspace(c.B, c.q.shape[1], c.n_kv, c.hd, d["prefix_table"].numel(),
                                             d["block_table"].shape[1], c.bs, c.dtype, DEV)
            assert ws is not None
            out = torch.empty_like(d["q"])
            calls.append((lambda s, d=d, ws=ws, out=out, c=c: sra.shared_prefix_attention(
                **d, scale=c.scale, workspace=ws, out=out, stream=s), out))
        y = torch.empty(64, 2048, device=DEV, dtype=torch.bfloat16)
        calls.append((lambda s: sra.rmsnorm_linear(x, w, W, y, workspace=lw, stream=s), y))
        want = []
        for call, out in calls:
            call(None)
            torch.cuda.synchronize()
            want.append(out.clone())
        for c, v in zip(cs, want):
            c.check(v)
        streams = [torch.cuda.Stream() for _ in calls]
        for _ in range(10):
            for _, out in calls:
                out.fill_(float("nan"))
            torch.cuda.synchronize()
            for _ in range(20):
                for (call, _), s in zip(calls, streams):
                    call(s)
            torch.cuda.synchronize()
            for (_, out), v in zip(calls, want):
                assert torch.equal(out, v)
        assert sra.wait_timeouts() == 0
    finally:
        sra.set_pdl(prev)


@pytest.mark.parametrize("dtype,hd", [(torch.bfloat16, 128), (torch.float16, 256), (torch.float32, 64)])
def test_cache_past_32_bit_offsets(dtype, hd, path):
    """The pages of a small cache at the far end of one whose planes have more than 2^31 elements: the same result."""
    c = Case(40, 48, 8, hd, 16, 1500, ragged(40, 1500, 60, 7), dtype, 7)
    d = c.dev()
    want = sra.shared_prefix_attention(**d, scale=c.scale)
    c.check(want)
    nb = 2 ** 31 // (16 * 8 * hd) + c.nb
    far = torch.empty(2, nb, 16, 8, hd, dtype=dtype, device=DEV)
    far[:, -c.nb:] = d["kv_cache"]
    move = lambda t: torch.where((t >= 0) & (t < c.nb), t + (nb - c.nb), t)
    d["kv_cache"], d["prefix_table"], d["block_table"] = far, move(d["prefix_table"]), move(d["block_table"])
    assert torch.equal(sra.shared_prefix_attention(**d, scale=c.scale), want)


def test_refusals():
    c = Case(8, 8, 2, 128, 16, 100, [120] * 8, torch.bfloat16, 2)
    d = c.dev()
    for k, v in (("prefix_len", d["prefix_len"].long()), ("prefix_len", d["seq_lens"]),
                 ("prefix_table", d["prefix_table"].cpu()), ("prefix_table", d["block_table"]),
                 ("block_table", d["block_table"].long()), ("q", d["q"].half()), ("seq_lens", d["seq_lens"][:3])):
        with pytest.raises(ValueError):
            sra.shared_prefix_attention(**{**d, k: v})
    with pytest.raises(sra.SRAError) as e:
        sra.shared_prefix_attention(**d, out=d["q"])
    assert e.value.status == -5
    with pytest.raises(sra.SRAError) as e:
        sra.shared_prefix_attention(**d, scale=float("inf"))
    assert e.value.status == -6


def test_a_prompt_and_its_samples(path):
    """The operators together, as a sampling loop uses them: a prompt is stored, forked into samples,
    each step grows the rows (the shared last page copied once), stores the new token's K and V by
    rope_kv_store's own slots and attends; then some samples end, the cache is compacted, and the
    attention of the others is what it was. Row 0 keeps the prompt (it does not grow), so the page in
    which the prompt ends stays held while the prefix's table names it."""
    torch.manual_seed(3)
    n_head, n_kv, hd, bs, nb, L = 12, 2, 128, 16, 120, 2
    rows, M, prompt, n = 20, 24, 197, 18
    caches = [torch.full((2, nb, bs, n_kv, hd), float("nan"), device=DEV, dtype=torch.bfloat16) for _ in range(L)]
    i = lambda a: torch.as_tensor(np.asarray(a), dtype=torch.int32).to(DEV)
    table, seq, ref = i(np.full((rows, M), -1)), i([0] * rows), i([0] * nb)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    cos, sin = torch.ones(512, hd // 2, device=DEV), torch.zeros(512, hd // 2, device=DEV)   # no rotation

    def store(layer, kv, pos, slot):
        sra.rope_kv_store(torch.zeros(len(pos), n_head, hd, device=DEV, dtype=torch.bfloat16), kv[0], kv[1], cos, sin,
                          pos, slot, caches[layer], err_count=err)

    def draw(t):
        return torch.randn(2, t, n_kv, hd, device=DEV).to(torch.bfloat16)

    sra.resize_kv_rows(table, seq, ref, i([0]), i([prompt]), caches, err_count=err)
    t = torch.arange(prompt, device=DEV)
    slots = table[0].long()[t // bs] * bs + t % bs
    history = [[None] * rows for _ in range(L)]
    for layer in range(L):
        kv = draw(prompt)
        store(layer, kv, t, slots)
        for r in range(n):
            history[layer][r] = kv
    sra.fork_kv_rows(table, seq, ref, i([0] * (n - 1)), i(range(1, n)), bs, err_count=err)
    ptable, plen = table[0].clone(), i([prompt])
    samples = list(range(1, n))
    live = i(samples)

    def attend(layer, r):
        q = torch.randn(len(r), n_head, hd, device=DEV, generator=torch.Generator(DEV).manual_seed(layer)).to(torch.bfloat16)
        sel = torch.tensor(r, device=DEV)
        got = sra.shared_prefix_attention(q, caches[layer], ptable, plen, table[sel].contiguous(),
                                          seq[sel].contiguous(), err_count=err)
        for k, row in enumerate(r):
            K, V = history[layer][row].double()
            for h in range(n_head):
                g = h // (n_head // n_kv)
                p = torch.softmax(q[k, h].double() @ K[:, g].T / hd ** 0.5, -1)
                o, A = p @ V[:, g], p @ V[:, g].abs()
                assert bool(((got[k, h].double() - o).abs() <= 2 ** -8 * o.abs() + (2 ** -8 + 6e-5) * A).all())
        return got

    for step in range(1, 14):
        pos, slot = sra.resize_kv_rows(table, seq, ref, live, i([prompt + step] * (n - 1)), caches,
                                       err_count=err)
        for layer in range(L):
            kv = draw(n - 1)
            store(layer, kv, pos, slot)
            for k, r in enumerate(samples):
                history[layer][r] = torch.cat([history[layer][r], kv[:, k:k + 1]], 1)
        if step in (1, 2, 11, 12, 13):
            attend(step % L, samples)
    left = [2, 3, 5, 7, 11, 13]
    before = [attend(layer, left) for layer in range(L)]
    gone = [r for r in samples if r not in left]
    sra.resize_kv_rows(table, seq, ref, i(gone), i([0] * len(gone)), caches, err_count=err)
    alive = sra.compact_kv_pages(table, seq, ref, caches, err_count=err)
    assert int(alive.item()) == 13 + len(left) * 2 and bool((ref[int(alive.item()):] == 0).all())
    ptable = table[0].clone()
    after = [attend(layer, left) for layer in range(L)]
    for x, y in zip(before, after):
        assert torch.equal(x, y)
    assert int(err.item()) == 0
