"""GPU: the quantised cache's calls in company: other streams, two calls at once, graphs, programmatic launches, caches past
2^32 bytes, batches at the forms' borders, long requests.

Results are compared bit for bit with the same call alone, on the current stream or in a small cache; values with the
formula in 64 bits, within the tolerances of the attention's tests.
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


def random_cache(nb, bs, n_kv, hd, fmt, seed, device=DEV):
    x = np.random.default_rng(seed).standard_normal((2, nb, n_kv, bs, hd)).astype(np.float32)
    return torch.tensor(qm.encode(x.astype(np.float64), fmt)).to(device)


def forced(variant):
    class Force:
        def __enter__(self):
            sra.force_variant("decode_attention_quant", variant)

        def __exit__(self, *_):
            sra.force_variant("decode_attention_quant", -1)
    return Force()


class Batch:
    """q, a cache, a table and lengths; the three calls over them."""

    def __init__(self, lens, n_head=6, n_kv=2, hd=128, bs=16, fmt="e2m1", dtype=BF, seed=0, spare=0):
        g = torch.Generator().manual_seed(seed)
        self.n_head, self.n_kv, self.hd, self.bs, self.fmt, self.dtype = n_head, n_kv, hd, bs, fmt, dtype
        mb = max(1, -(-max(lens) // bs)) + spare
        nb = len(lens) * mb
        self.cache = random_cache(nb, bs, n_kv, hd, fmt, seed)
        self.table = i32(np.random.default_rng(seed).permutation(nb).reshape(len(lens), mb))
        self.lens, self.cu = i32(lens), i32(np.concatenate([[0], np.cumsum(lens)]))
        self.total = int(sum(lens))
        self.q = torch.randn(len(lens), n_head, hd, generator=g).to(dtype).to(DEV)
        self.k, self.v = (torch.randn(len(lens), n_kv, hd, generator=g).to(dtype).to(DEV) for _ in "kv")
        a = torch.rand(64, hd // 2, generator=g) * 6
        self.cos, self.sin = a.cos().to(DEV), a.sin().to(DEV)
        self.pos = i64(np.arange(len(lens)) % 64)
        self.slot = self.table[:, -1].long() * bs + bs - 1

    def workspace(self):
        B, mb = self.table.shape
        return sra.decode_attention_quant_workspace(B, self.n_head, self.n_kv, self.hd, mb, self.bs, self.fmt, self.dtype, DEV)

    def store(self, q=None, **kw):
        sra.rope_kv_store_quant(self.q if q is None else q, self.k, self.v, self.cos, self.sin, self.pos, self.slot, self.cache, **kw)

    def attend(self, q=None, **kw):
        return sra.paged_decode_attention_quant(self.q if q is None else q, self.cache, self.table, self.lens, **kw)

    def read(self, **kw):
        return sra.read_kv_quant(self.cache, self.table, self.cu, self.total, self.hd, self.dtype, **kw)


def same(a, b):
    return a.dtype == b.dtype and a.shape == b.shape and torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


CALLS = {"attend": lambda b, s: [b.attend(stream=s)], "read": lambda b, s: list(b.read(stream=s))}


@pytest.fixture(params=["attend", "read"])
def call(request):
    b = Batch([100, 3, 128, 0, 77])
    torch.cuda.synchronize()
    return lambda s: CALLS[request.param](b, s)


@pytest.mark.parametrize("kind", ["object", "integer"])
def test_results_are_the_streams_own_memory(call, kind):
    s = torch.cuda.Stream()
    want = call(None)
    torch.cuda.synchronize()
    freed = [torch.empty_like(t) for t in want]
    ptrs = {t.data_ptr() for t in freed}
    del freed
    got = call(s if kind == "object" else s.cuda_stream)
    assert not ptrs & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    assert all(same(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("which", ["object", "integer", "default object", "default integer"])
def test_memory_is_filed_under_the_calls_stream(call, which):
    side, here = torch.cuda.Stream(), torch.cuda.Stream()
    s = torch.cuda.default_stream() if which.startswith("default") else side
    with torch.cuda.stream(here):
        got = call(s if which.endswith("object") else s.cuda_stream)
    torch.cuda.synchronize()
    segments = torch.cuda.memory_snapshot()
    for t in got:
        (owner,) = [g["stream"] for g in segments if g["address"] <= t.data_ptr() < g["address"] + g["total_size"]]
        assert owner == s.cuda_stream


def test_a_dropped_result_waits_for_the_current_stream(call):
    s = torch.cuda.Stream()
    for t in call(s):
        del t
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    got = call(s)
    shapes, ptrs = [(t.shape, t.dtype) for t in got], {t.data_ptr() for t in got}
    del got
    with torch.cuda.stream(s):
        again = [torch.empty(a[0], dtype=a[1], device=DEV) for a in shapes]
    assert not torch.cuda.current_stream().query(), "the work on the current stream ended before the check"
    assert not ptrs & {t.data_ptr() for t in again}
    torch.cuda.synchronize()


@pytest.mark.parametrize("variant", [0, 1])
def test_two_calls_at_once(variant):
    """Two batches on two streams, each with a workspace of its own, again and again."""
    with forced(variant):
        bs = [Batch([3000, 17, 900, 0, 2222] * 2, seed=1), Batch([5000, 1, 40] * 3, n_head=8, n_kv=1, dtype=HF, fmt="int8", seed=2)]
        ws = [b.workspace() for b in bs]
        want = [(b.attend(workspace=w), *b.read()) for b, w in zip(bs, ws)]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in bs]
        for _ in range(10):
            got = [(b.attend(workspace=w, stream=s), *b.read(stream=s)) for b, w, s in zip(bs, ws, streams)]
            torch.cuda.synchronize()
            assert all(same(x, y) for g, w in zip(got, want) for x, y in zip(g, w))


@pytest.mark.parametrize("variant", [0, 1])
@pytest.mark.parametrize("pdl", [False, True])
def test_a_graph_of_the_three(variant, pdl):
    """Store, attention and read in one graph, replayed over inputs, lengths and tables that change in place."""
    with forced(variant):
        b = Batch([700, 33, 0, 1500], seed=3, spare=1)
        w, q, out = b.workspace(), b.q.clone(), torch.empty_like(b.q)
        room = tuple(torch.zeros(2500, 2, 128, dtype=BF, device=DEV) for _ in "kv")
        err = torch.zeros(1, dtype=torch.int32, device=DEV)

        def step():
            b.store(q, err_count=err)
            b.attend(q, out=out, workspace=w, err_count=err)
            sra.read_kv_quant(b.cache, b.table, b.cu, 2500, 128, out=room, err_count=err)
        old = sra.set_pdl(pdl)
        try:
            start, q0 = b.cache.clone(), b.q.clone()
            step()
            torch.cuda.synchronize()
            g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
            with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
                step()
            r = np.random.default_rng(4)
            for k in range(6):
                lens = r.integers(0, 1500, 4) if k else np.zeros(4, dtype=int)
                b.lens.copy_(i32(lens))
                b.cu.copy_(i32(np.minimum(np.concatenate([[0], np.cumsum(lens)]), 2500)))
                b.slot.copy_(b.table[torch.arange(4, device=DEV), (b.lens // 16).long()].long() * 16 + b.lens % 16)
                b.lens += 1
                b.k.copy_(torch.randn(b.k.shape, device=DEV).to(BF))
                results = []
                for run in (step, g.replay):
                    b.cache.copy_(start)
                    q.copy_(q0)
                    out.fill_(9)
                    for t in room:
                        t.fill_(-9)
                    run()
                    torch.cuda.synchronize()
                    results.append([t.clone() for t in (b.cache, q, out, *room)])
                assert all(same(x, y) for x, y in zip(*results))
                assert not same(results[0][0], start)
            assert int(err.item()) == 0
        finally:
            sra.set_pdl(old)


def test_a_chain_of_launches():
    """A decode step's calls in a row under programmatic launches: each sees what the ones before wrote."""
    b = Batch([400, 90, 1, 1200], seed=5)
    w, start = b.workspace(), b.cache.clone()

    def chain():
        b.cache.copy_(start)
        q, keep = b.q.clone(), []
        for k in range(4):
            b.store(q)
            q = b.attend(q, workspace=w)
            keep += [q, *b.read()]
            b.k, b.v = q[:, :2].contiguous(), q[:, 2:4].contiguous()
        return [*keep, b.cache.clone()]
    k0, v0 = b.k, b.v
    old = sra.set_pdl(False)
    try:
        want = chain()
        torch.cuda.synchronize()
        sra.set_pdl(True)
        for _ in range(10):
            b.k, b.v = k0, v0
            got = chain()
            torch.cuda.synchronize()
            assert all(same(x, y) for x, y in zip(got, want))
    finally:
        sra.set_pdl(old)


@pytest.mark.parametrize("variant", [0, 1])
def test_offsets_past_32_bits(variant):
    """Planes of more than 2^32 bytes: the same bytes and results as in a small cache."""
    n_kv, bs, hd, fmt, nb = 8, 32, 256, "int8", 62000
    small = Batch([100, 31, 64, 200], n_head=16, n_kv=n_kv, hd=hd, bs=bs, fmt=fmt, seed=6)
    big = torch.empty((2, nb, n_kv, bs, qm.row_bytes(fmt, hd)), dtype=torch.uint8, device=DEV)
    assert big[0].numel() > 2 ** 32
    there = i64(nb - 1 - 7 * np.arange(small.cache.shape[1]))     # where the small cache's pages lie in the big one
    there[::2] = there[::2] - 61000
    big[:, there] = small.cache
    with forced(variant):
        table = there[small.table.long()].int()
        w = small.workspace()
        q2 = small.q.clone()
        small.store()
        sra.rope_kv_store_quant(q2, small.k, small.v, small.cos, small.sin, small.pos, there[small.slot // bs] * bs + small.slot % bs, big)
        assert same(q2, small.q) and same(big[:, there], small.cache)
        got = sra.paged_decode_attention_quant(q2, big, table, small.lens, workspace=w)
        assert same(got, small.attend(workspace=w))
        for x, y in zip(sra.read_kv_quant(big, table, small.cu, small.total, hd), small.read()):
            assert same(x, y)
    # pages copied across the border
    sra.copy_kv_pages(big, i32([int(there[0]), int(there[1])]), i32([nb - 2, 3]))
    assert same(big[:, nb - 2], small.cache[:, 0]) and same(big[:, 3], small.cache[:, 1])


def test_more_than_2_31_tasks():
    """A store of so many tokens that their tasks pass 2^31: first, middle and last tokens as in a small call."""
    n_head, hd, bs, few = 8, 64, 16, 70
    T = 2 ** 31 // (n_head * (hd // 16)) + few
    if torch.cuda.mem_get_info()[0] < 110 << 30:
        pytest.skip("needs 90 GB of device memory")
    small = Batch([1] * (3 * few), n_head=n_head, n_kv=1, hd=hd, bs=bs, dtype=HF, seed=11)
    at = torch.cat([torch.arange(few), torch.arange(T // 2, T // 2 + few), torch.arange(T - few, T)]).to(DEV)
    q, k, v = (torch.empty(T, n, hd, dtype=HF, device=DEV) for n in (n_head, 1, 1))
    pos, slot = torch.full((T,), -1, device=DEV), torch.full((T,), -1, device=DEV)     # (the others' positions are bad: left alone)
    q[at], k[at], v[at], pos[at], slot[at] = small.q, small.k, small.v, small.pos, small.slot
    cache, err = small.cache.clone(), torch.zeros(1, dtype=torch.int32, device=DEV)
    sra.rope_kv_store_quant(q, k, v, small.cos, small.sin, pos, slot, cache, err_count=err)
    small.store()
    assert int(err.item()) == T - 3 * few
    assert same(q[at], small.q) and same(cache, small.cache)


@pytest.mark.parametrize("B,variant", [(65536, 0), (65536, 1), (65537, 0), (100000, 0)])
def test_batches_at_the_border(B, variant):
    """As many requests as the stream form takes, and more: most of them empty or of a token or two."""
    r = np.random.default_rng(B)
    nb, bs, hd = 97, 8, 64
    cache = random_cache(nb, bs, 1, hd, "e2m1", 7)
    lens = r.integers(0, 4, B)
    lens[B // 2], lens[-1] = 8, 1
    table = r.integers(0, nb, (B, 1))
    q = torch.randn(B, 2, hd, generator=torch.Generator().manual_seed(B)).to(HF)
    with forced(variant):
        w = sra.decode_attention_quant_workspace(B, 2, 1, hd, 1, bs, "e2m1", HF, DEV)
        assert (w is not None) == (variant == 1)
        got = sra.paged_decode_attention_quant(q.to(DEV), cache, i32(table), i32(lens), workspace=w).double().cpu().numpy()
    kv = qm.decode(cache.cpu().numpy()[:, :, 0], "e2m1", hd)[:, table[:, 0]]      # [2, B, bs, hd]
    s = np.einsum("bhd,btd->bht", q.double().numpy(), kv[0]) * hd ** -0.5
    p = np.where(np.arange(bs) < lens[:, None, None], np.exp(s), 0.0)
    p /= np.maximum(p.sum(-1, keepdims=True), 1e-300)
    o, A = (np.einsum("bht,btd->bhd", p, x) for x in (kv[1], np.abs(kv[1])))
    assert (np.abs(got - o) <= 2.0 ** -11 * np.abs(o) + (2.0 ** -11 + 6e-5) * A + 2.0 ** -25 + 2.0 ** -39 * 8 * 6).all()
    assert (got[lens == 0] == 0).all()
    with forced(1):
        w = sra.decode_attention_quant_workspace(65537, 2, 1, hd, 1, bs, "e2m1", HF, DEV)
        assert w is None        # (no stream form for so many)


@pytest.mark.parametrize("fmt,dtype", [("e2m1", BF), ("int8", F32)])
@pytest.mark.parametrize("variant", [0, 1])
def test_a_long_request(fmt, dtype, variant):
    """A request of 200,001 tokens beside short ones."""
    with forced(variant):
        n, hd, bs = 200001, 64, 16
        mb = -(-n // bs)
        cache = random_cache(mb, bs, 1, hd, fmt, 8)
        table = np.stack([np.random.default_rng(9).permutation(mb) for _ in range(3)])
        lens = [5, n, 0]
        q = torch.randn(3, 4, hd, generator=torch.Generator().manual_seed(9)).to(dtype)
        w = sra.decode_attention_quant_workspace(3, 4, 1, hd, mb, bs, fmt, dtype, DEV)
        got = sra.paged_decode_attention_quant(q.to(DEV), cache, i32(table), i32(lens), workspace=w).double().cpu().numpy()
        host = cache.cpu().numpy()[:, :, 0]
        u, up = torch.finfo(dtype).eps / 2, 2.0 ** -22 if dtype == F32 else 2.0 ** -11
        for b in (0, 1):
            k, v = qm.decode(host[:, table[b]].reshape(2, mb * bs, -1)[:, :lens[b]], fmt, hd)
            s = q[b].double().numpy() @ k.T * hd ** -0.5
            p = np.exp(s - s.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            o, A, S = p @ v, p @ np.abs(v), np.abs(v).sum(0)
            assert (np.abs(got[b] - o) <= u * np.abs(o) + (up + 6e-5) * A + 2.0 ** -39 * S + 1e-30).all()
        assert (got[2] == 0).all()


@pytest.mark.parametrize("fmt,hd,bs,n_kv", [("e2m1", 64, 5, 3), ("int8", 128, 16, 2), ("e2m1", 256, 1, 1)])
def test_pages_of_bytes(fmt, hd, bs, n_kv):
    """Pages copied as bytes, whatever their size: within layers, of a table's shared last page, moved together."""
    nb, layers = 12, 2
    caches = torch.stack([random_cache(nb, bs, n_kv, hd, fmt, s) for s in range(layers)])
    before = caches.clone()
    sra.copy_kv_pages(caches, i32([0, 5, 11]), i32([7, 1, 2]))
    want = before.clone()
    want[:, :, [7, 1, 2]] = before[:, :, [0, 5, 11]]
    assert torch.equal(caches, want)
    table, seq, ref = i32(np.full((3, 4), -1)), i32([0] * 3), i32([0] * nb)
    n = 2 * bs + 1 if bs > 1 else 3
    sra.resize_kv_rows(table, seq, ref, i32([0]), i32([n]), caches)
    sra.fork_kv_rows(table, seq, ref, i32([0]), i32([1]), bs)
    sra.resize_kv_rows(table, seq, ref, i32([1]), i32([n + 1]), caches)
    a, b = table[0].tolist(), table[1].tolist()
    assert a[:2] == b[:2]
    if bs > 1:      # the page that both would write: row 1 has a copy
        assert a[2] != b[2] and torch.equal(caches[:, :, a[2]], caches[:, :, b[2]])
    kept = [caches[:, :, p].clone() for p in table[1].tolist() if p >= 0]
    sra.resize_kv_rows(table, seq, ref, i32([0]), i32([0]), caches)
    sra.compact_kv_pages(table, seq, ref, caches)
    assert all(torch.equal(caches[:, :, p], x) for p, x in zip(table[1].tolist(), kept))


def test_refusals():
    """What the documentation rules out, before anything runs."""
    b = Batch([40, 3], seed=10)
    q, c, t, n = b.q, b.cache, b.table, b.lens
    out = torch.full_like(q, 5.0)
    attend, read = sra.paged_decode_attention_quant, sra.read_kv_quant
    bad = [lambda: attend(q, c.view(torch.int8), t, n, out=out), lambda: attend(q, c.transpose(2, 3), t, n, out=out),
           lambda: attend(q[..., :64], c, t, n, out=out[..., :64]), lambda: attend(q, c, t.long(), n, out=out),
           lambda: attend(q, c, t, n[:1], out=out), lambda: attend(q, c, t[:1], n, out=out), lambda: attend(q.double(), c, t, n),
           lambda: attend(q, c, t, n, out=out.float()), lambda: attend(q, c, t, n, out=out[:, :5]),
           lambda: attend(q, c.cpu(), t, n, out=out), lambda: attend(q, c, t, n, out=out, workspace=torch.empty(64)),
           lambda: attend(q, c, t, n, out=q), lambda: attend(q, c, t, n, out=out, scale=float("nan")),
           lambda: attend(q[:, :5], c, t, n, out=out[:, :5]), lambda: attend(q.repeat(1, 3, 1), c, t, n),
           lambda: read(c, t, b.cu[:2], 43, 128, out=(out, out)), lambda: read(c, t, b.cu, 43, 64), lambda: read(c, t, b.cu, 43, 128, torch.int8),
           lambda: read(c, t, b.cu, 43, 128, starts=n[:1]), lambda: read(c, t, b.cu, 43, 128, out=(b.k, b.v)),
           lambda: sra.rope_kv_store_quant(q, b.k[:1], b.v, b.cos, b.sin, b.pos, b.slot, c),
           lambda: sra.rope_kv_store_quant(q, b.k, b.v.float(), b.cos, b.sin, b.pos, b.slot, c),
           lambda: sra.rope_kv_store_quant(q, b.k, b.v, b.cos, b.sin, b.pos.int(), b.slot, c),
           lambda: sra.rope_kv_store_quant(q, b.k, b.v, b.cos[:, :32], b.sin, b.pos, b.slot, c),
           lambda: sra.rope_kv_store_quant(q, b.k, b.v, b.cos, b.sin, b.pos, b.slot, c, max_pos=65),
           lambda: sra.rope_kv_store_quant(q, q[:, :2], b.v, b.cos, b.sin, b.pos, b.slot, c),
           lambda: sra.rope_kv_store_quant(q, b.k, b.v, b.cos, b.sin, b.pos, b.slot, c, style="other")]
    before = [x.clone() for x in (q, c)]
    for k, f in enumerate(bad):
        with pytest.raises((ValueError, sra.SRAError)):
            f()
            pytest.fail(f"call {k} was not refused")
    torch.cuda.synchronize()
    assert same(q, before[0]) and same(c, before[1]) and (out == 5.0).all()
