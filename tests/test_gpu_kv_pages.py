"""GPU: pages of the cache (copy, fork, resize, compact) against the plain model.

Everything is whole numbers or moved bits, so every comparison is exact: tables, lengths, counts,
positions, slots, error counts and the caches' bit patterns (sentinel NaNs among them), including
the words that a call must not touch."""
import numpy as np
import pytest
import torch

import swiglu_rmsnorm_add_gb300 as sra
from tests import kv_model as m

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BIG = 2 ** 31 - 1


def i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).to(DEV)


def make_caches(layers, nb, bs, n_kv, hd, dtype, seed):
    """Random bit patterns (every NaN and infinity among them)."""
    g = torch.Generator().manual_seed(seed)
    t = torch.int32 if dtype == torch.float32 else torch.int16
    info = torch.iinfo(t)
    return [torch.randint(info.min, info.max, (2, nb, bs, n_kv, hd), dtype=t, generator=g).view(dtype)
            for _ in range(layers)]


class Both:
    """One state on the GPU and in the model, driven by the same calls."""

    def __init__(self, st, caches):
        self.st, self.caches = st, caches
        self.dev_caches = [c.to(DEV) for c in caches]
        self.table, self.seq, self.ref = i32(st.table), i32(st.seq), i32(st.ref)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.errors = 0

    def check(self, what):
        torch.cuda.synchronize()
        assert self.table.cpu().tolist() == self.st.table.tolist(), what
        assert self.seq.cpu().tolist() == self.st.seq.tolist(), what
        assert self.ref.cpu().tolist() == self.st.ref.tolist(), what
        assert int(self.err.item()) == self.errors, what
        for g, c in zip(self.dev_caches, self.caches):
            assert torch.equal(m.bits(g.cpu()), m.bits(c)), what

    def fork(self, parents, children, **kw):
        self.errors += m.fork(self.st, parents, children)
        sra.fork_kv_rows(self.table, self.seq, self.ref, i32(parents), i32(children), self.st.bs,
                         err_count=self.err, **kw)
        self.check("fork")

    def resize(self, rows, lens, **kw):
        errors, pos, slot = m.resize(self.st, rows, lens, self.caches)
        self.errors += errors
        p, s = sra.resize_kv_rows(self.table, self.seq, self.ref, i32(rows), i32(lens), self.dev_caches,
                                  err_count=self.err, **kw)
        self.check("resize")
        assert p.cpu().tolist() == pos.tolist() and s.cpu().tolist() == slot.tolist()

    def compact(self, **kw):
        errors, live = m.compact(self.st, self.caches)
        self.errors += errors
        n = sra.compact_kv_pages(self.table, self.seq, self.ref, self.dev_caches, err_count=self.err, **kw)
        self.check("compact")
        assert n.cpu().tolist() == [live]


def empty(rows, M, nb, bs):
    return m.State(np.full((rows, M), -1), np.zeros(rows), np.zeros(nb), bs)


SHAPES = [  # layers, rows, M, nb, bs, n_kv, hd, dtype
    (1, 4, 3, 7, 16, 2, 128, torch.bfloat16),
    (3, 9, 5, 40, 8, 1, 64, torch.float16),
    (2, 17, 7, 95, 32, 4, 64, torch.float32),
    (2, 6, 130, 300, 1, 1, 3, torch.bfloat16),     # 6-byte tokens: 2-byte accesses; more columns than a CTA has
    (2, 5, 4, 33, 3, 1, 6, torch.float16),         # 12-byte tokens
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("seed", range(3))
def test_random_runs(shape, seed):
    layers, R, M, nb, bs, n_kv, hd, dtype = shape
    r = np.random.default_rng(seed)
    b = Both(empty(R, M, nb, bs), make_caches(layers, nb, bs, n_kv, hd, dtype, seed))
    for step in range(12):
        k = step % 4 if step < 4 else int(r.integers(0, 3))
        if k in (0, 3):
            n = int(r.integers(1, R + 1))
            b.resize(r.permutation(R)[:n], r.integers(0, M * bs + 1, n))
        elif k == 1:
            n = int(r.integers(1, R + 1))
            b.fork(r.integers(0, R, n), r.permutation(R)[:n])
        else:
            b.compact()
        assert b.st.consistent()
    assert bool((b.ref >= 0).all())


def test_generation_of_samples():
    """A prompt, 20 samples of it, steps that copy the shared last page once each, truncation of
    drafted tokens, the end of the samples."""
    R, M, nb, bs = 24, 8, 120, 16
    b = Both(empty(R, M, nb, bs), make_caches(2, nb, bs, 2, 64, torch.bfloat16, 5))
    b.resize([3], [41])
    rows = [r for r in range(R) if r != 3][:20]
    b.fork([3] * 20, rows)
    assert int(b.st.ref.max()) == 21
    b.resize(rows, [42] * 20)
    b.resize(rows, [50] * 20)          # past the page's end
    b.resize(rows, [44] * 20)          # drafts rejected
    b.fork(rows[:10], rows[10:])       # half of the beams are replaced
    b.resize(rows, [45] * 20)
    b.compact()
    b.resize(rows + [3], [0] * 21)
    assert not b.st.ref.any()


def test_bad_entries_are_counted_and_skipped():
    R, M, nb, bs = 6, 4, 12, 4
    st = m.State([[0, 1, 2, -1], [0, nb, -7, 3], [4, 5, -1, -1], [0, 0, 0, 0], [6, -1, -1, -1], [-1] * 4],
                 [10, 16, 7, 99, 3, 0], [1, 1, 1, 1, 1, 0, 1, -3, 0, 0, 0, 0], bs)
    b = Both(st, make_caches(1, nb, bs, 1, 8, torch.float32, 1))
    b.fork([0, BIG, 1, -1, 0, 3, 1], [5, 0, 2, 1, 5, 4, R])   # bad parent, bad child, the same child twice, a bad length
    b.resize([5, 1, BIG, 5, 0, 3, -2], [17, 0, 1, 3, 16, 4, 4])
    b.resize([2, 4], [2, 4])
    b.compact()


def test_growth_beside_a_bad_last_page_is_refused():
    st = m.State([[5, -1], [1, -1], [9, -1]], [3, 2, 1], [0, 1, 0, 0], 4)
    b = Both(st, make_caches(1, 4, 4, 1, 8, torch.float16, 1))
    b.resize([0, 1, 2], [4, 8, 0])


def test_a_full_cache_serves_what_fits():
    R, M, nb, bs = 5, 4, 6, 4
    b = Both(empty(R, M, nb, bs), make_caches(1, nb, bs, 1, 8, torch.bfloat16, 2))
    b.resize([0, 1, 2, 3], [8, 9, 1, 1])     # 2 + 3 + 1 of 6 pages; the last one is refused
    assert b.errors == 1
    b.resize([3, 0, 2], [4, 0, 4])           # the pages given back in the call are used in it
    b.resize([4, 1], [16, 10])               # entry 0 asks for more than there is; entry 1 needs none
    assert b.errors == 2 and b.st.seq[1] == 10


def test_empty_calls():
    b = Both(empty(3, 2, 4, 8), make_caches(1, 4, 8, 1, 8, torch.float32, 3))
    b.fork([], [])
    b.resize([], [])
    b.resize([1], [0])
    b.compact()
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    sra.copy_kv_pages(b.dev_caches, none, none)
    z = torch.empty(2, 0, 8, 1, 8, device=DEV)      # a cache without pages
    t, s = torch.empty(0, 2, dtype=torch.int32, device=DEV), none
    assert sra.compact_kv_pages(t, s, none, z).cpu().tolist() == [0]
    t, s = torch.full((2, 2), -1, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pos, slot = sra.resize_kv_rows(t, s, none, i32([0]), i32([3]), z, err_count=err)
    assert err.item() == 1 and pos.item() == -1 and s.tolist() == [0, 0]


@pytest.mark.parametrize("layers,nb,bs,n_kv,hd,dtype,off", [
    (1, 9, 16, 2, 128, torch.bfloat16, 0), (5, 30, 8, 1, 64, torch.float32, 0), (2, 12, 3, 1, 5, torch.float16, 0),
    (2, 20, 16, 1, 64, torch.float16, 1), (130, 6, 4, 1, 8, torch.bfloat16, 0)])
def test_copy(layers, nb, bs, n_kv, hd, dtype, off):
    """Repeated sources, padding, bad indexes; caches at an odd element; more layers than one launch takes."""
    caches = make_caches(layers, nb, bs, n_kv, hd, dtype, 7)
    dev = []
    for c in caches:
        flat = torch.empty(c.numel() + off, dtype=dtype, device=DEV)[off:]
        dev.append(flat.copy_(c.reshape(-1).to(DEV)).view(c.shape))
    src, dst = [0, 0, nb, -1, 1, 2, BIG, 3], [nb - 1, nb - 2, 1, 2, -1, nb, BIG - 1, nb - 3]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    sra.copy_kv_pages(dev, i32(src), i32(dst), err_count=err)
    assert int(err.item()) == m.copy(caches, src, dst) == 3
    for g, c in zip(dev, caches):
        assert torch.equal(m.bits(g.cpu()), m.bits(c))


def test_copy_one_tensor_of_layers():
    caches = make_caches(4, 10, 16, 2, 64, torch.bfloat16, 8)
    dev = torch.stack(caches).to(DEV)
    sra.copy_kv_pages(dev, i32([1, 2]), i32([8, 9]))
    m.copy(caches, [1, 2], [8, 9])
    assert torch.equal(m.bits(dev.cpu()), m.bits(torch.stack(caches)))


def test_many_entries_and_many_pages():
    """More entries than the planning CTA has threads and more pages than one of its steps, an odd
    count of them at an address that is not 16-byte aligned."""
    R, M, nb, bs = 1500, 20, 40003, 2
    r = np.random.default_rng(9)
    st = empty(R, M, nb, bs)
    st.ref[r.permutation(nb)[:20000]] = 1     # pages that some other table holds
    b = Both(st, make_caches(1, nb, bs, 1, 2, torch.float16, 9))
    b.ref = torch.cat([i32([0]), b.ref])[1:]
    b.resize(np.arange(R), r.integers(0, M * bs + 1, R))
    b.resize(r.permutation(R), r.integers(0, M * bs + 1, R))
    b.fork(r.integers(0, R, R), r.permutation(R))
    b.compact()
    b.resize(r.permutation(R), r.integers(0, M * bs + 1, R))


def test_graph_replay_and_another_stream():
    """A captured fork, step and free replayed: the same pages each time; and the same on another stream
    with workspaces of the call's own."""
    R, M, nb, bs = 10, 6, 50, 8
    b = Both(empty(R, M, nb, bs), make_caches(2, nb, bs, 1, 64, torch.bfloat16, 4))
    b.resize([0], [21])
    rows, parents = np.arange(1, R), np.zeros(R - 1, dtype=int)
    d = dict(p=i32(parents), c=i32(rows), up=i32([22] * (R - 1)), no=i32([0] * (R - 1)))
    fw, rw = sra.kv_fork_workspace(R - 1, M, DEV), sra.kv_resize_workspace(R - 1, nb, DEV)

    def generation():
        sra.fork_kv_rows(b.table, b.seq, b.ref, d["p"], d["c"], bs, workspace=fw, err_count=b.err)
        pos, slot = sra.resize_kv_rows(b.table, b.seq, b.ref, d["c"], d["up"], b.dev_caches, workspace=rw,
                                       err_count=b.err)
        sra.resize_kv_rows(b.table, b.seq, b.ref, d["c"], d["no"], b.dev_caches, workspace=rw, err_count=b.err)
        return pos, slot

    def model():
        assert m.fork(b.st, parents, rows) == 0
        _, pos, slot = m.resize(b.st, rows, [22] * (R - 1), b.caches)
        m.resize(b.st, rows, [0] * (R - 1), b.caches)
        return pos.tolist(), slot.tolist()

    want = model()
    generation()
    b.check("eager")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pos, slot = generation()
    for _ in range(3):
        g.replay()
        assert model() == want
        b.check("replay")
        assert (pos.cpu().tolist(), slot.cpu().tolist()) == want
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (s, s.cuda_stream):
        with torch.cuda.stream(s):
            sra.fork_kv_rows(b.table, b.seq, b.ref, d["p"], d["c"], bs, err_count=b.err, stream=stream)
            sra.resize_kv_rows(b.table, b.seq, b.ref, d["c"], d["up"], b.dev_caches, err_count=b.err, stream=stream)
            sra.resize_kv_rows(b.table, b.seq, b.ref, d["c"], d["no"], b.dev_caches, err_count=b.err, stream=stream)
        model()
        b.check("another stream")


def test_refusals():
    c = make_caches(1, 4, 4, 1, 8, torch.float32, 1)[0].to(DEV)
    t, s, ref = i32([[0, 1], [2, 3]]), i32([1, 1]), i32([1, 1, 1, 1])
    with pytest.raises(ValueError):
        sra.fork_kv_rows(t.long(), s, ref, i32([0]), i32([1]), 4)
    with pytest.raises(ValueError):
        sra.fork_kv_rows(t[:, :1], s, ref, i32([0]), i32([1]), 4)
    with pytest.raises(ValueError):
        sra.fork_kv_rows(t, s, ref, i32([0]), i32([1, 0]), 4)
    with pytest.raises(ValueError):
        sra.resize_kv_rows(t, s, ref[:3], i32([0]), i32([1]), c)
    with pytest.raises(ValueError):
        sra.copy_kv_pages(c[:, ::2], i32([0]), i32([1]))
    with pytest.raises(ValueError):
        sra.copy_kv_pages([c, c.half()], i32([0]), i32([1]))
    with pytest.raises(ValueError):
        sra.copy_kv_pages([], i32([0]), i32([1]))
    with pytest.raises(sra.SRAError) as e:
        sra.copy_kv_pages([c, c], i32([0]), i32([1]))
    assert e.value.status == -5
    with pytest.raises(sra.SRAError) as e:
        sra.fork_kv_rows(t, s, ref, s, i32([1, 0]), 4)       # an output as an input
    assert e.value.status == -5
    with pytest.raises(sra.SRAError) as e:
        sra.fork_kv_rows(t, s, ref, i32([0]), i32([1]), 4, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))
    assert e.value.status == -6
    assert t.tolist() == [[0, 1], [2, 3]]


def test_cache_past_32_bit_offsets():
    """A cache whose planes have more than 2^31 elements: pages copied, copied on write and moved at its far end."""
    bs, n_kv, hd = 16, 8, 128
    nb = 2 ** 31 // (bs * n_kv * hd) + 64
    cache = torch.empty(2, nb, bs, n_kv, hd, dtype=torch.bfloat16, device=DEV)
    cache[:, -64:] = torch.randn(2, 64, bs, n_kv, hd, device=DEV).to(torch.bfloat16)
    end = cache[:, -64:].clone()
    sra.copy_kv_pages(cache, i32([nb - 64, nb - 1]), i32([nb - 2, 5]))
    assert torch.equal(cache[:, nb - 2], end[:, 0]) and torch.equal(cache[:, 5], end[:, 63])
    # rows 0 and 1 hold a last page of 3 tokens together; every page but two at the end is taken
    table, seq = i32([[nb - 60, nb - 50], [nb - 60, nb - 50]]), i32([19, 19])
    ref = torch.ones(nb, dtype=torch.int32, device=DEV)
    ref[[nb - 60, nb - 50]] = 2
    ref[[nb - 40, nb - 30]] = 0
    pos, slot = sra.resize_kv_rows(table, seq, ref, i32([0, 1]), i32([20, 20]), cache)
    assert table.cpu().tolist() == [[nb - 60, nb - 40], [nb - 60, nb - 30]]
    assert slot.cpu().tolist() == [(nb - 40) * bs + 3, (nb - 30) * bs + 3] and pos.cpu().tolist() == [19, 19]
    for page in (nb - 40, nb - 30):
        assert torch.equal(cache[:, page, :3], end[:, 14, :3])
    # all but these rows' pages free: they move to the front
    ref.zero_()
    ref[[nb - 60, nb - 40, nb - 30]] = i32([2, 1, 1])
    kept = cache[:, [nb - 60, nb - 40, nb - 30]].clone()
    assert int(sra.compact_kv_pages(table, seq, ref, cache).item()) == 3
    assert table.cpu().tolist() == [[0, 1], [0, 2]] and torch.equal(cache[:, :3], kept)
    assert ref[:3].cpu().tolist() == [2, 1, 1] and int(ref.sum()) == 4
