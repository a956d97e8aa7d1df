"""GPU: the quantised cache as a server uses it: prompts stored, a prompt shared by samples, decode steps with copy on
write, rows ended, the cache compacted, a history read back, all against the host model of the bytes."""
import numpy as np
import pytest
import torch

import swiglu_rmsnorm_add_gb300 as sra
from tests import quant_model as qm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).to(DEV)


class Server:
    """Three layers' caches, the page state, and a model of every row's tokens (bytes of K and V)."""

    def __init__(self, fmt, dtype, hd=128, n_head=6, n_kv=2, bs=16, nb=48, rows=6, mb=12, layers=3):
        self.fmt, self.dtype, self.hd, self.n_head, self.n_kv, self.bs = fmt, dtype, hd, n_head, n_kv, bs
        self.caches = sra.quant_kv_cache(nb, bs, n_kv, hd, fmt, layers=layers, device=DEV).fill_(255)
        self.table, self.seq, self.ref = i32(np.full((rows, mb), -1)), i32([0] * rows), i32([0] * nb)
        a = torch.outer(torch.arange(mb * bs, dtype=torch.float64), 1e4 ** (-torch.arange(hd // 2, dtype=torch.float64) / (hd // 2)))
        self.cos, self.sin = a.cos().float().to(DEV), a.sin().float().to(DEV)
        self.held = [[np.zeros((2, 0, n_kv, qm.row_bytes(fmt, hd)), dtype=np.uint8) for _ in range(layers)] for _ in range(rows)]
        self.seed = 0

    def qkv(self, T):
        self.seed += 1
        g = torch.Generator().manual_seed(self.seed)
        return [torch.randn(T, n, self.hd, generator=g).to(self.dtype).to(DEV) for n in (self.n_head, self.n_kv, self.n_kv)]

    def store(self, rows, pos, slot):
        """A token for each (row, pos) at its slot, in every layer; the rows' models grow by them."""
        for layer, cache in enumerate(self.caches):
            q, k, v = self.qkv(len(rows))
            kk = qm.held_k(k.double().cpu().numpy(), self.cos.double().cpu().numpy()[pos.cpu()],
                           self.sin.double().cpu().numpy()[pos.cpu()], "neox", self.dtype)
            new = np.stack([qm.encode(kk, self.fmt), qm.encode(v.double().cpu().numpy(), self.fmt)])
            sra.rope_kv_store_quant(q, k, v, self.cos, self.sin, pos, slot, cache)
            for i, r in enumerate(rows):
                self.held[r][layer] = np.concatenate([self.held[r][layer], new[:, i:i + 1]], 1)

    def admit(self, row, n):
        sra.resize_kv_rows(self.table, self.seq, self.ref, i32([row]), i32([n]), self.caches)
        t = torch.arange(n, device=DEV)
        self.store([row] * n, t, self.table[row].long()[t // self.bs] * self.bs + t % self.bs)

    def step(self, rows):
        lens = [self.held[r][0].shape[1] + 1 for r in rows]
        pos, slot = sra.resize_kv_rows(self.table, self.seq, self.ref, i32(rows), i32(lens), self.caches)
        assert pos.tolist() == [n - 1 for n in lens]
        self.store(rows, pos, slot)

    def end(self, row):
        sra.resize_kv_rows(self.table, self.seq, self.ref, i32([row]), i32([0]), self.caches)
        self.held[row] = [h[:, :0] for h in self.held[row]]

    def fork(self, parent, children):
        sra.fork_kv_rows(self.table, self.seq, self.ref, i32([parent] * len(children)), i32(children), self.bs)
        for c in children:
            self.held[c] = list(self.held[parent])

    def check(self):
        lens = [h[0].shape[1] for h in self.held]
        assert self.seq.tolist() == lens
        cu = np.concatenate([[0], np.cumsum(lens)])
        for layer, cache in enumerate(self.caches):
            want = np.concatenate([qm.decode(h[layer], self.fmt, self.hd) for h in self.held], 1)
            k, v = sra.read_kv_quant(cache, self.table, i32(cu), int(cu[-1]), self.hd, torch.float32)
            assert np.array_equal(k.double().cpu().numpy(), want[0]) and np.array_equal(v.double().cpu().numpy(), want[1])
            q = self.qkv(len(lens))[0]
            for w in (None, sra.decode_attention_quant_workspace(len(lens), self.n_head, self.n_kv, self.hd, self.table.shape[1],
                                                                 self.bs, self.fmt, self.dtype, DEV)):
                got = sra.paged_decode_attention_quant(q, cache, self.table, self.seq, workspace=w).double().cpu().numpy()
                G = self.n_head // self.n_kv
                for b, n in enumerate(lens):
                    kv = want[:, cu[b]:cu[b + 1]]
                    for h in range(self.n_head if n else 0):
                        s = kv[0, :, h // G] @ q[b, h].double().cpu().numpy() * self.hd ** -0.5
                        p = np.exp(s - s.max())
                        p /= p.sum()
                        o, A = p @ kv[1, :, h // G], p @ np.abs(kv[1, :, h // G])
                        u = torch.finfo(self.dtype).eps / 2
                        assert (np.abs(got[b, h] - o) <= u * np.abs(o) + (2.0 ** -11 + 6e-5) * A).all()
                    if n == 0:
                        assert (got[b] == 0).all()


@pytest.mark.parametrize("fmt,dtype,hd", [("e2m1", torch.bfloat16, 128), ("int8", torch.float16, 64), ("e2m1", torch.float32, 256)])
def test_serving(fmt, dtype, hd):
    s = Server(fmt, dtype, hd)
    s.admit(0, 37)
    s.admit(4, 5)
    s.check()
    s.fork(0, [1, 2, 3])
    s.step([1, 2, 3])           # all copy the shared, partly filled page
    s.check()
    s.step([0, 1, 3, 4])
    s.end(2)
    s.check()
    live = int(sra.compact_kv_pages(s.table, s.seq, s.ref, s.caches).item())
    assert live == int((s.ref > 0).sum())
    s.check()
    s.admit(5, 64)
    s.step([5, 0])
    s.check()
    # a page copied by hand holds the same bytes
    free = int(torch.nonzero(s.ref == 0)[0])
    page = int(s.table[5, 0])
    sra.copy_kv_pages(s.caches, i32([page]), i32([free]))
    assert torch.equal(s.caches[:, :, free], s.caches[:, :, page])


def test_a_captured_decode_step():
    """resize, store and attention of a step in one graph, replayed step after step."""
    fmt, dtype = "e2m1", torch.bfloat16
    a, b = Server(fmt, dtype), Server(fmt, dtype)
    for s in (a, b):
        s.admit(0, 20)
        s.admit(1, 47)
    rows = i32([0, 1])
    cache = a.caches[0]
    q, k, v = (torch.empty_like(t) for t in a.qkv(2))
    lens = a.seq[:2].clone()
    ws_r = sra.kv_resize_workspace(2, cache.shape[1], DEV)
    ws_a = sra.decode_attention_quant_workspace(2, 6, 2, 128, 12, 16, fmt, dtype, DEV)
    pos, slot = torch.empty(2, dtype=torch.int64, device=DEV), torch.empty(2, dtype=torch.int64, device=DEV)
    out = torch.empty_like(q)

    def step(s, cache, q, k, v, lens, out):
        lens += 1
        sra.resize_kv_rows(s.table, s.seq, s.ref, rows, lens, s.caches, pos=pos, slot_mapping=slot, workspace=ws_r)
        sra.rope_kv_store_quant(q, k, v, s.cos, s.sin, pos, slot, cache)
        sra.paged_decode_attention_quant(q, cache, s.table[:2], s.seq[:2], out=out, workspace=ws_a)

    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(a, cache, q, k, v, lens, out)
    eager = b.seq[:2].clone()
    for _ in range(20):
        new = b.qkv(2)
        for t, n in zip((q, k, v), new):
            t.copy_(n)
        g.replay()
        want = torch.empty_like(out)
        step(b, b.caches[0], *(t.clone() for t in new), eager, want)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert torch.equal(a.caches[0][:, a.table[:2, :4].flatten().long()], b.caches[0][:, b.table[:2, :4].flatten().long()])
