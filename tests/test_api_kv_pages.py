"""Host-side checks of the page operators' C entry points (no GPU): every bad argument gives its
status before any CUDA call. Addresses are fakes, passed only with an argument that is invalid."""
import ctypes

import pytest

import swiglu_rmsnorm_add_gb300 as sra
from swiglu_rmsnorm_add_gb300 import build as sra_build

OK, NULL, SHAPE, DTYPE, ALIAS, ARG = 0, -1, -2, -4, -5, -6
BF16, F32 = 2, 0
P = 0x100000
T, S, R, A, B, W, E, POS, SLOT = (P + k * 0x10000 for k in range(9))
CACHE = P + 0x1000000


@pytest.fixture(scope="module")
def L():
    sra_build.build()
    return sra.lib()


def caches(*ptrs):
    return (ctypes.c_void_p * len(ptrs))(*ptrs)


def copy(L, c=None, k=1, src=A, dst=B, n=4, nb=8, bs=16, kv=2, hd=64, err=None, dt=BF16):
    return L.sra_kv_copy_pages(c if c is not None else caches(CACHE), k, src, dst, n, nb, bs, kv, hd, err, dt, None)


def fork(L, t=T, s=S, r=R, p=A, c=B, n=4, rows=8, M=4, nb=16, bs=16, ws=W, wb=1 << 12, err=None):
    return L.sra_kv_fork_rows(t, s, r, p, c, n, rows, M, nb, bs, ws, wb, err, None)


def resize(L, t=T, s=S, r=R, idx=A, lens=B, n=4, rows=8, M=4, c=None, k=1, nb=16, bs=16, kv=2, hd=64, pos=POS,
           slot=SLOT, ws=W, wb=1 << 12, err=None, dt=BF16):
    return L.sra_kv_resize_rows(t, s, r, idx, lens, n, rows, M, c if c is not None else caches(CACHE), k, nb, bs, kv,
                                hd, pos, slot, ws, wb, err, dt, None)


def compact(L, t=T, s=S, r=R, rows=8, M=4, c=None, k=1, nb=16, bs=16, kv=2, hd=64, live=None, ws=W, wb=1 << 12,
            err=None, dt=BF16):
    return L.sra_kv_compact_pages(t, s, r, rows, M, c if c is not None else caches(CACHE), k, nb, bs, kv, hd, live, ws,
                                  wb, err, dt, None)


def test_copy(L):
    assert copy(L, dt=9) == DTYPE
    for bad in (dict(n=-1), dict(k=-1), dict(nb=-1), dict(nb=1 << 31), dict(bs=0), dict(kv=0), dict(hd=-2),
                dict(bs=2 ** 31 - 1, kv=2 ** 31 - 1, hd=64)):
        assert copy(L, **bad) == SHAPE, bad
    assert copy(L, n=0, src=None, dst=None) == OK and copy(L, k=0) == OK
    assert copy(L, src=None) == NULL and copy(L, dst=None) == NULL and copy(L, c=caches(None)) == NULL
    assert copy(L, c=caches(CACHE + 1)) == ARG
    assert copy(L, c=caches(CACHE, CACHE + 64), k=2) == ALIAS
    assert copy(L, src=CACHE + 128) == ALIAS and copy(L, err=A) == ALIAS and copy(L, err=CACHE) == ALIAS


def test_caches_in_any_order(L):
    # a cache is 65536 bytes
    step = 1 << 16
    for bad in ((CACHE + step - 8, CACHE), (CACHE + step, CACHE, CACHE + step - 16), (CACHE, CACHE + 2 * step, CACHE),
                (CACHE + 3 * step, CACHE + step, CACHE + 2 * step - 2)):
        assert copy(L, c=caches(*bad), k=len(bad)) == ALIAS, bad
    apart = caches(CACHE + 6 * step, CACHE, CACHE + 3 * step)
    for src in (CACHE + 6 * step + 64, CACHE + 7 * step - 4, CACHE - 8, CACHE + 3 * step - 12, CACHE + 4 * step - 4):
        assert copy(L, c=apart, k=3, src=src) == ALIAS, hex(src)


def test_fork(L):
    for bad in (dict(n=-1), dict(rows=-1), dict(M=-1), dict(nb=-1), dict(bs=0), dict(n=524281), dict(rows=1 << 31)):
        assert fork(L, **bad) == SHAPE, bad
    assert fork(L, n=0, t=None, ws=None) == OK
    for bad in (dict(t=None), dict(s=None), dict(r=None), dict(p=None), dict(c=None), dict(ws=None)):
        assert fork(L, **bad) == NULL, bad
    assert fork(L, wb=-1) == ARG and fork(L, wb=64) == ARG and fork(L, ws=W + 4) == ARG
    for bad in (dict(s=T + 4), dict(r=T), dict(p=S), dict(c=T), dict(p=W), dict(err=R), dict(ws=T)):
        assert fork(L, **bad) == ALIAS, bad
    assert fork(L, p=A, c=A, ws=None) == NULL   # parents and children may be one array: both are read


def test_resize(L):
    assert resize(L, dt=3) == DTYPE
    for bad in (dict(n=-1), dict(rows=-1), dict(M=-1), dict(nb=-1), dict(bs=0), dict(k=0), dict(n=524281)):
        assert resize(L, **bad) == SHAPE, bad
    assert resize(L, n=0, t=None, ws=None) == OK
    for bad in (dict(t=None), dict(s=None), dict(r=None), dict(idx=None), dict(lens=None), dict(ws=None),
                dict(c=caches(None))):
        assert resize(L, **bad) == NULL, bad
    assert resize(L, wb=-1) == ARG and resize(L, wb=8) == ARG and resize(L, ws=W + 8) == ARG
    for bad in (dict(s=T + 4), dict(idx=S), dict(lens=S), dict(pos=SLOT), dict(pos=A), dict(ws=CACHE), dict(t=CACHE),
                dict(idx=CACHE), dict(c=caches(CACHE, CACHE), k=2)):
        assert resize(L, **bad) == ALIAS, bad


def test_compact(L):
    assert compact(L, dt=-1) == DTYPE
    for bad in (dict(rows=-1), dict(M=-1), dict(nb=-1), dict(bs=0), dict(k=0), dict(hd=0)):
        assert compact(L, **bad) == SHAPE, bad
    for bad in (dict(t=None), dict(s=None), dict(r=None), dict(ws=None), dict(c=caches(None))):
        assert compact(L, **bad) == NULL, bad
    assert compact(L, wb=16) == ARG
    for bad in (dict(s=T), dict(live=R), dict(live=T + 8), dict(ws=R), dict(s=CACHE), dict(err=W)):
        assert compact(L, **bad) == ALIAS, bad


def test_workspace_sizes(L):
    assert L.sra_kv_fork_workspace_size(4, 100) >= 4 * 108 * 4 // 4 and L.sra_kv_fork_workspace_size(0, 0) == 0
    assert L.sra_kv_fork_workspace_size(-1, 4) == SHAPE and L.sra_kv_fork_workspace_size(4, -1) == SHAPE
    assert L.sra_kv_resize_workspace_size(10, 1000) >= 8 + 200 + 4000
    assert L.sra_kv_resize_workspace_size(10, -1) == SHAPE
    assert L.sra_kv_compact_workspace_size(1000) >= 12008 and L.sra_kv_compact_workspace_size(1 << 31) == SHAPE


def attend(L, q=P, c=CACHE, pt=T, pl=S, bt=R, sl=A, out=B, batch=4, nh=8, kv=2, hd=64, qs=512, os_=512, nb=8, bs=16,
           pb=4, mb=4, scale=1.0, ws=None, wb=0, err=None, dt=BF16):
    return L.sra_shared_prefix_attention(q, c, pt, pl, bt, sl, out, batch, nh, kv, hd, qs, os_, nb, bs, pb, mb, scale,
                                         ws, wb, err, dt, None)


def test_shared_prefix(L):
    assert attend(L, dt=5) == DTYPE
    for bad in (dict(batch=-1), dict(nh=9), dict(nh=18), dict(hd=96), dict(bs=24), dict(nb=-1), dict(pb=-1),
                dict(mb=-1), dict(kv=0), dict(nb=1 << 31)):
        assert attend(L, **bad) == SHAPE, bad
    assert attend(L, qs=511) == -3 and attend(L, os_=100) == -3
    assert attend(L, scale=float("nan")) == ARG and attend(L, wb=-1) == ARG and attend(L, c=CACHE + 8) == ARG
    assert attend(L, batch=0, q=None) == OK
    for bad in (dict(q=None), dict(c=None), dict(pt=None), dict(pl=None), dict(bt=None), dict(sl=None), dict(out=None)):
        assert attend(L, **bad) == NULL, bad
    for bad in (dict(out=P), dict(out=CACHE + 64), dict(out=T), dict(out=S - 16), dict(out=R), dict(out=A),
                dict(err=B), dict(err=A), dict(err=P)):
        assert attend(L, **bad) == ALIAS, bad


def test_shared_prefix_workspace_size(L):
    f = L.sra_shared_prefix_workspace_size
    assert f(4, 8, 2, 64, 4, 4, 16, 7) == DTYPE
    for bad in ((-1, 8, 2, 64, 4, 4, 16), (4, 9, 2, 64, 4, 4, 16), (4, 8, 2, 60, 4, 4, 16), (4, 8, 2, 64, -1, 4, 16),
                (4, 8, 2, 64, 4, 4, 17)):
        assert f(*bad, BF16) == SHAPE
