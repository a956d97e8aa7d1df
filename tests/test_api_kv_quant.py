"""Host-side checks of the quantised cache's C entry points (no GPU): every bad argument gives its status before any
CUDA call. Addresses are fakes, passed only with an argument that is invalid."""
import pytest

import swiglu_rmsnorm_add_gb300 as sra
from swiglu_rmsnorm_add_gb300 import build as sra_build

OK, NULL, SHAPE, STRIDE, DTYPE, ALIAS, ARG = 0, -1, -2, -3, -4, -5, -6
BF16, BYTES = 2, 8
P = 0x10000000
Q, K, V, COS, SIN, POS, SLOT, QA, QG, KA, KG, OUT, TABLE, SEQ, WS = (P + k * 0x1000000 for k in range(15))
CACHE = P + 0x40000000


@pytest.fixture(scope="module")
def L():
    sra_build.build()
    return sra.lib()


def store(L, q=Q, k=K, v=V, cos=COS, sin=SIN, pos=POS, slot=SLOT, cache=CACHE, T=4, H=4, KV=2, D=64, qs=256, ks=128, vs=128,
          mp=32, nb=8, bs=16, err=None, style=0, pars=(None,) * 4, clip=(-1.0, 1.0), fmt=0, dt=BF16):
    return L.sra_rope_kv_store_quant(q, k, v, cos, sin, pos, slot, cache, T, H, KV, D, qs, ks, vs, mp, nb, bs, err, style, *pars,
                                     *clip, fmt, dt, None)


def read(L, cache=CACHE, table=TABLE, cu=SEQ, starts=None, k=K, v=V, rows=2, mb=4, total=9, KV=2, D=64, ks=128, vs=128, nb=8,
         bs=16, err=None, fmt=0, dt=BF16):
    return L.sra_kv_quant_read(cache, table, cu, starts, k, v, rows, mb, total, KV, D, ks, vs, nb, bs, err, fmt, dt, None)


def attn(L, q=Q, cache=CACHE, table=TABLE, seq=SEQ, out=OUT, B=3, H=4, KV=2, D=64, qs=256, os=256, nb=8, bs=16, mb=4, scale=0.1,
         ws=None, wb=0, err=None, fmt=0, dt=BF16):
    return L.sra_paged_decode_attention_quant(q, cache, table, seq, out, B, H, KV, D, qs, os, nb, bs, mb, scale, ws, wb, err, fmt,
                                              dt, None)


def test_row_bytes(L):
    f = L.sra_kv_quant_row_bytes
    assert [f(d, 0) for d in (64, 128, 256)] == [36, 72, 144] and [f(d, 1) for d in (64, 128, 256)] == [68, 136, 272]
    assert f(96, 0) == SHAPE and f(64, 2) == ARG and f(64, -1) == ARG


def test_store(L):
    assert store(L, dt=9) == DTYPE and store(L, dt=BYTES) == DTYPE
    assert store(L, fmt=2) == ARG and store(L, style=2) == ARG and store(L, cache=CACHE + 8) == ARG
    for bad in (dict(T=-1), dict(H=0), dict(KV=0), dict(H=3), dict(D=96), dict(D=32), dict(bs=0), dict(nb=-1), dict(mp=-1),
                dict(nb=1 << 60)):
        assert store(L, **bad) == SHAPE, bad
    for bad in (dict(qs=255), dict(ks=127), dict(vs=0)):
        assert store(L, **bad) == STRIDE, bad
    assert store(L, T=0, q=None, k=None) == OK
    for bad in ("q", "k", "v", "cos", "sin", "pos", "slot", "cache"):
        assert store(L, **{bad: None}) == NULL, bad
    assert store(L, pars=(QA, None, KA, KG)) == NULL
    assert store(L, pars=(QA, QG, KA, KG), clip=(1.0, -1.0)) == ARG
    assert store(L, pars=(QA, QG, KA, KG), clip=(float("nan"), 1.0)) == ARG
    for bad in (dict(k=Q), dict(v=Q + 64), dict(cache=Q), dict(cache=K), dict(pos=Q), dict(slot=CACHE), dict(cos=CACHE),
                dict(sin=Q), dict(pars=(QA, QG, Q, KG)), dict(pars=(CACHE, QG, KA, KG))):
        assert store(L, **bad) == ALIAS, bad


def test_read(L):
    assert read(L, dt=9) == DTYPE and read(L, fmt=3) == ARG and read(L, cache=CACHE + 4) == ARG
    for bad in (dict(rows=-1), dict(mb=-1), dict(total=-1), dict(total=1 << 31), dict(KV=0), dict(D=80), dict(bs=0), dict(nb=-2),
                dict(rows=1 << 31), dict(nb=1 << 60)):
        assert read(L, **bad) == SHAPE, bad
    assert read(L, ks=127) == STRIDE and read(L, vs=64) == STRIDE
    assert read(L, total=0, k=None, v=None) == OK
    for bad in ("cache", "table", "cu", "k", "v"):
        assert read(L, **{bad: None}) == NULL, bad
    for bad in (dict(k=V), dict(k=CACHE), dict(v=TABLE), dict(k=SEQ), dict(starts=K)):
        assert read(L, **bad) == ALIAS, bad


def test_attention(L):
    assert attn(L, dt=9) == DTYPE and attn(L, fmt=2) == ARG and attn(L, cache=CACHE + 8) == ARG
    assert attn(L, scale=float("inf")) == ARG and attn(L, scale=float("nan")) == ARG and attn(L, wb=-1) == ARG
    for bad in (dict(B=-1), dict(H=0), dict(H=18), dict(H=3), dict(KV=0), dict(D=80), dict(bs=4), dict(bs=64), dict(nb=-1),
                dict(mb=-1), dict(B=1 << 31), dict(mb=1 << 28), dict(nb=1 << 31)):
        assert attn(L, **bad) == SHAPE, bad
    assert attn(L, qs=255) == STRIDE and attn(L, os=0) == STRIDE
    assert attn(L, B=0, q=None) == OK
    for bad in ("q", "cache", "table", "seq", "out"):
        assert attn(L, **{bad: None}) == NULL, bad
    for bad in (dict(out=Q), dict(out=CACHE), dict(out=TABLE), dict(out=SEQ)):
        assert attn(L, **bad) == ALIAS, bad


def test_workspace_size(L):
    f = L.sra_paged_decode_attention_quant_workspace_size
    assert f(1, 4, 2, 64, 4, 16, 0, 9) == DTYPE and f(1, 4, 2, 64, 4, 16, 5, BF16) == ARG
    for bad in ((-1, 4, 2, 64, 4, 16), (1, 4, 3, 64, 4, 16), (1, 4, 2, 65, 4, 16), (1, 4, 2, 64, -4, 16), (1, 4, 2, 64, 4, 5)):
        assert f(*bad, 0, BF16) == SHAPE, bad


def test_page_calls_on_bytes(L):
    import ctypes

    caches = (ctypes.c_void_p * 1)(CACHE + 2)
    assert L.sra_kv_copy_pages(caches, 1, Q, K, 4, 8, 16, 2, 36, None, BYTES, None) == ARG
    caches = (ctypes.c_void_p * 1)(CACHE)
    assert L.sra_kv_copy_pages(caches, 1, Q, K, 4, 8, 16, 2, 34, None, BYTES, None) == SHAPE
    assert L.sra_kv_copy_pages(caches, 1, Q, K, 0, 8, 16, 2, 36, None, BYTES, None) == OK
    # a cache of bytes has those bytes: 2 * 8 * 16 * 2 * 36
    assert L.sra_kv_copy_pages(caches, 1, CACHE + 18428, K, 4, 8, 16, 2, 36, None, BYTES, None) == ALIAS


def test_binding_refuses():
    import torch

    with pytest.raises(ValueError):
        sra.quant_kv_cache(4, 16, 2, 128, "fp3", device="cpu")
    with pytest.raises(sra.SRAError):
        sra.quant_kv_cache(4, 16, 2, 100, device="cpu")
    c = sra.quant_kv_cache(4, 16, 2, 128, layers=3, device="cpu")
    assert c.shape == (3, 2, 4, 2, 16, 72) and c.dtype is torch.uint8
    with pytest.raises(ValueError):      # not on a GPU
        sra.paged_decode_attention_quant(torch.zeros(1, 4, 128), c[0], torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1))
    with pytest.raises(ValueError):
        sra.decode_attention_quant_workspace(1, 4, 2, 128, 4, 16, "int3")
