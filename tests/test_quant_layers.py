"""A cache in 4 or 8 bits of several layers, of any number of pages and tokens a page: each layer is a cache that every call takes."""
import numpy as np
import pytest
import torch

import swiglu_rmsnorm_add_gb300 as sra
from tests import quant_model as qm

DEV = "cuda:0"
SIZES = [(5, 1, 1, 64, "e2m1"), (5, 1, 1, 64, "int8"), (3, 7, 3, 64, "e2m1"), (1, 1, 1, 64, "int8"), (5, 3, 1, 128, "e2m1"), (4, 16, 2, 64, "e2m1")]


@pytest.mark.parametrize("nb,bs,n_kv,hd,fmt", SIZES)
def test_layers_are_aligned(nb, bs, n_kv, hd, fmt):
    c = sra.quant_kv_cache(nb, bs, n_kv, hd, fmt, layers=4, device="cpu")
    row = qm.row_bytes(fmt, hd)
    assert c.shape == (4, 2, nb, n_kv, bs, row) and not c.any()
    assert all(layer.is_contiguous() and (layer.data_ptr() - c.data_ptr()) % 16 == 0 for layer in c)
    assert c.is_contiguous() == (2 * nb * bs * n_kv * row % 16 == 0)


def i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).to(DEV)


@pytest.mark.gpu
@pytest.mark.parametrize("nb,bs,n_kv,hd,fmt", SIZES)
def test_every_layer_is_stored_into(nb, bs, n_kv, hd, fmt):
    T, layers = nb * bs, 3
    caches = sra.quant_kv_cache(nb, bs, n_kv, hd, fmt, layers=layers, device=DEV)
    g = torch.Generator().manual_seed(nb)
    one = torch.ones(T, hd // 2)
    vs = [torch.randn(T, n_kv, hd, generator=g) for _ in range(layers)]
    at = torch.arange(T, device=DEV)
    want = []
    for cache, v in zip(caches, vs):
        k = v.flip(0)
        sra.rope_kv_store_quant(torch.zeros(T, n_kv, hd, device=DEV), k.to(DEV), v.to(DEV), one.to(DEV), 0 * one.to(DEV), at, at, cache)
        want.append([qm.decode(qm.encode(x.double().numpy(), fmt), fmt, hd) for x in (k, v)])

    def held():
        return [[x.double().cpu().numpy() for x in sra.read_kv_quant(cache, i32(np.arange(nb)[None]), i32([0, T]), T, hd, torch.float32)]
                for cache in caches]
    assert all(np.array_equal(x, y) for a, b in zip(held(), want) for x, y in zip(a, b))
    if nb > 1:
        sra.copy_kv_pages(caches, i32([0]), i32([nb - 1]))
        for layer in want:
            for x in layer:
                x[(nb - 1) * bs:] = x[:bs]
        assert all(np.array_equal(x, y) for a, b in zip(held(), want) for x, y in zip(a, b))
