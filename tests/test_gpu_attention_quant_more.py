"""GPU: decode attention over a cache in 4 or 8 bits: rings filled again many times.
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
