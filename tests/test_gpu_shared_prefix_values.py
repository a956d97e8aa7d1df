"""GPU: attention over a shared prefix where scores or values leave the ordinary range, in every form, against
the formula in 64 bits with the tolerance of test_gpu_shared_prefix (it is relative to sum_t p_t |V_t|, so it holds for
values of any size that sums of them in fp32 can hold).

What the formula gives: a score of -inf has weight 0; a request with no score above -inf gets zeros; a NaN among a
request's scores makes its output NaN."""
import numpy as np
import pytest
import torch

import swiglu_rmsnorm_add_gb300 as sra
from tests.test_gpu_shared_prefix import DEV, Case, path, run  # noqa: F401  (path: the fixture)

pytestmark = pytest.mark.gpu

KINDS = [(torch.bfloat16, 64), (torch.bfloat16, 128), (torch.bfloat16, 256), (torch.float16, 64), (torch.float16, 128),
         (torch.float16, 256), (torch.float32, 64), (torch.float32, 128), (torch.float32, 256)]


def set_tokens(c, which, fill):
    """fill(plane K, page, row) for the tokens t of request b (None: of the prefix) in which(b)."""
    for b in [None] + list(range(c.B)):
        for t in which(b):
            shared = t < c.P
            if shared != (b is None) or (b is not None and t >= c.lens[b]):
                continue
            page = int(c.ptable[t // c.bs] if shared else c.table[b, t // c.bs])
            fill(c.cache, page, t % c.bs)


def close(c, got, what=""):
    """As Case.check, but with zeros for a request without a score above -inf and NaN exactly where the formula has it."""
    o, A = c.want()
    u = torch.finfo(c.dtype).eps / 2
    up = 0.0 if c.dtype == torch.float32 else u
    nothing = torch.zeros(c.q.shape[:2], dtype=torch.bool, device=DEV)
    G = c.q.shape[1] // c.n_kv
    for b in range(c.B):
        w = c.where(b)
        if w:
            k = c.cache.to(DEV).flatten(1, 2)[0, torch.tensor(w, device=DEV)].double()
            for h in range(c.n_kv):
                s = c.scale * c.q.to(DEV)[b, h * G:h * G + G].double() @ k[:, h].T
                nothing[b, h * G:h * G + G] = (s == -torch.inf).all(-1)
    o[nothing], A[nothing] = 0.0, 0.0
    assert torch.equal(got.isnan(), o.isnan()), (what, int(got.isnan().sum()), int(o.isnan().sum()))
    ok = ((got.double() - o).abs() <= u * o.abs() + (up + 6e-5) * A + 1e-30) | o.isnan()
    assert bool(ok.all()), (what, int((~ok).sum()), [int(x) for x in (~ok).nonzero()[0]])


@pytest.mark.parametrize("dtype,hd", KINDS)
def test_scores_of_minus_infinity(dtype, hd, path):
    """The first 40 tokens of the prefix, some later ones and the first 20 behind the prefix have no weight: whole
    leading tiles without a score above -inf, requests that end among such tokens, a prefix that ends in a page."""
    lens = [150, 160, 165, 300, 0, 7, 40, 41, 90, 151, 260, 171, 172, 400, 152, 149]
    c = Case(16, 12, 2, hd, 16, 150, lens, dtype, 21 + hd)
    c.q[..., 0] = c.q[..., 0].abs() + 0.5

    def fill(cache, page, row):
        cache[0, page, row, :, 0] = -torch.inf

    set_tokens(c, lambda b: [*range(40), 64, 100, *range(128, 144)] if b is None else range(150, 170), fill)
    d = c.dev()
    close(c, sra.shared_prefix_attention(**d, scale=c.scale))
    set_tokens(c, lambda b: range(150) if b is None else range(150, 172), fill)     # nothing in the prefix counts
    close(c, sra.shared_prefix_attention(**c.dev(), scale=c.scale), "none of the prefix")


@pytest.mark.parametrize("dtype,hd", KINDS)
def test_nan_queries_and_keys(dtype, hd, path):
    """NaN in one head of a request's query, or in a token that a request attends to, and nowhere else in the output."""
    c = Case(20, 12, 2, hd, 16, 150, [150 + 5 * (b % 7) for b in range(20)], dtype, 31 + hd)
    c.lens[9] = c.lens[10] = 33
    c.q[3, 5, 7] = torch.nan
    c.q[9, 0] = torch.nan
    page = int(c.table[12, 150 // 16])
    c.cache[0, page, 150 % 16, 1, 3] = torch.nan      # request 12's own first token, its second KV head
    close(c, sra.shared_prefix_attention(**c.dev(), scale=c.scale))


@pytest.mark.parametrize("B", [20, 130])
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_values_near_the_end_of_the_range(hd, B, path):
    """V of 1.5e36 and a maximum that rises by 2^7.875 in a later tile of a split. The 212 tokens' |V| add up to 3.2e38,
    within fp32 and bf16, so sums of them with weights of at most 1 are finite whatever their signs; a weight of 2^7.875
    would make one token's 3.5e38 infinite. (As many KV heads as SMs: a split has three tiles, of one row tile or two.)"""
    n_kv = torch.cuda.get_device_properties(0).multi_processor_count
    prefix, own = 192, 20
    c = Case(B, n_kv, n_kv, hd, 16, prefix, [prefix + own if b < 3 else prefix + 1 for b in range(B)], torch.bfloat16, 5,
             scale=float(np.log(2.0)))
    c.q.zero_()
    c.q[..., 0] = 1
    some = ~c.cache[0].isnan().any(-1)
    c.cache[0][some] = 0.0
    c.cache[1][some] = 1.5e36 * c.cache[1][some].sign()

    def fill(cache, page, row):
        cache[0, page, row, :, 0] = 7.875

    set_tokens(c, lambda b: [150] if b is None else [prefix + 15], fill)
    got = sra.shared_prefix_attention(**c.dev(), scale=c.scale)
    assert bool(got.isfinite().all())
    close(c, got)


@pytest.mark.parametrize("dtype,hd", KINDS)
def test_a_scale_of_zero(dtype, hd, path):
    """Every token has the same weight, whatever its score: also where scores are as large as the type allows; and
    0 times an infinite score is NaN."""
    c = Case(20, 12, 2, hd, 16, 150, [150 + 5 * (b % 7) for b in range(20)], dtype, 41 + hd, scale=0.0)
    big = 2.0 ** 7 if dtype == torch.float16 else 2.0 ** 61
    c.q[..., 0] = big
    some = ~c.cache[0].isnan().any(-1)
    c.cache[0][..., 0][some] = (torch.randint(0, 2, (int(some.sum()),), generator=torch.Generator().manual_seed(1)) * 2.0
                                - 1.0).to(dtype) * big
    close(c, sra.shared_prefix_attention(**c.dev(), scale=0.0))
    page = int(c.ptable[2])
    c.cache[0, page, 3, 1, 0] = -torch.inf      # token 35 of the prefix, for the second KV head
    c.lens[4] = 20
    close(c, sra.shared_prefix_attention(**c.dev(), scale=0.0), "an infinite score")
    c.q[7, 2, 5] = torch.inf
    close(c, sra.shared_prefix_attention(**c.dev(), scale=0.0), "an infinite query")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_an_empty_workspace_keeps_the_probabilities(dtype):
    """The form without a workspace, from Python: the forced decode form's result, with probabilities of 16 bits (2^-16 of
    A instead of the half step of the dtype that one rounding costs; a residual that is subnormal in fp16 is off by
    half a step of 2^-24, 2^-25 of the largest probability each)."""
    c = Case(70, 12, 2, 128, 16, 2000, [2000 + b % 50 for b in range(70)], dtype, 8)
    d = c.dev()
    got = sra.shared_prefix_attention(**d, scale=c.scale, workspace=torch.empty(0, dtype=torch.uint8, device=DEV))
    sra.force_variant("shared_prefix", 0)
    try:
        want = sra.shared_prefix_attention(**d, scale=c.scale)
    finally:
        sra.force_variant("shared_prefix", -1)
    assert torch.equal(got, want)
    assert not torch.equal(got, sra.shared_prefix_attention(**d, scale=c.scale))     # (this size is taken together)
    o, A = c.want()
    V = c.cache.to(DEV).float().nan_to_num().abs().max().double()
    tiny = 2.0 ** -25 * 2050 * V if dtype == torch.float16 else 0.0
    tol = torch.finfo(dtype).eps / 2 * o.abs() + (2.0 ** -16 + 6e-5) * A + tiny + 1e-30
    assert bool(((got.double() - o).abs() <= tol).all())
