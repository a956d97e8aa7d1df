"""GPU: calls on a stream other than the current one. What a call makes for the caller is memory of its own stream
(a block that was freed on the current stream may still be in use by work queued there), and a result that
is dropped is not handed out again on that stream before what the current stream has queued by then is done."""
import numpy as np
import pytest
import torch

import swiglu_rmsnorm_add_gb300 as sra

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).to(DEV)


def bf16(*shape):
    return torch.randn(shape, device=DEV).to(torch.bfloat16)


NAMES = ["rmsnorm", "add_rmsnorm", "glu", "uclip", "rmsnorm_linear", "glu_linear", "paged_decode_attention",
         "shared_prefix_attention", "resize_kv_rows", "compact_kv_pages"]


@pytest.fixture(params=NAMES)
def call(request):
    """A function of the stream that makes one call and returns the results that the call made."""
    torch.manual_seed(1)
    x, res, w, W = bf16(24, 1536), bf16(24, 1536), bf16(1536), bf16(320, 1536)
    gate_up, Wd, one = bf16(24, 1280), bf16(256, 640), torch.ones(1, device=DEV)
    q, cache = bf16(5, 12, 128), bf16(2, 40, 16, 2, 128)
    table, seq, plen = i32(np.arange(40).reshape(5, 8)), i32([100, 3, 128, 0, 77]), i32([64])
    state = i32(np.full((6, 4), -1)), i32([0] * 6), i32([0] * 40)
    rows, lens = i32(range(5)), i32([20, 0, 64, 1, 33])
    torch.cuda.synchronize()
    return {
        "rmsnorm": lambda s: [sra.rmsnorm(x, w, stream=s)],
        "add_rmsnorm": lambda s: [sra.add_rmsnorm(x, res, w, stream=s)],
        "glu": lambda s: [sra.glu(gate_up, stream=s)],
        "uclip": lambda s: [sra.uclip(x, one, one, stream=s)],
        "rmsnorm_linear": lambda s: [sra.rmsnorm_linear(x, w, W, stream=s)],
        "glu_linear": lambda s: [sra.glu_linear(gate_up, Wd, stream=s)],
        "paged_decode_attention": lambda s: [sra.paged_decode_attention(q, cache, table, seq, stream=s)],
        "shared_prefix_attention": lambda s: [sra.shared_prefix_attention(q, cache, table[0], plen, table, seq, stream=s)],
        "resize_kv_rows": lambda s: list(sra.resize_kv_rows(*state, rows, lens, cache, stream=s)),
        "compact_kv_pages": lambda s: [sra.compact_kv_pages(*state, cache, stream=s)],
    }[request.param]


@pytest.mark.parametrize("kind", ["object", "integer"])
def test_results_are_the_streams_own_memory(call, kind):
    s = torch.cuda.Stream()
    arg = s if kind == "object" else s.cuda_stream
    shapes = [(t.shape, t.dtype) for t in call(None)]
    torch.cuda.synchronize()
    freed = [torch.empty(a[0], dtype=a[1], device=DEV) for a in shapes]
    ptrs = {t.data_ptr() for t in freed}
    del freed
    got = call(arg)
    assert not ptrs & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    want = call(None)
    torch.cuda.synchronize()
    for g, v in zip(got, want):
        assert g.shape == v.shape and g.dtype == v.dtype


def test_a_dropped_result_waits_for_the_current_stream(call):
    s = torch.cuda.Stream()
    for t in call(s):       # (loads what the first call on a stream loads)
        del t
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)      # about 0.1 s of work on the current stream
    got = call(s)
    shapes, ptrs = [(t.shape, t.dtype) for t in got], {t.data_ptr() for t in got}
    del got
    with torch.cuda.stream(s):
        again = [torch.empty(a[0], dtype=a[1], device=DEV) for a in shapes]
    assert not torch.cuda.current_stream().query(), "the work on the current stream ended before the check"
    assert not ptrs & {t.data_ptr() for t in again}
    torch.cuda.synchronize()


@pytest.mark.parametrize("which", ["object", "integer", "default object", "default integer"])
def test_memory_is_filed_under_the_calls_stream(call, which):
    """What the allocator has on record: results belong to the stream that the call was given, also where that is the
    default stream (whose handle is 0) and another one is current."""
    side, here = torch.cuda.Stream(), torch.cuda.Stream()
    s = torch.cuda.default_stream() if which.startswith("default") else side
    with torch.cuda.stream(here):
        got = call(s if which.endswith("object") else s.cuda_stream)
    torch.cuda.synchronize()
    segments = torch.cuda.memory_snapshot()
    for t in got:
        (owner,) = [g["stream"] for g in segments if g["address"] <= t.data_ptr() < g["address"] + g["total_size"]]
        assert owner == s.cuda_stream


def test_values_on_another_stream_without_its_context():
    """The same results as on the current stream, outputs and workspaces made by the call."""
    torch.manual_seed(2)
    q, cache = bf16(40, 12, 128), bf16(2, 700, 16, 2, 128)
    table = i32(np.arange(300, 700).reshape(40, 10))
    rows = torch.cat([i32(np.tile(np.arange(300), (40, 1))), table], 1).contiguous()
    seq, plen, ptable = i32(4800 + np.arange(40)), i32([4800]), i32(np.arange(300))
    want = sra.shared_prefix_attention(q, cache, ptable, plen, rows, seq)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [sra.shared_prefix_attention(q, cache, ptable, plen, rows, seq, stream=a) for a in (s, s.cuda_stream, s)]
    torch.cuda.current_stream().wait_stream(s)
    for g in got:
        assert torch.equal(g, want)
