"""Outputs that the binding allocates for a call on another stream than the current one."""
import pytest
import torch

import tensor_core_gemm_tcgen05_gb300 as g

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def ctx():
    from tensor_core_gemm_tcgen05_gb300 import _build
    _build.build()
    c = g.Context(0)
    yield c
    c.close()


@pytest.mark.parametrize("call", ["gemm", "row_softmax", "attention"])
def test_outputs_for_another_stream_leave_freed_memory_alone(ctx, call):
    """A block that was freed on the current stream while queued work there still reads it must not become the
    output of a call on another stream."""
    gen = torch.Generator().manual_seed(1)
    a, b = (torch.randn(2048, 2048, generator=gen).half().to(DEV) for _ in range(2))
    heads = a.view(8, 4096, 128)
    run = {"gemm": lambda s: g.gemm(ctx, a, b, stream=s), "row_softmax": lambda s: g.row_softmax(ctx, a, stream=s),
           "attention": lambda s: g.attention(ctx, heads, heads, heads, stream=s)}[call]
    want = run(None).clone()
    copy = torch.zeros_like(want)
    side, main = torch.cuda.Stream(), torch.cuda.default_stream()
    torch.cuda.synchronize()
    for current, stream in ((main, side), (main, side.cuda_stream), (side, main)):
        with torch.cuda.stream(current):
            old = torch.full_like(want, 3.0)
            torch.cuda.synchronize()
            torch.cuda._sleep(200_000_000)   # (about 0.1 s)
            copy.add_(old)
            del old
            out = run(stream)
            torch.cuda.synchronize()
            assert torch.all(copy == 3.0), "a block still in use became the output"
            assert torch.equal(out, want)
            copy.zero_()
            del out
    assert g.gemm_last_device_error(ctx) == (g.GEMM_OK, 0)
