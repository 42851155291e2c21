"""Outputs that a call allocates itself, on a stream other than the current one.

The allocator hands a freed block out again in the order of the stream that it belongs to.  An output from the current
stream's memory would race twice: with work of the current stream that is still pending on the block when the call
writes it, and with the next owner of the block when the caller drops the output before the call has run.  Both are
made to happen here with a delay kernel on the stream that has to come second, and so is the third: the call's stream
takes the block of a dropped output that work queued on the current stream still reads."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DELAY = 50_000_000                # clock cycles: about 25 ms


@pytest.fixture(scope="module")
def mt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mtp_speculative_decode_gb300 as m
    from mtp_speculative_decode_gb300 import _native
    _native.lib()   # raises if the library is missing: no fallback
    return m


def calls(m):
    """name -> (call on a stream, with no output given)."""
    g = torch.Generator(device="cuda").manual_seed(3)
    a = torch.randint(0, 120, (64, 256), generator=g, device="cuda").to(torch.uint8)
    w = torch.randint(0, 120, (20000, 256), generator=g, device="cuda").to(torch.uint8)
    sa, sw = torch.rand(64, 2, generator=g, device="cuda"), torch.rand(20000, 2, generator=g, device="cuda")
    tokens = torch.randint(0, 50000, (9000,), generator=g, device="cuda")
    offsets = torch.from_numpy(np.arange(0, 9001, 1000, dtype=np.uint32)).cuda()
    logits = torch.randn(300000, 3, generator=g, device="cuda")
    rows = torch.from_numpy(np.arange(300001, dtype=np.uint32)).cuda()
    x = torch.randn(4000, 256, generator=g, device="cuda")
    return {"gemm_fp8_block128": lambda s: m.gemm_fp8_block128(a, sa, w, sw, stream=s),
            "token_counts_build": lambda s: m.token_counts_build(tokens, offsets, 50000, stream=s),
            "process_logits": lambda s: m.process_logits(logits, rows, stream=s),
            "quantize_fp8_block128": lambda s: m.quantize_fp8_block128(x, stream=s)[0]}


NAMES = ["gemm_fp8_block128", "token_counts_build", "process_logits", "quantize_fp8_block128"]


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_pending_work_on_a_freed_block(mt, name, raw):
    call = calls(mt)[name]
    side = torch.cuda.Stream()
    handle = side.cuda_stream if raw else side
    want = call(None).clone()
    torch.empty_like(want).fill_(1)      # the first launch of a kernel loads it, which can wait for the device
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    block = torch.empty_like(want)
    torch.cuda._sleep(DELAY)
    block.fill_(1)                # pending behind the delay
    del block
    got = call(handle)            # runs at once
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_output_dropped_before_the_call_has_run(mt, name, raw):
    call = calls(mt)[name]
    side = torch.cuda.Stream()
    handle = side.cuda_stream if raw else side
    like = call(None)
    call(side)                    # the side stream has memory of its own
    torch.full_like(like, 3)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(DELAY)
    call(handle)                  # pending behind the delay, its output dropped
    others = [torch.full_like(like, 3) for _ in range(3)]
    torch.cuda.synchronize()
    assert all((o == 3).all() for o in others)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_output_dropped_while_the_current_stream_reads_it(mt, name, raw):
    call = calls(mt)[name]
    side = torch.cuda.Stream()
    handle = side.cuda_stream if raw else side
    want = call(None)
    torch.empty_like(want).copy_(want)
    torch.full_like(want, 3)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    got = call(handle)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(DELAY)
    seen = torch.empty_like(want).copy_(got)      # pending behind the delay
    del got
    with torch.cuda.stream(side):
        others = [torch.full_like(want, 3) for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(seen, want) and all((o == 3).all() for o in others)


@pytest.mark.parametrize("name", NAMES)
def test_side_stream_inside_a_capture(mt, name):
    call = calls(mt)[name]
    want = call(None).clone()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        call(side)                       # dropped inside the capture
        got = call(side)
        torch.cuda.current_stream().wait_stream(side)
        seen = got.clone()
    for _ in range(3):
        got.zero_(), seen.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(seen, want)


def test_default_stream_by_its_handle(mt):
    for name, call in calls(mt).items():
        want = call(None)
        with torch.cuda.stream(torch.cuda.Stream()):
            got = call(torch.cuda.default_stream().cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(got, want), name
