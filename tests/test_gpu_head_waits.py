"""The waits of the head's kernels: nothing is on its way to a CTA that has left."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mtp_speculative_decode_gb300 as m
    from mtp_speculative_decode_gb300 import _native
    _native.lib()   # raises if the library is missing: no fallback
    return m


def operands(M, N, K, w_rows, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n_sc = N if w_rows == 1 else -(-N // 128)
    rand = lambda rows: torch.randint(0, 127, (rows, K), generator=g, device="cuda").to(torch.uint8)  # noqa: E731
    return (rand(M), torch.rand(M, K // 128, generator=g, device="cuda"), rand(N),
            torch.rand(n_sc, K // 128, generator=g, device="cuda"))


def test_products_on_pairs_back_to_back(mt):
    """A CTA of the next launch takes the shared memory and TMEM of one that has just left: short launches of pairs (few
    blocks, so that the last commits make up most of a launch) and of the other kernels, on two streams in turn."""
    sizes = [(65, 64, 128, 1), (300, 200, 128, 128), (129, 1000, 768, 1), (256, 256, 1152, 128), (8, 576, 512, 1),
             (513, 385, 384, 128), (70, 40000, 256, 1)]
    cases = [operands(*s, seed=i) for i, s in enumerate(sizes)]
    want = [mt.gemm_fp8_block128(*c, out_dtype=torch.float32).clone() for c in cases]
    streams = [torch.cuda.Stream() for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for turn in range(20):
        got = []
        for s in streams:
            with torch.cuda.stream(s):
                got += [mt.gemm_fp8_block128(*c, out_dtype=torch.float32, dev_status=status) for c in cases]
        torch.cuda.synchronize()
        assert status.item() == 0
        for i, o in enumerate(got):
            assert torch.equal(o, want[i % len(want)]), (turn, sizes[i % len(want)])
