"""The waits of the head's kernels: nothing is on its way to a CTA that has left, and a launch whose wait expires flags
it, leaves what it could not finish and leaves the GPU usable.

For the latter the kernels are compiled once more so that a wait which is not over at its first probe has expired: the
copies and arrivals in flight are then the same as when the limit of 2 s passes, and no wait is left out.  The launches
run to their end, without a fault, and the ordinary library's results are compared after them."""
import ctypes as C
import glob
import os
import subprocess

import numpy as np
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


ONE_PROBE = ["k_logits.cu", "k_gemm_fp8.cu"]


@pytest.fixture(scope="module")
def one_probe(mt, tmp_path_factory):
    """The library with the waits of the head's kernels cut to one probe."""
    from mtp_speculative_decode_gb300 import _native, build
    objs = glob.glob(os.path.join(build.BUILD, "*.o"))
    if not objs:
        build.build()
        objs = glob.glob(os.path.join(build.BUILD, "*.o"))
    d = tmp_path_factory.mktemp("one_probe")
    jobs = []
    for src in ONE_PROBE:
        obj = str(d / src.replace(".cu", ".o"))
        cmd = [build.nvcc(), *build.ARCH, *build.NVCC_FLAGS, "-DMTPSD_HEAD_ONE_PROBE", "-I", build.INCLUDE, "-c",
               os.path.join(build.CSRC, src), "-o", obj]
        jobs.append((obj, subprocess.Popen(cmd, stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL)))
        objs = [o for o in objs if os.path.basename(o) != os.path.basename(obj)] + [obj]
    assert all(p.wait() == 0 for _, p in jobs)
    so = str(d / "libmtpsd_one_probe.so")
    subprocess.run([build.nvcc(), *build.ARCH, "-shared", "-cudart", "static", "-o", so, *objs], check=True)
    lib = C.CDLL(so)
    for name, (res, args) in _native.SIGNATURES.items():
        getattr(lib, name).restype, getattr(lib, name).argtypes = res, args
    return lib


def u32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.uint32)).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,K,V,outputs", [
    (400, 5, 12000, "apo"), (400, 5, 12000, "a"),                    # one CTA per row
    (150, 5, 50001, "apo"), (150, 5, 50001, "a"),                    # clusters, rows that are not 16-byte aligned
    (64, 5, 154880, "apo"), (64, 5, 154880, "ap"), (64, 5, 154880, "a")])
def test_logits_after_an_expired_wait(mt, one_probe, monkeypatch, B, K, V, outputs, dtype):
    from mtp_speculative_decode_gb300 import _native as N
    g = torch.Generator(device="cuda").manual_seed(V)
    R = B * (K + 1)
    x = torch.randn(R, V, generator=g, device="cuda").to(dtype)
    temp = torch.rand(B, generator=g, device="cuda") + 0.5
    temp[::3] = 0                                                    # greedy requests among them
    kw = dict(temperature=temp, repetition=torch.full((B,), 1.2, device="cuda"),
              draft=torch.randint(0, V, (B, K), generator=g, device="cuda"),
              bitmask=torch.randint(-2 ** 31, 2 ** 31, (R, -(-V // 32)), generator=g, device="cuda").to(torch.int32))
    off = u32(np.arange(0, R + 1, K + 1))
    MARK = -7.0

    def run():
        out = dict(argmax=torch.full((R,), int(MARK), dtype=torch.int64, device="cuda"))
        if "p" in outputs:
            out["probs"] = torch.full((R, V), MARK, device="cuda")
        if "o" in outputs:
            out["out_logits"] = torch.full((R, V), MARK, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        mt.process_logits(x, off, dev_status=st, **kw, **out)
        torch.cuda.synchronize()
        return out, st.item()

    want, st = run()
    assert st == 0 and (want["argmax"] >= 0).all()
    with monkeypatch.context() as mp:
        mp.setattr(N, "_lib", one_probe)
        got, st = run()
    # a copy of a few rows of one CTA may be there at the first probe; the values of a cluster's other CTAs never all are
    assert st == N.STATUS_WAIT_TIMEOUT or (st == 0 and V < 20000)
    left = got["argmax"] == MARK
    assert left.any() == (st != 0) and torch.equal(got["argmax"][~left], want["argmax"][~left])
    if "p" in outputs:
        assert (got["probs"][left] == MARK).all() and torch.equal(got["probs"][~left], want["probs"][~left])
    if "o" in outputs:
        o, w = got["out_logits"], want["out_logits"]
        assert torch.equal(o[~left], w[~left]) and ((o == w) | (o == MARK)).all()
    again, st = run()                                                # the device works on
    assert st == 0 and all(torch.equal(again[k], want[k]) for k in want)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K,w_rows", [(1, 576, 6144, 1), (64, 640, 12288, 128), (33, 2049, 1920, 1),      # K split over a cluster
                                          (64, 6144, 12288, 128), (16, 40001, 640, 1), (33, 60000, 256, 128)])
def test_few_row_product_after_an_expired_wait(mt, one_probe, monkeypatch, M, N, K, w_rows, out):
    from mtp_speculative_decode_gb300 import _native as nat
    case = operands(M, N, K, w_rows, seed=N)

    def run():
        o = torch.full((M, N), -7.0, dtype=out, device="cuda")       # every product is positive
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        mt.gemm_fp8_block128(*case, out=o, dev_status=st)
        torch.cuda.synchronize()
        return o, st.item()

    want, st = run()
    assert st == 0 and (want > 0).all()
    with monkeypatch.context() as mp:
        mp.setattr(nat, "_lib", one_probe)
        got, st = run()
    left = got == -7
    assert st == nat.STATUS_WAIT_TIMEOUT and left.any() and torch.equal(got[~left], want[~left])
    again, st = run()                                                # the device works on
    assert st == 0 and torch.equal(again, want)
