"""The attention over 4-bit rows when a wait expires: the launch flags it, leaves what it could not finish, awaits the copies in flight
and leaves the GPU usable.

The kernel is compiled once more so that a wait which is not over at its first probe has expired: the copies in flight are then the
same as when the limit of 2 s passes, and no wait is left out.  Those for copies in flight keep their limit: a launch that came near it
would not have accounted for all of its copies."""
import ctypes as C
import glob
import os
import subprocess
import time

import numpy as np
import pytest
import torch

from test_gpu_cache import SCALE, dev, mla_case, mt, u32  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def one_probe(mt, tmp_path_factory):  # noqa: F811
    """The library with the kernel's waits cut to one probe."""
    from mtp_speculative_decode_gb300 import _native, build
    objs = glob.glob(os.path.join(build.BUILD, "*.o"))
    if not objs:
        build.build()
        objs = glob.glob(os.path.join(build.BUILD, "*.o"))
    d = tmp_path_factory.mktemp("one_probe")
    obj = str(d / "k_mla4_tc.o")
    subprocess.run([build.nvcc(), *build.ARCH, *build.NVCC_FLAGS, "-DMTPSD_HEAD_ONE_PROBE", "-I", build.INCLUDE, "-c",
                    os.path.join(build.CSRC, "k_mla4_tc.cu"), "-o", obj], check=True, capture_output=True)
    so = str(d / "libmtpsd_one_probe.so")
    rest = [o for o in objs if os.path.basename(o) != "k_mla4_tc.o"]
    subprocess.run([build.nvcc(), *build.ARCH, "-shared", "-cudart", "static", "-o", so, *rest, obj], check=True)
    lib = C.CDLL(so)
    for name, (res, args) in _native.SIGNATURES.items():
        getattr(lib, name).restype, getattr(lib, name).argtypes = res, args
    return lib


@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("B,W,H,n_idx", [(1, 1, 128, 64), (1, 1, 128, 2048), (2, 1, 48, 700), (3, 2, 128, 2048), (35, 2, 128, 300)])
def test_attention_after_an_expired_wait(mt, one_probe, monkeypatch, B, W, H, n_idx, page):  # noqa: F811
    from mtp_speculative_decode_gb300 import _native as N
    rng = np.random.default_rng(B)
    q, rows, caps, start, pos, idx = mla_case(rng, B, W, H, n_idx, [2500] * B)
    paged, cs = None, dev(start)
    if page:
        n = -(-caps[0] // page)
        pool = np.zeros((B * n * page, 416), np.uint8)
        for b in range(B):
            pool[b * n * page:b * n * page + caps[b]] = rows[start[b]:start[b] + caps[b]]
        rows, paged, cs = pool, (dev(np.arange(B * n, dtype=np.int32).reshape(B, n)), page), None
    args = (q.cuda(), dev(rows), cs, u32(np.arange(B + 1) * W), dev(pos), dev(idx), SCALE)
    MARK = -1e4

    def run():
        out, st = torch.full((B * W, H, 512), MARK, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        t0 = time.monotonic()
        mt.sparse_mla_decode(*args, out=out, dev_status=st, paged=paged)
        torch.cuda.synchronize()
        return out, st.item(), time.monotonic() - t0

    want, st, _ = run()
    assert st == 0 and (want.float().abs() < 100).all()
    with monkeypatch.context() as mp:
        mp.setattr(N, "_lib", one_probe)
        got, st, took = run()
    # a row's CTAs finish or leave their half of its values (rows without a selected position need no wait)
    left = got == MARK
    assert st == N.STATUS_WAIT_TIMEOUT and took < 1.0 and left.any() and torch.equal(got[~left], want[~left])
    again, st, _ = run()                                             # the device works on
    assert st == 0 and torch.equal(again, want)
