"""Pins of the oracle of the FP8 product, the logits processing and the token
table against facts fixed outside it, and the refusals of the calls (host
checks, before any launch).  CPU only."""
import ctypes as C
import math
import os

import numpy as np
import pytest
import torch

from oracle import fp8, gemm, logits


# --------------------------------------------------------------------- FP8 product

@pytest.mark.parametrize("rows", [1, 128])
def test_gemm_equals_the_dequantized_product(rows):
    rng = np.random.default_rng(0)
    M, N, K = 3, 200, 256
    a, w = rng.integers(0, 0x7F, (M, K)).astype(np.uint8), rng.integers(0, 0x7F, (N, K)).astype(np.uint8)
    a ^= rng.integers(0, 2, a.shape).astype(np.uint8) << 7
    sa = rng.uniform(0.1, 2, (M, 2)).astype(np.float32)
    sw = rng.uniform(0.1, 2, (N if rows == 1 else 2, 2)).astype(np.float32)
    got = gemm.gemm_fp8_block128(a, sa, w, sw, rows)
    da = torch.from_numpy(a).view(torch.float8_e4m3fn).double() * torch.from_numpy(sa).double().repeat_interleave(128, 1)
    full = torch.from_numpy(sw).double().repeat_interleave(128, 1).repeat_interleave(rows, 0)[:N]
    dw = torch.from_numpy(w).view(torch.float8_e4m3fn).double() * full
    want = (da @ dw.T).numpy()
    assert np.allclose(got, want, rtol=1e-13, atol=1e-13 * np.abs(want).max())


def test_gemm_hand_worked():
    # one-hot rows pick single weights: 1.0 * 2^-1 (scale) * value * scale of the block that holds it
    a = np.zeros((2, 256), np.uint8)
    a[0, 5], a[1, 130] = 0x38, 0xB8                      # 1.0, -1.0
    w = np.zeros((130, 256), np.uint8)
    w[0, 5], w[129, 130] = 0x40, 0x7E                    # 2.0, 448
    sa = np.array([[0.5, 9.0], [7.0, 0.25]], np.float32)
    sw = np.array([[3.0, 11.0], [13.0, 2.0]], np.float32)
    out = gemm.gemm_fp8_block128(a, sa, w, sw, 128)
    assert out[0, 0] == 0.5 * 2.0 * 3.0 and out[1, 129] == -0.25 * 448 * 2.0
    assert np.count_nonzero(out) == 2
    assert gemm.abs_terms(a, sa, w, sw, 128)[1, 129] == 0.25 * 448 * 2.0


# --------------------------------------------------------------------- logits

def test_row_hand_worked():
    x = [2.0, -1.0, 4.0, 0.5, 3.0]
    word = [-32768, -32768, 2, 0, 0]                      # 0 and 1 in the prompt, 2 put out twice
    y, arg, p = logits.process_row(x, word, drafts=[2, 3], repetition=2.0, frequency=0.25, presence=0.5,
                                   biases=[(4, 1.0), (1, 10.0), (4, -3.5), (99, 5.0)], mask=[0b11110])
    # 0: masked; 1: -1 * 2 + 10; 2: 4 / 2 - 0.25 * 3 - 0.5; 3: 0.5 / 2 - 0.25 - 0.5; 4: 3 + 1 - 3.5
    assert y.tolist() == [-math.inf, 8.0, 0.75, -0.5, 0.5] and arg == 1
    e = np.exp(np.array([-math.inf, 0.0, -7.25, -8.5, -7.5]))
    assert np.allclose(p, e / e.sum(), rtol=1e-15)


def test_row_plain_softmax_and_temperature():
    x = np.random.default_rng(1).normal(size=50)
    _, arg, p = logits.process_row(x, temperature=0.7)
    assert arg == int(np.argmax(x))
    assert np.allclose(p, torch.softmax(torch.from_numpy(x) / 0.7, 0).numpy(), rtol=1e-13)
    assert logits.process_row(x, temperature=0.0)[2].tolist() == [float(t == arg) for t in range(50)]


def test_row_edges():
    inf, nan = math.inf, math.nan
    y, arg, p = logits.process_row([1.0, 2.0], mask=[0])
    assert arg == -1 and p.tolist() == [0.0, 0.0] and y.tolist() == [-inf, -inf]
    _, arg, p = logits.process_row([nan, 2.0, inf], mask=[0b010])       # what is masked does not matter
    assert arg == 1 and p.tolist() == [0.0, 1.0, 0.0]
    _, arg, p = logits.process_row([1.0, inf, inf, -inf])
    assert arg == 1 and p.tolist() == [0.0, 0.5, 0.5, 0.0]
    _, arg, p = logits.process_row([1.0, nan, 3.0])
    assert arg == 1 and np.isnan(p).all()
    lowest = float(np.finfo(np.float32).min)
    _, arg, p = logits.process_row([lowest, lowest])
    assert arg == 0 and p.tolist() == [0.5, 0.5]


def test_token_table_hand_worked():
    V = 5
    t = np.full((3, 8), 7, np.int16)
    got = logits.token_counts_build(t, [1, 1, 4, 1, 9, 2, 2, 2], [0, 5, 8], V, n_prompt=[3, 0])
    assert got[0].tolist() == [0, -32767, 0, 0, -32768, 0, 0, 0]        # 1: prompt and one output; 9 is no token
    assert got[1].tolist() == [0, 0, 3, 0, 0, 0, 0, 0] and got[2].tolist() == [7] * 8
    got = logits.token_counts_accept(got, V, np.array([[1, 4, 0], [3, 3, 3]]), [2, 5], np.array([1, 2]))
    assert got[0].tolist() == [0, -32765, 0, 0, -32767, 0, 0, 0]
    assert got[1].tolist() == [0, 0, 4, 3, 0, 0, 0, 0]
    full = np.array([[32767, -1]], np.int16)                             # counts at the limit stay there
    assert logits.token_counts_accept(full, 2, None, None, np.array([0])).tolist() == [[32767, -1]]
    assert logits.token_counts_accept(full, 2, None, None, np.array([1])).tolist() == [[32767, -1]]
    rows = logits.token_counts_build(t, [1, 2], [0, 1, 2], V, count_rows=[2, -1])
    assert rows[2].tolist() == [0, -32768, 0, 0, 0, 0, 0, 0] and rows[0].tolist() == [7] * 8


# --------------------------------------------------------------------- refusals

@pytest.fixture(scope="module")
def native():
    from mtp_speculative_decode_gb300 import _native
    if not os.path.exists(_native.LIB_PATH):
        from mtp_speculative_decode_gb300 import build
        build.build()
    _native.lib()
    return _native


def test_struct_layout(native):
    import test_abi
    fields = [f for f, _ in native.LogitsArgs._fields_]
    got = test_abi._c_offsets("mtpsd_logits_args", fields)
    assert got == [C.sizeof(native.LogitsArgs)] + [getattr(native.LogitsArgs, f).offset for f in fields]


def test_gemm_refusals(native):
    f = native.lib().mtpsd_gemm_fp8_block128
    E, U = native.MTPSD_EINVAL, native.MTPSD_EUNSUPPORTED
    ok = dict(a=16, sa=16, w=16, sw=16, rows=1, M=4, N=8, K=256, dt=native.MTPSD_BF16, out=16, ld=8)
    for change, code in ((dict(M=-1), E), (dict(N=1 << 31), E), (dict(M=(1 << 31) - 255), E), (dict(K=64), U), (dict(rows=2), U),
                         (dict(dt=native.MTPSD_FP8_E4M3), U), (dict(ld=7), E), (dict(a=None), E), (dict(sw=None), E),
                         (dict(out=None), E), (dict(a=8), E), (dict(w=17), E), (dict(out=17), E),
                         (dict(out=18, dt=native.MTPSD_F32), E), (dict(sa=18), E)):
        assert f(*{**ok, **change}.values(), None, None) == code, change
        assert b"gemm_fp8_block128" in native.lib().mtpsd_last_error()
    for change in (dict(M=0), dict(N=0, ld=0), dict(M=0, a=None, out=None)):      # nothing to do
        assert f(*{**ok, **change}.values(), None, None) == 0


def test_token_table_refusals(native):
    L = native.lib()
    E = native.MTPSD_EINVAL
    assert [L.mtpsd_token_counts_ld(v) for v in (1, 8, 9, 154880, 0)] == [8, 8, 16, 154880, 0]
    ok = dict(tokens=8, S=4, offsets=8, n_prompt=None, B=2, V=10, counts=16, ld=16, n_rows=2, rows=None)
    for change in (dict(B=-1), dict(S=-1), dict(S=1 << 32), dict(V=0), dict(V=1 << 31), dict(counts=None),
                   dict(counts=8), dict(ld=8), dict(ld=12), dict(n_rows=1), dict(offsets=None), dict(tokens=None),
                   dict(n_rows=-1, rows=8)):
        assert L.mtpsd_token_counts_build(*{**ok, **change}.values(), None, None) == E, change
    assert L.mtpsd_token_counts_build(*{**ok, "B": 0, "counts": None}.values(), None, None) == 0
    ok = dict(draft=8, n_acc=8, nxt=8, B=2, K=3, V=10, counts=16, ld=16, n_rows=2, rows=None)
    for change in (dict(B=-1), dict(K=-1), dict(B=1 << 20, K=1 << 20), dict(V=0), dict(counts=None), dict(ld=9),
                   dict(n_rows=1), dict(draft=None), dict(n_acc=None), dict(nxt=None)):
        assert L.mtpsd_token_counts_accept(*{**ok, **change}.values(), None, None) == E, change
    assert L.mtpsd_token_counts_accept(*{**ok, "B": 0}.values(), None, None) == 0


def test_process_refusals(native):
    L = native.lib()
    E, U = native.MTPSD_EINVAL, native.MTPSD_EUNSUPPORTED
    ok = dict(B=2, R=4, V=40, dtype=native.MTPSD_F32, logits=16, ld=40, row_offsets=8, argmax=8)
    for change, code in ((dict(B=0), E), (dict(R=-1), E), (dict(V=0), E), (dict(V=393217, ld=393217), U),
                         (dict(R=(1 << 24) + 1), U), (dict(dtype=native.MTPSD_FP8_E4M3), U), (dict(ld=39), E),
                         (dict(probs=16, probs_ld=39), E), (dict(out_logits=16, out_ld=0), E), (dict(argmax=None), E),
                         (dict(K=-1), E), (dict(K=2), E), (dict(logits=None), E), (dict(row_offsets=None), E),
                         (dict(counts=16, counts_ld=39, counts_rows=2), E),
                         (dict(counts=16, counts_ld=40, counts_rows=1), E),
                         (dict(counts=8, counts_ld=40, counts_rows=2), E),
                         (dict(bias_offsets=8, n_bias=-1), E), (dict(bias_offsets=8, n_bias=3), E),
                         (dict(bias_offsets=8, bias_tokens=8, bias_values=8, n_bias=(1 << 31) - 1, K=1, draft=8), E),
                         (dict(bitmask=8, n_masks=3), E), (dict(bitmask=8, n_masks=-1, mask_rows=8), E),
                         (dict(logits=18), E), (dict(probs=18, probs_ld=40), E),
                         (dict(out_logits=16, out_ld=48), E),                                  # in place, other stride
                         (dict(out_logits=16, out_ld=40, dtype=native.MTPSD_BF16), E)):        # in place, bf16
        a = native.LogitsArgs(**{**ok, **change})
        assert L.mtpsd_process_logits(C.byref(a), None) == code, change
        assert b"process_logits" in L.mtpsd_last_error()
    assert L.mtpsd_process_logits(None, None) == E
    a = native.LogitsArgs(**{**ok, "R": 0, "logits": None})
    assert L.mtpsd_process_logits(C.byref(a), None) == 0


def test_misaligned_arrays_are_refused(native):
    """Every array of integers and floats has to be aligned to its elements: the kernels load whole elements."""
    L, E = native.lib(), native.MTPSD_EINVAL
    st = dict(status=None, stream=None)
    ok = dict(a=16, sa=16, w=16, sw=16, rows=1, M=4, N=8, K=256, dt=native.MTPSD_BF16, out=16, ld=8, **st)
    for change in (dict(sw=6), dict(status=2)):
        assert L.mtpsd_gemm_fp8_block128(*{**ok, **change}.values()) == E, change
    ok = dict(tokens=8, S=4, offsets=8, n_prompt=8, B=2, V=10, counts=16, ld=16, n_rows=2, rows=None, **st)
    for change in (dict(tokens=12), dict(offsets=6), dict(n_prompt=12), dict(rows=6), dict(status=2)):
        assert L.mtpsd_token_counts_build(*{**ok, **change}.values()) == E, change
    ok = dict(draft=8, n_acc=8, nxt=8, B=2, K=3, V=10, counts=16, ld=16, n_rows=2, rows=None, **st)
    for change in (dict(draft=12), dict(n_acc=6), dict(nxt=12), dict(rows=6), dict(status=2)):
        assert L.mtpsd_token_counts_accept(*{**ok, **change}.values()) == E, change
    ok = dict(B=2, R=4, V=40, K=1, dtype=native.MTPSD_F32, logits=16, ld=40, row_offsets=8, argmax=8, draft=8,
              counts=16, counts_ld=40, counts_rows=2, bias_tokens=8, bias_values=8, n_bias=1, n_masks=4)
    for field in ("row_offsets", "repetition", "frequency", "presence", "bias_offsets", "bias_tokens", "bias_values",
                  "bitmask", "mask_rows", "temperature", "dev_status", "count_rows"):
        a = native.LogitsArgs(**{**ok, field: 10})
        assert L.mtpsd_process_logits(C.byref(a), None) == E, field
    for field in ("draft", "argmax"):
        a = native.LogitsArgs(**{**ok, field: 12})
        assert L.mtpsd_process_logits(C.byref(a), None) == E, field


def test_binding_refuses_host_tensors():
    import mtp_speculative_decode_gb300 as m
    x = torch.zeros(2, 128, dtype=torch.uint8)
    with pytest.raises(ValueError):
        m.gemm_fp8_block128(x, torch.zeros(2, 1), x, torch.zeros(2, 1))
    with pytest.raises(ValueError):
        m.process_logits(torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError):
        m.process_logits(None, None)
    with pytest.raises(ValueError):
        m.token_counts_build(torch.zeros(2, dtype=torch.int64), None, 8)
    assert fp8.BLOCK == 128
