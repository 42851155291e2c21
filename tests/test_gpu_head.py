"""The FP8 block-128 product, the logits processing and the token table through
the binding, against the float64 oracle (oracle.gemm, oracle.logits), and the
verify head that runs them together with the quantizer and the acceptance.

Tolerances, derived from the arithmetic:
* product: a block sum of 128 products and the sum of the block sums are held in float32.  An
  addition is off by at most one unit in the last place of its result (2^-23, truncation allowed), a
  scale multiplication by half (2^-24), each relative to no more than T = sum |terms|: at most
  (128 + K/128 + 3) 2^-23 T; then half a step of the output type.
* processed logits: at most 5 roundings plus one per bias of the token, each at most 2^-24 of the
  largest magnitude on the way, bounded by the sum S of the magnitudes of all terms.
* probabilities: the exponent d / T moves by the error of the two logits over T plus 2^-22 |d / T|
  (difference, division), exp is good to 2^-22, the sum of V positive terms to 2^-23 per addition of
  the longest chain (at most 512 below), the division to 2^-24.  Values below 2^-126 may flush to 0."""
import math

import numpy as np
import pytest
import torch

from oracle import accept as oaccept
from oracle import fp8 as ofp8
from oracle import gemm as ogemm
from oracle import logits as ologits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mtp_speculative_decode_gb300 as m
    from mtp_speculative_decode_gb300 import _native
    _native.lib()   # raises if the library is missing: no fallback
    return m


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)) if isinstance(x, np.ndarray) else torch.as_tensor(x)
    return (t if dtype is None else t.to(dtype)).cuda().contiguous()


def u32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.uint32)).cuda()


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ----------------------------------------------------------------------------- FP8 product

def codes(rng, rows, K):
    """Codes of quantized normal values: every block reaches 448."""
    x = rng.normal(size=(rows, K)).astype(np.float32)
    if K == 0:
        return np.zeros((rows, 0), np.uint8)
    c, _ = ofp8.quantize_block128(x)
    return c


def product_case(seed, M, N, K, w_rows):
    rng = np.random.default_rng(seed)
    a, w = codes(rng, M, K), codes(rng, N, K)
    sa = np.exp(rng.normal(size=(M, K // 128)) * 2 - 6).astype(np.float32)
    sw = np.exp(rng.normal(size=(N if w_rows == 1 else -(-N // 128), K // 128)) * 2 - 6).astype(np.float32)
    return a, sa, w, sw


def check_product(got, a, sa, w, sw, w_rows):
    K = a.shape[1]
    want = ogemm.gemm_fp8_block128(a, sa, w, sw, w_rows)
    T = ogemm.abs_terms(a, sa, w, sw, w_rows)
    tol = (128 + K // 128 + 3) * 2.0 ** -23 * T
    tol += torch.finfo(got.dtype).eps / 2 * (np.abs(want) + tol) + 1e-37
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), f"worst error / tolerance {np.max(err / tol)}"


@pytest.mark.parametrize("w_rows", [1, 128])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(1, 1, 128), (1, 576, 6144), (2, 127, 256), (3, 128, 384), (15, 129, 128),
                                   (16, 640, 1920), (17, 300, 512), (33, 2049, 256), (64, 512, 12288), (65, 130, 1152),
                                   (129, 257, 640), (192, 1000, 768), (193, 264, 128), (255, 136, 2048),
                                   (257, 200, 896), (300, 1030, 256), (513, 385, 384), (1025, 129, 128)])
def test_product(mt, M, N, K, out, w_rows):
    a, sa, w, sw = product_case(M * 7 + N, M, N, K, w_rows)
    st = status()
    got = mt.gemm_fp8_block128(dev(a), dev(sa), dev(w), dev(sw), out_dtype=out, dev_status=st)
    assert got.dtype == out and st.item() == 0
    check_product(got, a, sa, w, sw, w_rows)


@pytest.mark.parametrize("w_rows", [1, 128])
@pytest.mark.parametrize("M,N,K", [(1, 40000, 384), (16, 40001, 640), (20, 60011, 128), (32, 30000, 1408), (33, 40007, 640),
                                   (64, 60000, 1152), (65, 50001, 384), (200, 40000, 640), (300, 30001, 896)])
def test_product_many_tiles_per_cta(mt, M, N, K, w_rows):
    """Several tiles a CTA, with numbers of blocks that are no multiple of the rings, slots, buffers and sets."""
    a, sa, w, sw = product_case(M + N, M, N, K, w_rows)
    st = status()
    got = mt.gemm_fp8_block128(dev(a), dev(sa), dev(w), dev(sw), dev_status=st)
    assert st.item() == 0
    check_product(got, a, sa, w, sw, w_rows)


@pytest.mark.parametrize("M,N,K", [(0, 128, 256), (4, 0, 256), (5, 130, 0), (0, 0, 0)])
def test_product_empty(mt, M, N, K):
    a, sa, w, sw = product_case(0, M, N, K, 1)
    got = mt.gemm_fp8_block128(dev(a), dev(sa), dev(w), dev(sw))
    assert got.shape == (M, N) and not got.float().any()


@pytest.mark.parametrize("M,N,K", [(5, 130, 256), (70, 77, 1920), (300, 385, 384)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_product_strided_output_leaves_the_rest(mt, M, N, K, out):
    a, sa, w, sw = product_case(3, M, N, K, 128)
    buf = torch.full((M + 2, N + 5), 7.0, dtype=out, device="cuda")
    view = buf[1:M + 1, 3:N + 3]           # odd start and stride
    assert mt.gemm_fp8_block128(dev(a), dev(sa), dev(w), dev(sw), out=view) is view
    check_product(view, a, sa, w, sw, 128)
    keep = torch.ones_like(buf, dtype=torch.bool)
    keep[1:M + 1, 3:N + 3] = False
    assert (buf[keep] == 7).all()


@pytest.mark.parametrize("M,N,K", [(7, 300, 512), (200, 129, 384), (300, 130, 256)])
def test_product_bad_values_stay_in_their_row_and_column(mt, M, N, K):
    a, sa, w, sw = product_case(4, M, N, K, 1)
    ref = mt.gemm_fp8_block128(dev(a), dev(sa), dev(w), dev(sw), out_dtype=torch.float32)
    a[2, 130], w[77, 3] = 0x7F, 0xFF
    sa[5, 0], sw[126, 1] = np.inf, np.nan
    got = mt.gemm_fp8_block128(dev(a), dev(sa), dev(w), dev(sw), out_dtype=torch.float32)
    hit = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    hit[[2, 5]] = True
    hit[:, [77, 126]] = True
    assert torch.equal(got[~hit], ref[~hit])
    assert torch.isnan(got[2]).all() and torch.isnan(got[:, 77]).all() and torch.isnan(got[:, 126]).all()
    assert not torch.isfinite(got[5]).any()


def test_product_extreme_and_zero_scales(mt):
    a, sa, w, sw = product_case(5, 9, 140, 512, 1)
    sa[:, 1] = 0
    sa[3], sw[3] = 1e-20, 1e18
    sa[4, 2] = -1.5
    got = mt.gemm_fp8_block128(dev(a), dev(sa), dev(w), dev(sw), out_dtype=torch.float32)
    check_product(got, a, sa, w, sw, 1)


def test_product_repeats_bit_for_bit(mt):
    for M, N, K in ((1, 576, 6144), (64, 640, 2048), (300, 700, 1024)):
        a, sa, w, sw = [dev(x) for x in product_case(6, M, N, K, 128)]
        ref = mt.gemm_fp8_block128(a, sa, w, sw, out_dtype=torch.float32)
        for _ in range(5):
            assert torch.equal(mt.gemm_fp8_block128(a, sa, w, sw, out_dtype=torch.float32), ref)


def test_product_of_a_quantized_weight(mt):
    """The quantizer's codes and scales go in as they come out."""
    rng = np.random.default_rng(8)
    x, wt = rng.normal(size=(6, 640)).astype(np.float32), rng.normal(size=(200, 640)).astype(np.float32)
    a, sa = mt.quantize_fp8_block128(dev(x))
    w, sw = mt.quantize_fp8_block128(dev(wt))
    got = mt.gemm_fp8_block128(a, sa, w, sw, out_dtype=torch.float32)
    check_product(got, *[t.cpu().numpy() for t in (a, sa, w, sw)], 1)
    rel = np.linalg.norm(got.cpu().numpy() - x @ wt.T) / np.linalg.norm(x @ wt.T)
    assert rel < 2 * 2.0 ** -4      # each factor is rounded by at most 2^-4 of its value


def test_product_on_another_stream_and_in_a_graph(mt):
    a, sa, w, sw = product_case(9, 64, 512, 1024, 128)
    t = [dev(x) for x in (a, sa, w, sw)]
    outs = [torch.empty(64, 512, device="cuda") for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for s, o in zip(streams, outs):            # two calls at once
        mt.gemm_fp8_block128(*t, out=o, stream=s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mt.gemm_fp8_block128(*t, out=outs[2])
    outs[2].zero_()
    g.replay()
    torch.cuda.synchronize()
    check_product(outs[0], a, sa, w, sw, 128)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    a2 = codes(np.random.default_rng(10), 64, 1024)
    t[0].copy_(dev(a2))
    g.replay()
    torch.cuda.synchronize()
    check_product(outs[2], a2, sa, w, sw, 128)


def test_product_binding_refusals(mt):
    a, sa, w, sw = [dev(x) for x in product_case(11, 4, 130, 256, 1)]
    for bad in ((a[:, ::2], sa, w, sw), (a, sa[:2].contiguous(), w, sw), (a, sa, w, sw[:3].contiguous()),
                (a[:, :200].contiguous(), sa, w[:, :200].contiguous(), sw)):
        with pytest.raises(ValueError):
            mt.gemm_fp8_block128(*bad)
    with pytest.raises(TypeError):
        mt.gemm_fp8_block128(a.float(), sa, w, sw)
    with pytest.raises(TypeError):
        mt.gemm_fp8_block128(a, sa, w, sw, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        mt.gemm_fp8_block128(a, sa, w, sw, out=torch.empty(4, 131, device="cuda"))
    with pytest.raises(ValueError):
        mt.gemm_fp8_block128(a, sa, w, sw, out=torch.empty(130, 4, device="cuda").t())
    with pytest.raises(ValueError):
        mt.gemm_fp8_block128(a, sa, w, sw, out=torch.empty(1, 130, device="cuda").expand(4, 130))


# ----------------------------------------------------------------------------- token table

def table_case(seed, lens, V, rows=None, n_rows=None):
    rng = np.random.default_rng(seed)
    tok = (rng.integers(0, V, sum(lens)) * rng.integers(0, 2, sum(lens))).astype(np.int64)    # token 0 is hot
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.uint32)
    n_prompt = np.array([rng.integers(0, n + 1) for n in lens], dtype=np.int64)
    before = rng.integers(-32768, 32768, (n_rows or len(lens), ologits.token_counts_ld(V))).astype(np.int16)
    return tok, off, n_prompt, before


@pytest.mark.parametrize("lens,V", [([1], 1), ([0, 1, 2], 7), ([5, 0, 300, 0], 1000), ([4097, 33], 8),
                                    ([20000, 1, 7000], 50001), ([3000] * 9, 154880), ([40000, 10], 262147)])
@pytest.mark.parametrize("prompt", [True, False])
def test_table_build(mt, lens, V, prompt):
    tok, off, n_prompt, before = table_case(len(lens) + V, lens, V)
    st = status()
    table = dev(before)
    got = mt.token_counts_build(dev(tok), u32(off), V, n_prompt=dev(n_prompt) if prompt else None, counts=table,
                                dev_status=st)
    assert got is table and st.item() == 0
    want = ologits.token_counts_build(before, tok, off, V, n_prompt if prompt else None)
    assert np.array_equal(table.cpu().numpy(), want)


def test_table_prompt_lengths_past_the_tokens(mt):
    """Prompt lengths outside 0 .. the request's tokens are cut to that range."""
    V, toks = 50, np.arange(40, dtype=np.int64)
    off = np.array([0, 7, 7, 20, 40], np.uint32)
    big = np.iinfo(np.int64)
    want = ologits.token_counts_build(np.zeros((4, 56), np.int16), toks, off, V, [0, 0, 13, 20])
    got = mt.token_counts_build(dev(toks), u32(off), V, n_prompt=dev(np.array([big.min, -1, 13, big.max], np.int64)))
    assert np.array_equal(got.cpu().numpy(), want)


def test_table_build_saturates(mt):
    V = 40
    tok = np.array([3] * 40000 + [4] * 32767 + [5] * 32766 + [2] * 7, np.int64)
    off = np.array([0, len(tok)])
    got = mt.token_counts_build(dev(tok), u32(off), V, n_prompt=dev(np.array([2])))
    want = ologits.token_counts_build(np.zeros((1, 40), np.int16), tok, off, V, [2])
    assert got[0, 3].item() == -1 and np.array_equal(got.cpu().numpy(), want)


def test_table_rows_and_bad_values(mt):
    from mtp_speculative_decode_gb300 import _native as N
    V = 100
    lens = [50, 60, 70, 80, 90]
    tok, off, n_prompt, before = table_case(5, lens, V, n_rows=6)

    def build(rows, tok=tok, off=off):
        st, table = status(), dev(before)
        mt.token_counts_build(dev(tok), u32(off), V, n_prompt=dev(n_prompt), counts=table,
                              count_rows=dev(np.array(rows, np.int32)), dev_status=st)
        return table.cpu().numpy(), st.item()

    got, st = build([5, -1, 0, 2, 3])
    assert st == 0 and np.array_equal(got, ologits.token_counts_build(before, tok, off, V, n_prompt, [5, -1, 0, 2, 3]))
    got, st = build([5, 6, -7, 2, 3])
    assert st == N.STATUS_ROW_RANGE
    assert np.array_equal(got, ologits.token_counts_build(before, tok, off, V, n_prompt, [5, 6, -7, 2, 3]))
    got, st = build([5, 4, 5, 2, 4])                  # the same row twice: the first request keeps it
    assert st == N.STATUS_INDEX_RANGE
    assert np.array_equal(got, ologits.token_counts_build(before, tok, off, V, n_prompt, [5, 4, 5, 2, 4]))
    bad = tok.copy()
    bad[[3, 77, 200]] = [-1, V, 1 << 40]
    got, st = build([0, 1, 2, 3, 4], tok=bad)
    assert st == N.STATUS_INDEX_RANGE
    assert np.array_equal(got, ologits.token_counts_build(before, bad, off, V, n_prompt, [0, 1, 2, 3, 4]))
    far = off.copy()
    far[-1] += 1000                                   # past the tokens
    got, st = build([0, 1, 2, 3, 4], off=far)
    assert st == N.STATUS_ROW_RANGE
    assert np.array_equal(got, ologits.token_counts_build(before, tok, off, V, n_prompt, [0, 1, 2, 3, 4]))
    back = off.copy()
    back[2] = 10                                      # segment 1 ends before it starts
    got, st = build([0, 1, 2, 3, 4], off=back)
    assert st == 0
    assert np.array_equal(got, ologits.token_counts_build(before, tok, back, V, n_prompt, [0, 1, 2, 3, 4]))


@pytest.mark.parametrize("B,K,V", [(1, 0, 9), (1, 5, 9), (40, 3, 11), (300, 7, 1001)])
def test_table_accept(mt, B, K, V):
    from mtp_speculative_decode_gb300 import _native as N
    rng = np.random.default_rng(B + K)
    before = rng.integers(-32768, 32768, (B, ologits.token_counts_ld(V))).astype(np.int16)
    before[:, ::3] |= 0x7FFF                           # at the limit
    draft = rng.integers(0, V, (B, K)).astype(np.int64)
    n_acc = rng.integers(-1, K + 2, B).astype(np.int32)
    nxt = rng.integers(0, V, B).astype(np.int64)
    nxt[0] = -1                                        # the greedy token of an empty row
    st, table = status(), dev(before)
    mt.token_counts_accept(table, V, dev(draft) if K else None, dev(n_acc) if K else None, dev(nxt), dev_status=st)
    assert st.item() == N.STATUS_INDEX_RANGE
    assert np.array_equal(table.cpu().numpy(), ologits.token_counts_accept(before, V, draft if K else None, n_acc, nxt))
    rows = rng.permutation(B).astype(np.int32)
    rows[B // 2] = rows[0]                             # two requests that share a row both count
    table = dev(before)
    mt.token_counts_accept(table, V, dev(draft), dev(n_acc), dev(nxt), count_rows=dev(rows))
    assert np.array_equal(table.cpu().numpy(), ologits.token_counts_accept(before, V, draft, n_acc, nxt, rows))


# ----------------------------------------------------------------------------- logits

class Case:
    """Random rows with the given parts switched on."""

    def __init__(self, seed, B, K, V, dtype=torch.float32, counts=False, pen=False, bias=0, mask=False, temp=False,
                 rows_per=None):
        rng = np.random.default_rng(seed)
        self.B, self.K, self.V = B, K, V
        n = rows_per if rows_per is not None else [K + 1] * B
        self.off = np.concatenate([[0], np.cumsum(n)]).astype(np.uint32)
        self.R = R = int(self.off[-1])
        self.logits = torch.from_numpy((rng.normal(size=(R, V)) * 3).astype(np.float32)).to(dtype)
        self.draft = rng.integers(0, V, (B, K)).astype(np.int64) if K else None
        self.counts = None
        if counts:
            c = rng.integers(0, 4, (B, ologits.token_counts_ld(V))) * (rng.random((B, ologits.token_counts_ld(V))) < 0.1)
            self.counts = (c - 32768 * (rng.random(c.shape) < 0.1)).astype(np.int16)
        f32 = lambda lo, hi: rng.uniform(lo, hi, B).astype(np.float32)  # noqa: E731
        self.rep, self.freq, self.pres = (f32(0.8, 1.6), f32(-0.2, 0.7), f32(0, 1)) if pen else (None, None, None)
        self.temp = f32(0.3, 1.5) if temp else None
        if temp:
            self.temp[::3] = 0
        self.bias = None
        if bias:
            nb = rng.integers(0, bias + 1, B)
            nb[0] = bias
            self.bias = (np.concatenate([[0], np.cumsum(nb)]).astype(np.uint32),
                         rng.integers(0, V, nb.sum()).astype(np.int32),     # repeated ids among them
                         rng.uniform(-8, 8, nb.sum()).astype(np.float32))
        self.mask = self.mask_rows = None
        if mask:
            words = -(-V // 32)
            self.mask = rng.integers(-2 ** 31, 2 ** 31, (max(R // 2, 1) + 1, words)).astype(np.int32)
            self.mask[0] = 0
            self.mask[0, words // 2] = 1                # one token left
            self.mask_rows = rng.integers(-1, len(self.mask), R).astype(np.int32)
            if R:
                self.mask_rows[0] = 0

    def call(self, mt, **kw):
        a = dict(draft=None if self.draft is None else dev(self.draft),
                 counts=None if self.counts is None else dev(self.counts), repetition=self.rep, frequency=self.freq,
                 presence=self.pres, temperature=self.temp)
        for k in ("repetition", "frequency", "presence", "temperature"):
            a[k] = None if a[k] is None else dev(a[k])
        if self.bias is not None:
            a.update(bias_offsets=u32(self.bias[0]), bias_tokens=dev(self.bias[1]), bias_values=dev(self.bias[2]))
        if self.mask is not None:
            a.update(bitmask=dev(self.mask), mask_rows=dev(self.mask_rows))
        a.update(kw)
        return mt.process_logits(a.pop("logits", None) if "logits" in a else self.logits.cuda(), u32(self.off), **a)

    def oracle(self, r):
        """Row r: (processed, argmax, probs, error bound of processed)."""
        b = int(np.searchsorted(self.off, r, side="right")) - 1
        i = r - int(self.off[b])
        g = lambda x, d: d if x is None else float(x[b])  # noqa: E731
        word = None if self.counts is None else self.counts[b]
        drafts = [] if self.draft is None else [int(t) for t in self.draft[b, :min(i, self.K)]]
        biases = []
        if self.bias is not None:
            lo, hi = int(self.bias[0][b]), int(self.bias[0][b + 1])
            biases = list(zip(self.bias[1][lo:hi].tolist(), self.bias[2][lo:hi].astype(float).tolist()))
        m = -1 if self.mask is None else int(self.mask_rows[r])
        x = self.logits[r].double().numpy()
        y, arg, p = ologits.process_row(x, word, drafts, g(self.rep, 1.0), g(self.freq, 0.0), g(self.pres, 0.0), biases,
                                        self.mask[m] if m >= 0 else None, g(self.temp, 1.0))
        rep = g(self.rep, 1.0)
        n = np.zeros(self.V) if word is None else (word[:self.V] & 32767).astype(float)
        S = np.abs(x) * max(rep, 1 / rep)
        for t in drafts:
            n[t] += 1
        # nothing is computed on a token that was never seen and has no bias
        k = np.where((n > 0) | (False if word is None else word[:self.V] < 0), 5.0, 0.0)
        S = S + abs(g(self.freq, 0.0)) * n + abs(g(self.pres, 0.0))
        for t, v in biases:
            if 0 <= t < self.V:
                S[t] += abs(v)
                k[t] += 1
        return y, arg, p, k * 2.0 ** -24 * S, g(self.temp, 1.0)

    def check(self, argmax=None, probs=None, processed=None, rows=None):
        for r in range(self.R) if rows is None else rows:
            y, arg, p, tol, temp = self.oracle(r)
            fin = np.isfinite(y)
            if processed is not None:
                got = processed[r].double().cpu().numpy()
                assert np.array_equal(got[~fin], y[~fin]) and (np.abs(got[fin] - y[fin]) <= tol[fin]).all()
            if argmax is not None:
                assert int(argmax[r]) == arg
            if probs is not None:
                got = probs[r].double().cpu().numpy()
                if arg < 0 or not temp > 0:
                    assert np.array_equal(got, p)
                    continue
                # where p is 0 in float64 the exponent is below -745, far below float32's range too
                d = np.where(p > 0, y - y[arg], 0.0)
                rel = (tol + tol[arg]) / temp + 2.0 ** -22 * np.abs(d / temp)
                rel = np.where(p > 0, np.expm1(rel + rel[arg]) + 2.0 ** -22 + 513 * 2.0 ** -23, 0.0)
                # the sum's own error is at most the weighted mean of the terms'
                rel = rel + float((p * rel).sum())
                assert (np.abs(got - p) <= rel * p + 2.0 ** -126).all()


ALL = dict(counts=True, pen=True, bias=9, mask=True, temp=True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,K,V,parts", [
    (1, 0, 1, {}), (3, 0, 7, dict(temp=True)), (2, 3, 33, dict(pen=True)), (4, 2, 64, dict(mask=True)),
    (3, 1, 100, dict(bias=30)), (2, 4, 127, dict(counts=True, pen=True)), (5, 5, 1000, ALL), (3, 2, 2049, ALL),
    (2, 1, 8200, ALL), (1, 2, 50001, ALL), (1, 1, 154880, ALL)])
def test_logits(mt, B, K, V, parts, dtype):
    c = Case(B * 31 + V, B, K, V, dtype, **parts)
    st = status()
    probs = torch.full((c.R, V), 9.0, device="cuda")
    out = torch.full((c.R, V), 9.0, device="cuda")
    argmax = torch.full((c.R,), 9, dtype=torch.int64, device="cuda")
    assert c.call(mt, argmax=argmax, probs=probs, out_logits=out, dev_status=st) is argmax
    c.check(argmax, probs, out)
    masked_out = any(c.oracle(r)[1] < 0 for r in range(c.R)) if V < 2000 else False
    if V < 2000:
        assert st.item() == (16 if masked_out else 0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,K,V", [(400, 5, 701), (150, 5, 20000), (90, 7, 40003)])
def test_logits_many_rows_per_cluster(mt, B, K, V, dtype):
    """More rows than run at once, ragged requests (empty ones too): rows of one and of several requests in a run."""
    rng = np.random.default_rng(B + V)
    n = rng.integers(0, K + 3, B)
    n[1] = 0
    c = Case(B, B, K, V, dtype, rows_per=n, **{**ALL, "bias": 40})
    probs, out = torch.full((c.R, V), 9.0, device="cuda"), torch.full((c.R, V), 9.0, device="cuda")
    argmax = c.call(mt, argmax=torch.empty(c.R, dtype=torch.int64, device="cuda"), probs=probs, out_logits=out)
    rows = rng.permutation(c.R)[:150]
    c.check(argmax, probs, out, rows)
    again = torch.empty_like(out)
    assert torch.equal(c.call(mt), argmax)             # the greedy token alone
    c.call(mt, out_logits=again)
    assert torch.equal(again.nan_to_num(nan=1.5), out.nan_to_num(nan=1.5))
    other = torch.empty_like(probs)
    c.call(mt, probs=other)
    assert torch.equal(other, probs)


@pytest.mark.parametrize("V", [262144, 393216])
def test_logits_largest_vocabularies(mt, V):
    c = Case(V, 1, 0, V, torch.float32, counts=True, pen=True, bias=5)
    probs = torch.empty(1, V, device="cuda")
    am = c.call(mt, probs=probs, argmax=torch.empty(1, dtype=torch.int64, device="cuda"))
    c.check(am, probs)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,n,tokens", [(5000, 300, 290), (5001, 300, 235), (5001, 300, 100), (1001, 700, 40), (64, 700, 1)])
def test_logits_tokens_with_several_entries(mt, V, n, tokens, dtype):
    """Biases of a token that other biases and drafts have too, few and many of them, are added in list order."""
    rng = np.random.default_rng(n + tokens)
    c = Case(V + n, 3, 5, V, dtype, counts=True, pen=True, bias=n, temp=True)
    some = rng.permutation(V)[:tokens].astype(np.int32)
    c.bias[1][:] = some[rng.integers(0, tokens, len(c.bias[1]))]
    c.bias[1][:tokens] = some
    c.draft[:] = some[rng.integers(0, tokens, c.draft.shape)]
    c.draft[0, 3] = c.draft[0, 1]
    argmax = torch.empty(c.R, dtype=torch.int64, device="cuda")
    probs, out = torch.empty(c.R, V, device="cuda"), torch.empty(c.R, V, device="cuda")
    for _ in range(2):                                 # the same bits again
        before = out.clone()
        c.call(mt, argmax=argmax, probs=probs, out_logits=out)
        c.check(argmax, probs, out)
    assert torch.equal(before, out)
    c.check(c.call(mt))                                # nothing kept but the greedy token


def test_logits_argmax_only_and_default(mt):
    c = Case(1, 4, 3, 3000, torch.bfloat16, **ALL)
    c.check(c.call(mt))


def test_logits_outputs_alone(mt):
    c = Case(2, 3, 2, 1500, torch.float32, **ALL)
    probs = torch.empty(c.R, 1500, device="cuda")
    assert c.call(mt, probs=probs) is None
    out = torch.empty(c.R, 1500, device="cuda")
    c.call(mt, out_logits=out)
    c.check(None, probs, out)


def test_logits_in_place_and_strided(mt):
    V = 1003
    c = Case(3, 3, 2, V, torch.float32, **ALL)
    buf = torch.full((c.R, V + 9), 5.0, device="cuda")
    buf[:, 2:V + 2] = c.logits.cuda()
    x = buf[:, 2:V + 2]
    pbuf = torch.full((c.R, V + 3), 6.0, device="cuda")
    am = torch.empty(c.R, dtype=torch.int64, device="cuda")
    c.call(mt, logits=x, out_logits=x, probs=pbuf[:, 1:V + 1], argmax=am)
    c.check(am, pbuf[:, 1:V + 1], x)
    assert (buf[:, :2] == 5).all() and (buf[:, V + 2:] == 5).all()
    assert (pbuf[:, :1] == 6).all() and (pbuf[:, V + 1:] == 6).all()


def test_logits_ragged_rows_and_padded_batch(mt):
    """Rows behind the last request are left as they were; requests may have no row or more rows than drafts."""
    V = 500
    c = Case(4, 5, 2, V, torch.float32, counts=True, pen=True, rows_per=[1, 0, 3, 6, 2])
    pad = 4
    x = torch.cat([c.logits, torch.zeros(pad, V)]).cuda()
    am = torch.full((c.R + pad,), 77, dtype=torch.int64, device="cuda")
    probs = torch.full((c.R + pad, V), 3.0, device="cuda")
    out = torch.full((c.R + pad, V), 4.0, device="cuda")
    c.call(mt, logits=x, argmax=am, probs=probs, out_logits=out)
    c.check(am, probs, out)
    assert (am[c.R:] == 77).all() and (probs[c.R:] == 3).all() and (out[c.R:] == 4).all()


@pytest.mark.parametrize("V", [40, 5000, 154880])
def test_logits_edges(mt, V):
    """Rows whose mask leaves nothing, the lowest value, infinities and NaN in masked and in open places, ties."""
    inf, nan, low = math.inf, math.nan, float(np.finfo(np.float32).min)
    x = torch.zeros(9, V)
    x[0] = nan                                   # everything masked
    x[1] = inf
    x[1, V - 3] = 1.0                            # only V-3 allowed
    x[2] = low
    x[3, 5], x[3, V - 1] = inf, inf
    x[4, 7], x[4, V - 2] = nan, nan
    x[5, V // 2], x[5, V // 2 + 9] = 4.0, 4.0    # a tie
    x[6] = -inf
    x[7] = low
    x[7, 11] = -low
    x[8] = -0.0
    x[8, 3] = 0.0                                # equal zeros: the lowest position
    words = -(-V // 32)
    mask = np.zeros((2, words), np.uint32)
    mask[1, (V - 3) // 32] |= np.uint32(1 << ((V - 3) % 32))
    if V % 32:
        mask[0, -1] = np.uint32((0xFFFFFFFF << (V % 32)) & 0xFFFFFFFF)     # bits past the vocabulary are ignored
    st = status()
    am = torch.empty(9, dtype=torch.int64, device="cuda")
    probs, out = torch.empty(9, V, device="cuda"), torch.empty(9, V, device="cuda")
    mt.process_logits(x.cuda(), u32(np.arange(10)), argmax=am, probs=probs, out_logits=out,
                      bitmask=dev(mask.view(np.int32)), mask_rows=dev(np.array([0, 1] + [-1] * 7, np.int32)), dev_status=st)
    assert st.item() == 16
    assert am.tolist() == [-1, V - 3, 0, 5, 7, V // 2, -1, 11, 0]
    assert not probs[0].any() and not probs[6].any() and (out[0] == -inf).all()
    assert probs[1].sum() == 1 and probs[1, V - 3] == 1 and out[1, V - 3] == 1
    assert torch.allclose(probs[2], torch.full((V,), 1.0 / V, device="cuda"), rtol=1e-5)
    assert probs[3, 5] == 0.5 and probs[3, V - 1] == 0.5 and probs[3].sum() == 1
    assert torch.isnan(probs[4]).all()
    assert probs[5, V // 2] == probs[5, V // 2 + 9] > probs[5, 0]
    assert probs[7, 11] == 1 and probs[7].sum() == 1
    assert torch.allclose(probs[8], torch.full((V,), 1.0 / V, device="cuda"), rtol=1e-5)
    t0 = torch.zeros(9, device="cuda")
    mt.process_logits(x.cuda(), u32(np.arange(10)), probs=probs, temperature=t0)
    assert probs[4].sum() == 1 and probs[4, 7] == 1 and probs[5, V // 2] == 1 and not probs[6].any()


def test_logits_temperatures(mt):
    V = 300
    c = Case(6, 6, 0, V, torch.float32)
    c.temp = np.array([1e-30, 1e-3, 1.0, 50.0, 1e30, 3e38], np.float32)
    probs = torch.empty(6, V, device="cuda")
    c.call(mt, probs=probs)
    c.check(None, probs)
    assert torch.isfinite(probs).all()
    for t in (-1.0, float("nan"), float("-inf"), -0.0):
        c.temp = np.full(6, t, np.float32)
        am = torch.empty(6, dtype=torch.int64, device="cuda")
        c.call(mt, probs=probs, argmax=am)
        assert torch.equal(probs, torch.nn.functional.one_hot(am, V).float())


def test_logits_bad_device_values(mt):
    from mtp_speculative_decode_gb300 import _native as N
    V, B, K = 200, 3, 2
    base = Case(7, B, K, V, torch.float32, **ALL)

    def run(change, **kw):
        c = Case(7, B, K, V, torch.float32, **ALL)
        c.mask_rows[:] = -1
        change(c)
        st = status()
        out = torch.empty(c.R, V, device="cuda")
        c.call(mt, out_logits=out, dev_status=st, **kw)
        return c, out, st.item()

    def ids(c):
        c.draft[1] = [-5, V]
        c.bias[1][0], c.bias[1][3] = -1, V

    c, out, st = run(ids)
    assert st == N.STATUS_INDEX_RANGE
    c.draft = np.where((c.draft < 0) | (c.draft >= V), 0, c.draft)   # compare the rows without those drafts
    c.check(None, None, out, rows=[r for r in range(c.R) if r // (K + 1) != 1])

    def offs(c):
        c.bias[0][-1] += 100
    c, out, st = run(offs)
    assert st == N.STATUS_INDEX_RANGE
    c.bias[0][-1] -= 100
    c.check(None, None, out)

    def masks(c):
        c.mask_rows[2], c.mask_rows[4] = len(c.mask), -2
    c, out, st = run(masks)
    assert st == N.STATUS_ROW_RANGE
    c.mask_rows[:] = -1
    c.check(None, None, out)
    c, out, st = run(lambda c: None, count_rows=dev(np.array([2, 3, -1], np.int32)))
    assert st == N.STATUS_ROW_RANGE
    c.counts = np.stack([base.counts[2], base.counts[0] * 0, base.counts[0] * 0])
    c.check(None, None, out)


def test_logits_offsets_past_the_rows(mt):
    """Offsets that pass the rows of the arrays are cut to them and flagged; offsets that fall stay inside them."""
    from mtp_speculative_decode_gb300 import _native as N
    c = Case(17, 4, 2, 300, torch.float32, counts=True, pen=True, bias=5)
    want = torch.empty(c.R, 300, device="cuda")
    c.call(mt, out_logits=want)
    off = c.off.copy()
    off[-1] += 7
    st, out = status(), torch.full((c.R + 2, 300), 9.0, device="cuda")
    args = dict(draft=dev(c.draft), counts=dev(c.counts), repetition=dev(c.rep), frequency=dev(c.freq), presence=dev(c.pres),
                bias_offsets=u32(c.bias[0]), bias_tokens=dev(c.bias[1]), bias_values=dev(c.bias[2]))
    mt.process_logits(c.logits.cuda(), u32(off), out_logits=out[:c.R], dev_status=st, **args)
    assert st.item() == N.STATUS_ROW_RANGE and torch.equal(out[:c.R], want) and (out[c.R:] == 9).all()
    off[:] = [0, 9, 3, 6, 12]
    out.fill_(9.0)
    mt.process_logits(c.logits.cuda(), u32(off), out_logits=out[:c.R], dev_status=status(), **args)
    assert (out[c.R:] == 9).all()


def test_logits_and_table_on_two_streams_and_in_two_graphs(mt):
    V = 30011
    cases = [Case(90 + i, 20, 3, V, (torch.float32, torch.bfloat16)[i], **{**ALL, "bias": 20}) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    off, tokens = u32(np.arange(0, 2001, 100)), dev(np.random.default_rng(3).integers(0, V, 2000).astype(np.int64))
    ld = mt.token_counts_ld(V)
    tables = [torch.zeros(20, ld, dtype=torch.int16, device="cuda") for _ in range(2)]
    argmax = [torch.zeros(c.R, dtype=torch.int64, device="cuda") for c in cases]
    probs = [torch.zeros(c.R, V, device="cuda") for c in cases]
    inputs = []
    for c in cases:
        a = dict(draft=dev(c.draft), repetition=dev(c.rep), frequency=dev(c.freq), presence=dev(c.pres),
                 temperature=dev(c.temp), bias_offsets=u32(c.bias[0]), bias_tokens=dev(c.bias[1]),
                 bias_values=dev(c.bias[2]), bitmask=dev(c.mask), mask_rows=dev(c.mask_rows))
        inputs.append((c.logits.cuda(), u32(c.off), a))
        c.counts = ologits.token_counts_build(np.zeros((20, ld), np.int16), tokens.cpu().numpy(), off.cpu().numpy(), V)
    torch.cuda.synchronize()

    def step(i, stream=None):
        mt.token_counts_build(tokens, off, V, counts=tables[i], stream=stream)
        x, o, a = inputs[i]
        mt.process_logits(x, o, counts=tables[i], argmax=argmax[i], probs=probs[i], stream=stream, **a)

    def check():
        torch.cuda.synchronize()
        for i, c in enumerate(cases):
            c.check(argmax[i], probs[i], rows=range(0, c.R, 9))
            tables[i].zero_(), argmax[i].zero_(), probs[i].zero_()
        torch.cuda.synchronize()

    for _ in range(3):
        for i, s in enumerate(streams):
            step(i, s)
    check()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i, g in enumerate(graphs):
        with torch.cuda.graph(g):
            step(i)
    assert not any(t.any() for t in tables)            # captured, not run
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    check()


def test_logits_mask_by_row_and_empty_batch(mt):
    V = 70
    c = Case(8, 2, 1, V)
    c.mask = np.random.default_rng(0).integers(-2 ** 31, 2 ** 31, (4, 3)).astype(np.int32)
    c.mask_rows = np.arange(4, dtype=np.int32)
    probs = torch.empty(4, V, device="cuda")
    mt.process_logits(c.logits.cuda(), u32(c.off), draft=dev(c.draft), bitmask=dev(c.mask), probs=probs)
    c.check(None, probs)
    e = mt.process_logits(torch.empty(0, V, device="cuda"), u32([0, 0]))
    assert e.shape == (0,)


def test_logits_binding_refusals(mt):
    x = torch.zeros(4, 64, device="cuda")
    off = u32([0, 2, 4])
    f = torch.ones(2, device="cuda")
    bad = [dict(draft=torch.zeros(3, 1, dtype=torch.int64, device="cuda")), dict(repetition=torch.ones(3, device="cuda")),
           dict(counts=torch.zeros(2, 60, dtype=torch.int16, device="cuda")),
           dict(counts=torch.zeros(1, 64, dtype=torch.int16, device="cuda")),
           dict(count_rows=torch.zeros(2, dtype=torch.int32, device="cuda")), dict(bias_offsets=u32([0, 0, 0])),
           dict(bitmask=torch.zeros(4, 3, dtype=torch.int32, device="cuda")),
           dict(bitmask=torch.zeros(4, 2, dtype=torch.int32, device="cuda"),
                mask_rows=torch.zeros(3, dtype=torch.int32, device="cuda")),
           dict(argmax=torch.zeros(3, dtype=torch.int64, device="cuda")), dict(probs=torch.zeros(4, 65, device="cuda")),
           dict(probs=torch.zeros(64, 4, device="cuda").t()), dict(probs=x[:1].expand(4, 64)), dict(temperature=f.cpu())]
    for kw in bad:
        with pytest.raises(ValueError):
            mt.process_logits(x, off, **kw)
    with pytest.raises(TypeError):
        mt.process_logits(x.half(), off)
    with pytest.raises(TypeError):
        mt.process_logits(x, off, out_logits=x.bfloat16())
    from mtp_speculative_decode_gb300._native import MtpsdError
    with pytest.raises(MtpsdError):                     # fewer masks than rows
        mt.process_logits(x, off, bitmask=torch.zeros(3, 2, dtype=torch.int32, device="cuda"))
    with pytest.raises(MtpsdError):
        mt.process_logits(torch.zeros(1, 393217, device="cuda"), u32([0, 1]))


# ----------------------------------------------------------------------------- together

@pytest.mark.parametrize("sampling", [False, True])
def test_verify_head(mt, sampling):
    """Hidden states to the advanced token table, eagerly and as a replayed graph, against the oracle chain."""
    from mtp_speculative_decode_gb300.pipeline import VerifyHead
    rng = np.random.default_rng(21)
    B, K, V, D = 5, 3, 777, 256
    R = B * (K + 1)
    wt = rng.normal(size=(V, D)).astype(np.float32)
    w, sw = mt.quantize_fp8_block128(dev(wt))
    c = Case(22, B, K, V, torch.float32, **{**ALL, "mask": False})
    c.temp = rng.uniform(0.5, 1.5, B).astype(np.float32)
    params = dict(repetition=dev(c.rep), frequency=dev(c.freq), presence=dev(c.pres), temperature=dev(c.temp),
                  bias_offsets=u32(c.bias[0]), bias_tokens=dev(c.bias[1]), bias_values=dev(c.bias[2]))
    extra = {}
    if sampling:
        q = rng.dirichlet(np.ones(V) * 0.1, (B, K)).astype(np.float32)
        ua, us = rng.random((B, K)).astype(np.float32) * 0.2, rng.random(B).astype(np.float32)
        extra = dict(draft_probs=dev(q), u_accept=dev(ua), u_sample=dev(us))
    head = VerifyHead(w, sw, B, K, counts=dev(c.counts), params=params, logits_dtype=torch.float32, **extra)
    hidden = rng.normal(size=(R, D)).astype(np.float32)
    head.hidden.copy_(dev(hidden))

    def run_and_check(step):
        # drafts that follow the greedy chain part of the way, so that some are accepted
        before = head.counts.clone()
        probe = torch.empty(R, dtype=torch.int64, device="cuda")
        draft = torch.zeros(B, K, dtype=torch.int64, device="cuda")
        head.project()
        for j in range(K):
            mt.process_logits(head.logits, head.row_offsets, draft=draft, counts=before, argmax=probe, **params)
            draft[:, j] = probe.view(B, K + 1)[:, j]
        draft[1, 1], draft[2, 0] = (draft[1, 1] + 1) % V, (draft[2, 0] + 1) % V
        head.draft.copy_(draft)
        step()
        torch.cuda.synchronize()
        assert head.status.item() == 0
        a, sa = ofp8.quantize_block128(head.hidden.cpu().numpy())
        check_product(head.logits, a, sa, w.cpu().numpy(), sw.cpu().numpy(), 1)
        c.logits, c.draft, c.counts = head.logits.cpu(), draft.cpu().numpy(), before.cpu().numpy()
        probs = None if head.target_probs is None else head.target_probs.view(R, V)
        c.check(head.target_argmax.view(-1), probs)
        if sampling:
            n, t = oaccept.accept_stochastic(c.draft, q, head.target_probs.cpu().numpy(), ua, us)
        else:
            n, t = oaccept.accept_greedy(c.draft, head.target_argmax.cpu().numpy())
            assert n.tolist() == [3, 1, 0, 3, 3]
        assert np.array_equal(head.num_accepted.cpu().numpy(), n) and np.array_equal(head.next_tokens.cpu().numpy(), t)
        want = ologits.token_counts_accept(c.counts, V, c.draft, n, t)
        assert np.array_equal(head.counts.cpu().numpy(), want)

    run_and_check(head.step)
    before = head.counts.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        head.step()
    assert torch.equal(head.counts, before)              # captured, not run
    head.hidden.copy_(dev(rng.normal(size=(R, D)).astype(np.float32)))
    run_and_check(g.replay)
    assert head.launches_per_step() == 5
