"""The head's operators where a launch takes another path than its ordinary one: table builds whose CTAs go through
several blocks of 32768 tokens, token ids that are no 32-bit numbers inside a run of wide loads, prompts, long draft
chains, arrays past 2^31 elements, and the verify head with grammar masks, bf16 logits and without drafts.  Tolerances are
those of test_gpu_head.py."""
import numpy as np
import pytest
import torch

from oracle import accept as oaccept
from oracle import fp8 as ofp8
from oracle import logits as ologits
from test_gpu_head import ALL, Case, check_product, dev, mt, product_case, status, u32  # noqa: F401

pytestmark = pytest.mark.gpu

# one CTA goes through all tokens of a request where more CTAs than SMs would come of two parts: from 77 requests (152 SMs)
ONE_PART = 80


def long_request(seed, before, n, V):
    """ONE_PART short requests, but the one after `before` of three tokens each has n; its first half is nearly all one
    even id, with the odd neighbour (the other half of the same counter word) here and there."""
    rng = np.random.default_rng(seed)
    lens = [3] * before + [n] + [2] * (ONE_PART - before - 1)
    tok = rng.integers(0, V, sum(lens)).astype(np.int64)
    at = 3 * before
    hot = tok[at:at + n // 2]
    hot[:] = 6
    hot[rng.integers(0, n // 2, 700)] = 7
    return tok, lens, at


@pytest.mark.parametrize("prompt", [0, 32768, 40001, 70000, 149999, None])
@pytest.mark.parametrize("before", [40, 41])                       # an even and an odd first token: aligned pairs or not
def test_table_build_over_several_blocks(mt, before, prompt):  # noqa: F811
    """Counts pass 2 x 32767 before they are cut to the limit, the prompt ends in a later block or on a border."""
    V, n = 40, 150000
    tok, lens, at = long_request(before, before, n, V)
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.uint32)
    n_prompt = None
    if prompt is not None:
        n_prompt = np.array([k // 2 for k in lens], np.int64)
        n_prompt[before] = prompt
    st = status()
    got = mt.token_counts_build(dev(tok), u32(off), V, n_prompt=None if n_prompt is None else dev(n_prompt),
                                dev_status=st).cpu().numpy()
    want = ologits.token_counts_build(np.zeros((ONE_PART, 40), np.int16), tok, off, V, n_prompt)
    assert st.item() == 0 and np.array_equal(got, want)
    if prompt == 0:
        assert got[before, 6] == 32767 and 0 < got[before, 7] < 8000


@pytest.mark.parametrize("requests", [1, ONE_PART])                 # eight parts, one part
@pytest.mark.parametrize("prompt", [0, 50000, None])
@pytest.mark.parametrize("V", [40, 50001, 154880])
def test_table_build_ids_that_are_no_tokens(mt, requests, prompt, V):  # noqa: F811
    """Ids outside the vocabulary between good ones of the same wide load: negative ones, V, and ids whose lower 32 bits
    are a good token."""
    from mtp_speculative_decode_gb300 import _native as N
    rng = np.random.default_rng(V + requests)
    n = 100000
    lens = [n] + [2] * (requests - 1)
    tok = rng.integers(0, V, sum(lens)).astype(np.int64)
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.uint32)
    n_prompt = None if prompt is None else np.array([prompt] + [1] * (requests - 1), np.int64)

    def build(tok):
        st = status()
        got = mt.token_counts_build(dev(tok), u32(off), V, n_prompt=None if n_prompt is None else dev(n_prompt),
                                    dev_status=st).cpu().numpy()
        for b in {0, requests - 1}:
            want = ologits.token_counts_build(np.zeros((1, ologits.token_counts_ld(V)), np.int16), tok, off[b:b + 2], V,
                                              None if n_prompt is None else n_prompt[b:b + 1])
            assert np.array_equal(got[b], want[0])
        return st.item()

    assert build(tok) == 0
    for bad in (-1, V, 1 << 40, (1 << 32) + 3, -(1 << 32) + 5, np.iinfo(np.int64).min):
        t = tok.copy()
        t[rng.integers(0, n, 5)] = bad
        assert build(t) == N.STATUS_INDEX_RANGE, bad
        one = tok.copy()
        one[50000 + int(rng.integers(0, 40000))] = bad
        assert build(one) == N.STATUS_INDEX_RANGE, bad


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sampling", [False, True])
def test_verify_head_under_a_grammar(mt, sampling, dtype):  # noqa: F811
    """Hidden states to the advanced token table with masks for some rows, eagerly and as a replayed graph."""
    from mtp_speculative_decode_gb300.pipeline import VerifyHead
    rng = np.random.default_rng(31)
    B, K, V, D = 5, 3, 777, 256
    R = B * (K + 1)
    w, sw = mt.quantize_fp8_block128(dev(rng.normal(size=(V, D)).astype(np.float32)))
    c = Case(32, B, K, V, dtype, **ALL)
    c.mask[0] = rng.integers(-2 ** 31, 2 ** 31, c.mask.shape[1])     # no row without an open token
    c.mask_rows[2::5] = -1
    c.temp = rng.uniform(0.5, 1.5, B).astype(np.float32)
    params = dict(repetition=dev(c.rep), frequency=dev(c.freq), presence=dev(c.pres), temperature=dev(c.temp),
                  bias_offsets=u32(c.bias[0]), bias_tokens=dev(c.bias[1]), bias_values=dev(c.bias[2]), bitmask=dev(c.mask),
                  mask_rows=dev(c.mask_rows))
    extra = {}
    if sampling:
        q = rng.dirichlet(np.ones(V) * 0.1, (B, K)).astype(np.float32)
        ua, us = rng.random((B, K)).astype(np.float32) * 0.2, rng.random(B).astype(np.float32)
        extra = dict(draft_probs=dev(q), u_accept=dev(ua), u_sample=dev(us))
    head = VerifyHead(w, sw, B, K, counts=dev(c.counts), params=params, **extra,
                      **(dict(logits_dtype=dtype) if dtype != torch.bfloat16 else {}))
    assert head.logits.dtype == dtype
    head.hidden.copy_(dev(rng.normal(size=(R, D)).astype(np.float32)))

    def run_and_check(step):
        before = head.counts.clone()
        probe = torch.empty(R, dtype=torch.int64, device="cuda")
        draft = torch.zeros(B, K, dtype=torch.int64, device="cuda")
        head.project()
        for j in range(K):                               # drafts that follow the greedy chain part of the way
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
        c.check(head.target_argmax.view(-1), None if head.target_probs is None else head.target_probs.view(R, V))
        for r in range(R):                               # the greedy tokens are open
            m, t = int(c.mask_rows[r]), int(head.target_argmax.view(-1)[r])
            assert m < 0 or int(c.mask[m, t // 32]) >> (t % 32) & 1
        if sampling:
            n, t = oaccept.accept_stochastic(c.draft, q, head.target_probs.cpu().numpy(), ua, us)
        else:
            n, t = oaccept.accept_greedy(c.draft, head.target_argmax.cpu().numpy())
            assert n.tolist() == [3, 1, 0, 3, 3]
        assert np.array_equal(head.num_accepted.cpu().numpy(), n) and np.array_equal(head.next_tokens.cpu().numpy(), t)
        assert np.array_equal(head.counts.cpu().numpy(), ologits.token_counts_accept(c.counts, V, c.draft, n, t))

    run_and_check(head.step)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        head.step()
    head.hidden.copy_(dev(rng.normal(size=(R, D)).astype(np.float32)))
    run_and_check(g.replay)


@pytest.mark.parametrize("sampling", [False, True])
def test_verify_head_without_drafts(mt, sampling):  # noqa: F811
    """K = 0: one row per request, its token and nothing to accept."""
    from mtp_speculative_decode_gb300.pipeline import VerifyHead
    rng = np.random.default_rng(41)
    B, V, D = 7, 1003, 128
    w, sw = mt.quantize_fp8_block128(dev(rng.normal(size=(V, D)).astype(np.float32)))
    c = Case(42, B, 0, V, torch.float32, counts=True, pen=True)
    c.temp = rng.uniform(0.5, 1.5, B).astype(np.float32)
    params = dict(repetition=dev(c.rep), frequency=dev(c.freq), presence=dev(c.pres), temperature=dev(c.temp))
    us = rng.random(B).astype(np.float32)
    extra = dict(draft_probs=torch.empty(B, 0, V, device="cuda"), u_accept=torch.empty(B, 0, device="cuda"),
                 u_sample=dev(us)) if sampling else {}
    head = VerifyHead(w, sw, B, 0, counts=dev(c.counts), params=params, logits_dtype=torch.float32, **extra)
    head.hidden.copy_(dev(rng.normal(size=(B, D)).astype(np.float32)))
    head.step()
    torch.cuda.synchronize()
    c.logits = head.logits.cpu()
    c.check(head.target_argmax.view(-1), head.target_probs.view(B, V) if sampling else None)
    n, t = np.zeros(B, np.int32), head.target_argmax.view(-1).cpu().numpy()
    if sampling:
        n, t = oaccept.accept_stochastic(np.zeros((B, 0), np.int64), np.zeros((B, 0, V), np.float32),
                                         head.target_probs.cpu().numpy(), np.zeros((B, 0), np.float32), us)
    assert head.status.item() == 0 and np.array_equal(head.num_accepted.cpu().numpy(), n)
    assert np.array_equal(head.next_tokens.cpu().numpy(), t)
    assert np.array_equal(head.counts.cpu().numpy(), ologits.token_counts_accept(c.counts, V, None, n, t))


@pytest.mark.parametrize("w_rows", [1, 128])
@pytest.mark.parametrize("M,N,K", [(2048, 640, 384), (4099, 300, 256), (20001, 129, 128), (3000, 2049, 640)])
def test_product_of_a_prompt(mt, M, N, K, w_rows):  # noqa: F811
    a, sa, w, sw = product_case(M + N, M, N, K, w_rows)
    st = status()
    got = mt.gemm_fp8_block128(dev(a), dev(sa), dev(w), dev(sw), dev_status=st)
    assert st.item() == 0
    check_product(got, a, sa, w, sw, w_rows)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K,V", [(700, 3000), (513, 40)])
def test_logits_long_draft_chains(mt, K, V, dtype):  # noqa: F811
    """More drafts than fit the entries in shared memory, most of them several times."""
    c = Case(K, 2, K, V, dtype, **ALL)
    out = torch.empty(c.R, V, device="cuda")
    argmax = c.call(mt, argmax=torch.empty(c.R, dtype=torch.int64, device="cuda"), out_logits=out)
    rows = [0, 1, 2, 300, 511, 512, K - 1, K, K + 1, K + 2, c.R - 2, c.R - 1]
    c.check(argmax, None, out, rows)


def far_rows(R, V, dtype, last):
    """A view [R, V] whose last row starts `last` elements behind the first."""
    ld = last // (R - 1) // 64 * 64
    buf = torch.empty((R - 1) * ld + V, dtype=dtype, device="cuda")
    return buf.as_strided((R, V), (ld, 1))


@pytest.mark.parametrize("M", [5, 70])
def test_product_offsets_past_32_bits(mt, M):  # noqa: F811
    a, sa, w, sw = product_case(M, M, 200, 256, 1)
    for out in (torch.bfloat16, torch.float32):
        o = far_rows(M, 200, out, 4_500_000_000)
        mt.gemm_fp8_block128(dev(a), dev(sa), dev(w), dev(sw), out=o)
        check_product(o.contiguous(), a, sa, w, sw, 1)
        del o
    # a weight of 4.3 GB: its last rows
    N, K = 700_001, 6144
    wide = torch.zeros(N, K, dtype=torch.uint8, device="cuda")
    a, sa, w, sw = product_case(M, M, 300, K, 128)
    wide[-300:] = dev(w)
    scale = torch.ones(-(-N // 128), K // 128, device="cuda")
    first = (N - 300) // 128 * 128                      # block rows of the last 300 weight rows
    got = mt.gemm_fp8_block128(dev(a), dev(sa), wide, scale)
    assert not got[:, :-300].any() and first > 0
    check_product(got[:, -300:].contiguous(), a, sa, w, np.ones((3, K // 128), np.float32), 128)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_logits_and_table_offsets_past_32_bits(mt, dtype):  # noqa: F811
    V, R = 50001, 6
    c = Case(51, 2, 2, V, dtype, **ALL)
    x = far_rows(R, V, dtype, 4_500_000_000)
    x.copy_(c.logits)
    probs, out = far_rows(R, V, torch.float32, 4_500_000_000), far_rows(R, V, torch.float32, 2_300_000_000)
    table = torch.zeros(90_000, mt.token_counts_ld(V), dtype=torch.int16, device="cuda")      # 4.5e9 words
    rows = torch.tensor([89_999, 45_000], dtype=torch.int32, device="cuda")
    tokens, lens = dev(np.random.default_rng(5).integers(0, V, 6000).astype(np.int64)), [5000, 1000]
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.uint32)
    mt.token_counts_build(tokens, u32(off), V, n_prompt=dev(np.array([100, 900])), counts=table, count_rows=rows)
    mt.token_counts_accept(table, V, dev(c.draft), dev(np.array([2, 1], np.int32)), dev(np.array([7, 9])), count_rows=rows)
    want = ologits.token_counts_build(np.zeros((2, table.shape[1]), np.int16), tokens.cpu().numpy(), off, V, [100, 900])
    want = ologits.token_counts_accept(want, V, c.draft, np.array([2, 1]), np.array([7, 9]))
    assert np.array_equal(table[rows.long()].cpu().numpy(), want) and int(torch.count_nonzero(table)) == np.count_nonzero(want)
    c.counts = want
    argmax = torch.empty(R, dtype=torch.int64, device="cuda")
    c.call(mt, logits=x, counts=table, count_rows=rows, argmax=argmax, probs=probs, out_logits=out)
    c.check(argmax, probs, out)


def test_logits_very_high_temperatures(mt):  # noqa: F811
    """Temperatures up to the largest float, with logits of that size: log2(e) / T is subnormal there (spacing 2^-149, at
    least 2^-127.5 here, so that it is off by up to 2^-22.5 of its value), its product with a difference is not."""
    V, temps = 64, [1e38, 1.3e38, 1.5e38, 2.5e38, 3.4e38]
    rng = np.random.default_rng(61)
    x = (rng.uniform(-1.6e38, 1.6e38, (len(temps), V))).astype(np.float32)
    probs = torch.empty(len(temps), V, device="cuda")
    mt.process_logits(dev(x), u32(np.arange(len(temps) + 1)), temperature=dev(np.array(temps, np.float32)), probs=probs)
    for r, t in enumerate(np.array(temps, np.float32).astype(np.float64)):
        d = (x[r].astype(np.float64) - x[r].max()) / t
        want = np.exp(d) / np.exp(d).sum()
        # three roundings, the constant and the subnormal quotient: below 2^-21.3 of an exponent of at most 3.2; then as
        # in test_gpu_head.py
        rel = np.expm1(2 * 2.0 ** -21.3 * 3.2) + 2.0 ** -22 + (V + 1) * 2.0 ** -23
        assert (np.abs(probs[r].double().cpu().numpy() - want) <= 2 * rel * want).all()
    t = torch.full((len(temps),), float("inf"), device="cuda")          # every open token alike
    mask = dev(np.full((1, 2), 0x0F0F0F0F, np.int32))
    mt.process_logits(dev(x), u32(np.arange(len(temps) + 1)), temperature=t, bitmask=mask,
                      mask_rows=dev(np.zeros(len(temps), np.int32)), probs=probs)
    got = probs.cpu().numpy().reshape(len(temps), -1, 8)
    assert (got[:, :, 4:] == 0).all() and np.allclose(got[:, :, :4], 1 / 32, rtol=1e-6, atol=0)
