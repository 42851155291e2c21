"""The head's operators where a launch takes another path than its ordinary one: table builds whose CTAs go through
several blocks of 32768 tokens, token ids that are no 32-bit numbers inside a run of wide loads, and the verify head with
grammar masks and bf16 logits.  Tolerances are those of test_gpu_head.py."""
import numpy as np
import pytest
import torch

from oracle import accept as oaccept
from oracle import fp8 as ofp8
from oracle import logits as ologits
from test_gpu_head import ALL, Case, check_product, dev, mt, status, u32  # noqa: F401

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
