"""The head's operators where a launch takes another path than its ordinary one: table builds whose CTAs go through
several blocks of 32768 tokens, and token ids that are no 32-bit numbers inside a run of wide loads."""
import numpy as np
import pytest

from oracle import logits as ologits
from test_gpu_head import dev, mt, status, u32  # noqa: F401

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
