"""Calls that fill and read the caches, at the edges of what they document: lengths without a bound, request counts at the limits of
shared memory, values next to zero, misaligned buffers, padded batches, layers on several streams.  Each against the float64
oracle or the exact result."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from mtp_speculative_decode_gb300 import _native as N
from oracle import fp8 as ofp8
from oracle import latent4 as o4
from oracle import mla as omla
from oracle import paged as opaged
from oracle import tables as otab
import parity
from test_gpu_cache import SCALE, STATUS, check_mla, dev, i32, mla_case, mt, status, rope_table, table_case, u32  # noqa: F401
from test_gpu_cache_step import tokens

pytestmark = pytest.mark.gpu

# ----------------------------------------------------------------------------- block tables

@pytest.mark.parametrize("keep_len", [2 ** 63 - 1, 2 ** 63 - 64, 2 ** 62, 2 ** 32 + 5])
@pytest.mark.parametrize("ps", [1, 64])
def test_release_keeping_more_than_any_length(mt, ps, keep_len):  # noqa: F811
    """The largest int64 says that a request keeps everything: its pages stay, the others' go."""
    rng = np.random.default_rng(ps)
    t, old, _, free = table_case(rng, 6, ps, 20, 20 * ps, True)
    free, n_free = np.concatenate([free, np.full(120, -3, np.int32)]), len(free)
    keep = np.array([keep_len, 0, keep_len, 3, keep_len, 0], np.int64)
    d_t, d_f, d_n, st = dev(t), dev(free), i32([n_free]), status()
    mt.block_table_release(d_t, ps, dev(old), d_f, d_n, keep_len=dev(keep), dev_status=st)
    w_t, w_f, w_n, w_st = otab.release(t, ps, old, free, n_free, keep)
    assert w_st == 0 and st.item() == 0 and d_n.item() == w_n > n_free
    assert np.array_equal(d_t.cpu().numpy(), w_t) and np.array_equal(d_f.cpu().numpy(), w_f)


@pytest.mark.parametrize("B", [4073, 4074, 4096, 4097])
def test_grow_with_request_counts_at_the_limit_of_shared_memory(mt, B):  # noqa: F811
    """Each count in a process of its own: what an earlier call asked for holds for the rest of a process."""
    here = os.path.dirname(os.path.abspath(__file__))
    code = ("import sys; sys.path[:0] = [%r, %r]\n"
            "import numpy as np, mtp_speculative_decode_gb300 as m\n"
            "from test_gpu_cache import check_grow, table_case\n"
            "t, old, new, free = table_case(np.random.default_rng(%d), %d, 4, 3, 12, True)\n"
            "for in_place in (True, False):\n"
            "    check_grow(m, t, 4, new, free, len(free), old, in_place, [1] * %d)\n" % (os.path.dirname(here), here, B, B, B))
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]


# ----------------------------------------------------------------------------- norms, rotation, codes

@pytest.mark.parametrize("kind", ["quantizer", "heads", "elements", "rows", "pack"])
def test_scales_of_values_next_to_zero(mt, kind):  # noqa: F811
    """The largest magnitude of a block over 448 in float32 has no value left below about 3e-43: the scale is then 1, as for a block
    of zeros, and the codes are zeros that keep their signs."""
    step = 2.0 ** -149
    top = np.array([0, 1, 200, 223, 225, 448, 630, 700, 10000]) * step
    x = np.zeros((len(top), 128))
    x[:, 3], x[:, 70], x[:, 127] = top, -top / 2, -step * (top > 0)
    x = x.astype(np.float32)
    amax = np.abs(x).max(1)
    scale = amax / np.float32(448)
    scale = np.where(scale > 0, scale, np.float32(1))
    codes = ofp8.encode_e4m3_rne_satfinite((x / scale[:, None]).astype(np.float64))
    assert (scale[:4] == 1).all() and (scale[4:] < 1e-40).all() and (codes[:4] & 127 == 0).all() and (codes[4:] & 127).max() == 126
    T = len(top)
    if kind == "quantizer":
        got, sc = mt.quantize_fp8_block128(dev(x))
    elif kind in ("heads", "elements"):
        wide = torch.zeros(T, 129, device="cuda")
        wide[:, :128] = dev(x)
        q = dev(x) if kind == "heads" else wide[:, :128]             # (rows off 16 bytes: the kernel for any shape)
        got, sc = torch.full((T, 128), 9, dtype=torch.uint8, device="cuda"), torch.full((T, 1), 9.0, device="cuda")
        mt.norm_rope(None, None, q=q, q_out=got, q_scale=sc)
    else:
        latent = torch.zeros(T, 576, device="cuda")
        latent[:, 256:384] = dev(x)
        packed = torch.full((T, 656), 9, dtype=torch.uint8, device="cuda")
        if kind == "rows":
            mt.norm_rope(None, None, k=latent, k_out=packed)
        else:
            mt.pack_latent_fp8(latent, packed)
        got, sc = packed[:, 256:384], packed[:, 520:524].contiguous().view(torch.float32)
        assert (packed[:, :256] == 0).all() and (packed[:, 384:512] == 0).all()
    assert np.array_equal(got.cpu().numpy(), codes) and np.array_equal(sc.cpu().numpy().reshape(-1), scale)


@pytest.mark.parametrize("D,rot", [(128, 0), (128, 128), (90, 0), (90, 90)])
def test_norm_whose_reciprocal_root_is_infinite(mt, D, rot):  # noqa: F811
    """eps 0 and a head whose squares have no float32 value: x times infinity times the weight, as the formula's three factors give
    it; zeros give NaN."""
    x = torch.tensor([1e-30, -3e-25, 0.0, 2e-38, 1e-45]).cuda().repeat(D)[:D].view(1, 1, D).repeat(3, 2, 1)
    x[1] = torch.randn(2, D, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    w = torch.linspace(0.5, 2, D, device="cuda")
    w[1], w[8], w[20] = -1.0, 3e38, 0.0
    pos, cs = (None, None) if not rot else (dev(np.zeros(3, np.int64)), torch.tensor([0.8, 0.6]).cuda().repeat_interleave(rot // 2)[None])
    got, _ = mt.norm_rope(pos, cs, q=x, q_norm="rms", q_weight=w, eps=0.0)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True))
    want = x * r * w
    size = want.abs()
    assert r[0].isinf().all() and want[0].isinf().any() and want[0].isnan().any() and r[1].isfinite().all()
    if rot:
        a, b = want[..., :rot // 2], want[..., rot // 2:]
        want = torch.cat([a * 0.8 - b * 0.6, a * 0.6 + b * 0.8], -1)
        size = (a.abs() + b.abs()).repeat(1, 1, 2)
    plain = ~want.isfinite()
    assert plain[0].all() and torch.equal(got.isnan(), want.isnan()) and torch.equal(got[plain].nan_to_num(), want[plain].nan_to_num())
    # (two sums of up to 128 squares: 2^-17 of each other)
    assert ((got - want).abs() <= 2.0 ** -15 * size)[~plain].all()


# ----------------------------------------------------------------------------- attention over 4-bit rows

def attention_bound(q, c):
    """(o, bound of its error, lse, bound) of one row in 64 bits: q [H, 576], c [n, 576].

    A score is the sum of two halves of the dims, 256..511 and the rest.  Each CTA of a pair keeps its own half (float32, at most
    2^-17 of the sum of the products' magnitudes off) and gets the other rounded to half precision: 2^-11 of it, or 2^-25.  A score off by e
    weighs its position by 2^e, so the output moves by the weighted distances of the rows from it; probabilities are
    rounded to bf16 (2^-8), the output too.  A probability below 2^-126 of the reference (which is one of the scores, so the sum is
    at least 1) is zero: n of them move a value by up to n 2^-126 of the largest entry, all that there is where the other rows hold
    zeros."""
    k = SCALE / math.log(2)
    s = q @ c.T
    p = np.exp(SCALE * (s - s.max(1, keepdims=True)))
    lse = SCALE * s.max(1) + np.log(p.sum(1))
    p /= p.sum(1, keepdims=True)
    o = p @ c[:, :512]
    mags = np.abs(q) @ np.abs(c).T * k
    upper = q[:, 256:512] @ c[:, 256:512].T * k
    bound, lse_bound = np.zeros_like(o), None
    for dims, other in ((slice(0, 256), upper), (slice(256, 512), s * k - upper)):
        eps = math.log(2) * (2.0 ** -11 * np.abs(other) + 2.0 ** -25 + 2.0 ** -17 * mags) + 2.0 ** -20
        least = (p * np.exp(-eps)).sum(1)
        for h in range(len(q)):
            moved = (p[h] * np.expm1(eps[h])) @ np.abs(c[:, dims] - o[h, dims])
            bound[h, dims] = (moved + (p[h] * np.exp(eps[h])) @ np.abs(c[:, dims]) * 2.0 ** -8) / least[h]
        if lse_bound is None:              # the first half's CTA writes it
            lse_bound = np.log((p * np.exp(eps)).sum(1)) + np.abs(lse) * 2.0 ** -22
    return o, bound + (np.abs(o) + bound) * 2.0 ** -8 + len(c) * 2.0 ** -126 * np.abs(c).max(), lse, lse_bound


@pytest.mark.parametrize("H", [128, 48])
@pytest.mark.parametrize("factor", [1, 10, 40])
def test_mla_error_of_every_value(mt, factor, H):  # noqa: F811
    """Scores up to several hundred, rising through the list so that the reference maximum moves in every tile: each value within
    the bound of the roundings, which stays far below the output (2 % of a row, 15 % of any head)."""
    rng = np.random.default_rng(78)
    q, rows, caps, start, pos, idx = mla_case(rng, 1, 2, H, 512, [4000])
    q = (q.float() * factor).to(torch.bfloat16)
    c = o4.unpack(rows)
    idx[0] = np.argsort((q[0].float().numpy() @ c[:4000].T).mean(0))[-512:]
    lse, st = torch.empty(2, H, device="cuda"), status()
    out = mt.sparse_mla_decode(q.cuda(), dev(rows), dev(start), u32([0, 2]), dev(pos), dev(idx), SCALE, lse=lse, dev_status=st)
    assert st.item() == 0
    for r in range(2):
        o, bound, want_lse, lse_bound = attention_bound(q[r].double().numpy(), c[idx[r][idx[r] >= 0]])
        norm = lambda x: np.linalg.norm(x, axis=1)  # noqa: E731
        assert np.linalg.norm(bound) < 0.02 * np.linalg.norm(o) and (norm(bound) < 0.15 * norm(o)).all()
        assert (np.abs(out[r].double().cpu().numpy() - o) <= bound).all()
        assert (np.abs(lse[r].double().cpu().numpy() - want_lse) <= lse_bound).all()


@pytest.mark.parametrize("page", [0, 4, 64])
@pytest.mark.parametrize("H", [16, 128])
def test_mla_into_a_misaligned_output(mt, H, page, monkeypatch):  # noqa: F811
    """An output that no TMA store can write takes the kernel for any alignment: short and split lists, codes of 0.5, empty rows."""
    rng = np.random.default_rng(H + page)
    for B, W, n_idx, lens in ((1, 1, 1, [0]), (2, 3, 65, [70, 3]), (1, 2, 2048, [5000])):
        q, rows, caps, start, pos, idx = mla_case(rng, B, W, H, n_idx, lens)
        rows[0, :256] = 0x11                                     # 0.5 throughout
        pool, paged, cs = rows, None, dev(start)
        if page:
            t = np.full((B, max(otab.n_pages(n, page) for n in caps)), -1, np.int32)
            ids, at = rng.permutation(sum(otab.n_pages(n, page) for n in caps)), 0
            pool = rng.integers(0, 256, (len(ids) * page, 416)).astype(np.uint8)
            for b in range(B):
                n = otab.n_pages(caps[b], page)
                t[b, :n] = ids[at:at + n]
                at += n
                for s in range(caps[b]):
                    pool[opaged.slot_of(t, page, b, s)] = rows[start[b] + s]
            paged, cs = (dev(t), page), None
        lse, st = torch.empty(B * W, H, device="cuda"), status()
        buf = torch.full((B * W * H * 512 + 4,), 5.0, dtype=torch.bfloat16, device="cuda")
        out = buf[2:-2].view(B * W, H, 512)
        got = mt.sparse_mla_decode(q.cuda(), dev(pool), cs, u32(np.arange(B + 1) * W), dev(pos), dev(idx), SCALE, out=out, lse=lse,
                                   dev_status=st, paged=paged)
        assert got is out and st.item() == 0 and (buf[:2] == 5).all() and (buf[-2:] == 5).all()
        check_mla(out, lse, q, rows, start, W, idx)
        # the same kernel by choice (the bits of its own sums), and the one for aligned outputs
        args = (q.cuda(), dev(pool), cs, u32(np.arange(B + 1) * W), dev(pos), dev(idx), SCALE)
        other = mt.sparse_mla_decode(*args, paged=paged)
        monkeypatch.setenv("MTPSD_MLA", "mma")
        assert torch.equal(mt.sparse_mla_decode(*args, paged=paged), out)
        monkeypatch.delenv("MTPSD_MLA")
        assert torch.equal(mt.sparse_mla_decode(*args, paged=paged), other) and (n_idx == 1 or not torch.equal(other, out))


@pytest.mark.parametrize("kind", ["fp4", "fp8", "bf16", "f32"])
def test_mla_with_a_misaligned_workspace(mt, kind):  # noqa: F811
    """Split partials at any multiple of 8 bytes: joined by loads that such a buffer allows; at less the call is refused."""
    rng = np.random.default_rng(15)
    H = 16 if kind == "f32" else 128
    q, rows, caps, start, pos, idx = mla_case(rng, 1, 2, H, 2048, [5000])
    dt = {"fp4": N.MTPSD_FP4_MLA, "fp8": N.MTPSD_FP8_DS_MLA, "bf16": N.MTPSD_BF16, "f32": N.MTPSD_F32}[kind]
    c = o4.unpack(rows)
    latent = dev(rows) if kind == "fp4" else torch.tensor(c, dtype=torch.float32).cuda()
    if kind == "fp8":
        latent = mt.pack_latent_fp8(latent)
        c = omla.unpack_fp8_ds_mla(latent.cpu().numpy())
    elif kind == "bf16":
        latent = latent.bfloat16()
    qd = q.float() if kind == "f32" else q
    want = omla.sparse_mla(q, c, start, [0, 0], idx, SCALE)
    need = mt.sparse_mla_workspace_size(2, H, 2048, 0, dt)
    assert need > 0
    for off in (0, 8, 16, 24, 4, 1):
        buf = torch.full((need + 64,), 0xff, dtype=torch.uint8, device="cuda")
        ws, st = buf[off:off + need], status()
        call = lambda: mt.sparse_mla_decode(qd.cuda(), latent, dev(start), u32([0, 2]), dev(pos), dev(idx), SCALE,  # noqa: E731
                                            workspace=ws, dev_status=st)
        if off % (4 if kind == "f32" else 8):
            with pytest.raises(RuntimeError, match="aligned"):
                call()
            torch.cuda.synchronize()
            assert (buf == 0xff).all()
            continue
        out = call()
        assert st.item() == 0 and (buf[:off] == 0xff).all() and (buf[off + need:] == 0xff).all()
        for r, (o, _) in want.items():
            parity.check_attention_row(out[r].float().cpu().numpy(), o, parity.ATT_TOL_F32 if kind == "f32" else parity.ATT_TOL_BF16)


# ----------------------------------------------------------------------------- the layer

def layer(row_bytes, max_len=320, page=16, max_tokens=64, H=32, n_pages=60):
    from mtp_speculative_decode_gb300 import pipeline
    rng = np.random.default_rng(5)
    w = lambda n: dev((1 + 0.2 * rng.normal(size=n)).astype(np.float32))  # noqa: E731
    return pipeline.PagedAttention(3, max_len, n_pages, page, dev(rope_table(max_len + page, 64)), w(128), w(128), w(512), H=H, H_I=32,
                                   topk=64, max_tokens=max_tokens, row_bytes=row_bytes)


def lens(x):
    return dev(np.array(x, np.int64))


def state(L):
    return [x.clone() for x in (L.block_table, L.free_pages, L.n_free, L.lengths, L.latent, L.k_cache, L.k_scale)]


@pytest.mark.parametrize("row_bytes", [416, 656, 1152])
def test_layer_with_a_padded_batch(mt, row_bytes):  # noqa: F811
    """Tokens behind the last request's: nothing of them reaches the caches (their slots are not those of an earlier step), their
    outputs are zeros; the others are those of a step without them."""
    L, M = layer(row_bytes), layer(row_bytes)
    rng = np.random.default_rng(6)
    x = tokens(rng, 30, 32)
    for a in (L, M):
        a.step(lens([10, 10, 10]), u32([0, 10, 20, 30]), **{k: v.clone() for k, v in x.items()})
    assert L.status.item() == 0
    x = tokens(rng, 30, 32)
    want = M.step(lens([14, 14, 14]), u32([0, 4, 8, 12]), **{k: v[:12].clone() for k, v in x.items()}).clone()
    out = L.step(lens([14, 14, 14]), u32([0, 4, 8, 12]), **x)
    assert L.status.item() == STATUS["ROW_RANGE"] and M.status.item() == 0
    assert all(torch.equal(a, b) for a, b in zip(state(L), state(M)))
    assert torch.equal(out[:12], want) and (out[12:] == 0).all()
    fresh = layer(row_bytes)                                     # and in the first step of all
    fresh.step(lens([2, 0, 0]), u32([0, 2, 2, 2]), **tokens(rng, 9, 32))
    assert (fresh.k_scale != 0).sum() == 2 and fresh.status.item() == STATUS["ROW_RANGE"]


def misfits(x):
    """name -> arguments of a step that the layer has to refuse."""
    def but(**kw):
        return {**x, **kw}

    def off(t):
        wide = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
        return wide[1:].view(t.shape).copy_(t)

    return {"many": {k: torch.cat([v] * 3) for k, v in x.items()}, "kv": but(kv=x["kv"][:-1]), "k_idx": but(k_idx=x["k_idx"][1:]),
            "q_idx": but(q_idx=x["q_idx"][:, :-1]), "w_idx": but(w_idx=x["w_idx"][:-1]), "w_type": but(w_idx=x["w_idx"].double()),
            "heads": but(q=x["q"][:, 1:]), "strided": but(q=x["q"].transpose(0, 1).contiguous().transpose(0, 1)),
            "f32": but(q=x["q"].float()), "kv_width": but(kv=x["kv"][:, :512]), "k_type": but(k_idx=x["k_idx"].half()),
            "kv_off": but(kv=off(x["kv"])), "q_off": but(q=off(x["q"])), "host": but(w_idx=x["w_idx"].cpu()),
            "w_strided": but(w_idx=x["w_idx"].t().contiguous().t()), "k_heads": but(k_idx=x["k_idx"].t().contiguous().t())}


MISFITS = ["many", "kv", "k_idx", "q_idx", "w_idx", "w_type", "heads", "strided", "f32", "kv_width", "k_type", "kv_off", "q_off", "host",
           "w_strided", "k_heads"]


@pytest.mark.parametrize("name", MISFITS)
def test_refused_step_leaves_the_layer_as_it_was(mt, name):  # noqa: F811
    L = layer(416)
    rng = np.random.default_rng(7)
    L.step(lens([3, 0, 7]), u32([0, 3, 3, 10]), **tokens(rng, 10, 32))
    x = tokens(rng, 24, 32)
    before = state(L)
    with pytest.raises((ValueError, TypeError)):
        L.step(lens([11, 8, 15]), u32([0, 8, 16, 24]), **misfits(x)[name])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(state(L), before)) and L.status.item() == 0
    L.step(lens([11, 8, 15]), u32([0, 8, 16, 24]), **x)
    assert L.status.item() == 0 and L.lengths.tolist() == [11, 8, 15]


def test_refused_lengths_and_layers(mt):  # noqa: F811
    from mtp_speculative_decode_gb300 import pipeline
    L = layer(416)
    x = tokens(np.random.default_rng(8), 6, 32)
    before = state(L)
    for new, off in ((lens([6, 0]), u32([0, 6, 6, 6])), (lens([6, 0, 0]), u32([0, 6, 6])), (lens([6, 0, 0]).int(), u32([0, 6, 6, 6])),
                     (L.lengths, u32([0, 6, 6, 6])), (lens([6, 0, 0]).cpu(), u32([0, 6, 6, 6]))):
        with pytest.raises((ValueError, TypeError)):
            L.step(new, off, **x)
        assert all(torch.equal(a, b) for a, b in zip(state(L), before))
    cs, w = dev(rope_table(400, 64)), torch.ones(512, device="cuda")
    args = dict(B=3, max_len=320, n_pages=60, page_size=16, cos_sin=cs, k_weight=w[:128], k_bias=w[:128], latent_weight=w)
    for bad in (dict(page_size=24), dict(cos_sin=cs[:, :32]), dict(k_weight=w), dict(latent_weight=w.double()), dict(row_bytes=500),
                dict(B=0), dict(max_len=0), dict(k_bias=w[:127]), dict(max_tokens=0), dict(topk=0), dict(H=20)):
        with pytest.raises((ValueError, TypeError)):
            pipeline.PagedAttention(**{**args, **bad})


def test_layer_step_without_tokens(mt):  # noqa: F811
    L = layer(416)
    x = tokens(np.random.default_rng(16), 4, 32)
    L.step(lens([4, 0, 0]), u32([0, 4, 4, 4]), **x)
    out = L.step(lens([4, 20, 0]), u32([0, 0, 0, 0]), **{k: v[:0] for k, v in x.items()})
    assert out.shape == (0, 32, 512) and L.status.item() == 0 and L.lengths.tolist() == [4, 20, 0] and L.n_free.item() == 57


def test_layer_lengths_up_to_the_last_page(mt):  # noqa: F811
    """max_len ends inside a page: a length that the tables accept is seen whole by the selection."""
    rng = np.random.default_rng(9)
    x = tokens(rng, 128, 32)
    got = []
    for max_len in (100, 128):
        L = layer(416, max_len=max_len, page=64, max_tokens=128)
        got.append(L.step(lens([128, 0, 0]), u32([0, 128, 128, 128]), **{k: v.clone() for k, v in x.items()}).clone())
        assert L.status.item() == 0 and (L.topk_idx[127] >= 100).any() and (L.topk_idx[:128].max(1).values <= dev(np.arange(128))).all()
    assert torch.equal(*got)


def test_layer_release_of_lengths_that_are_none(mt):  # noqa: F811
    """A negative length releases nothing (flagged) and is not taken over; the largest one keeps everything."""
    L = layer(416)
    L.step(lens([20, 5, 40]), u32([0, 20, 25, 60]), **{k: v[:60] for k, v in tokens(np.random.default_rng(10), 60, 32).items()})
    table, n_free = L.block_table.clone(), L.n_free.item()
    keep = lens([-1, 2 ** 63 - 1, 17])
    L.release(keep)
    assert L.lengths.tolist() == [20, 5, 17] and L.n_free.item() == n_free + 1 and L.status.item() == STATUS["ROW_RANGE"]
    assert torch.equal(L.block_table[:2], table[:2]) and (L.block_table[2, 2:] == -1).all()
    L.release()
    assert L.n_free.item() == 60 and (L.block_table == -1).all() and (L.lengths == 0).all()


@pytest.mark.parametrize("raw", [False, True])
def test_layer_release_on_a_stream(mt, raw):  # noqa: F811
    """Behind a step on the same stream, with work in front of both that takes a while."""
    L = layer(416)
    x = tokens(np.random.default_rng(17), 60, 32)
    new, off, keep = lens([20, 5, 35]), u32([0, 20, 25, 60]), lens([16, 5, 0])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    on = s.cuda_stream if raw else s
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    L.step(new, off, **x, stream=on)
    L.release(keep, stream=on)
    s.synchronize()
    assert L.lengths.tolist() == [16, 5, 0] and L.n_free.item() == 58 and L.status.item() == 0
    L.release(stream=on)
    s.synchronize()
    assert L.n_free.item() == 60 and (L.block_table == -1).all() and (L.lengths == 0).all()


@pytest.mark.parametrize("row_bytes", [416, 656, 1152])
def test_layer_keeps_its_scratch_to_itself(mt, row_bytes):  # noqa: F811
    """No buffer that other calls use too: those are replaced by larger ones, and written by whoever comes next."""
    from mtp_speculative_decode_gb300 import api
    L = layer(row_bytes, H=128)
    api._default_ws.clear()
    L.step(lens([5, 0, 9]), u32([0, 5, 5, 14]), **tokens(np.random.default_rng(11), 14, 128))
    torch.cuda.synchronize()
    assert not api._default_ws


@pytest.mark.parametrize("row_bytes", [416, 656, 1152])
def test_two_layers_at_once(mt, row_bytes):  # noqa: F811
    """Layers stepped on two streams at the same time, of different sizes: the bits of a step alone."""
    rng = np.random.default_rng(12)
    xs = [tokens(rng, 64, 128), tokens(rng, 9, 128)]
    new, off = [lens([50, 4, 10]), lens([3, 3, 3])], [u32([0, 50, 54, 64]), u32([0, 3, 6, 9])]

    def step(L, i, s=None):
        x = {k: v.clone() for k, v in xs[i].items()}
        torch.cuda.synchronize()
        return L, L.step(new[i], off[i], **x, stream=s), x

    want = [step(layer(row_bytes, H=128), i)[1].clone() for i in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        layers = [layer(row_bytes, H=128) for _ in range(2)]
        copies = [{k: v.clone() for k, v in x.items()} for x in xs]
        torch.cuda.synchronize()
        got = [layers[i].step(new[i], off[i], **copies[i], stream=(streams[0], streams[1].cuda_stream)[i]) for i in range(2)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(L.status.item() == 0 for L in layers)


@pytest.mark.parametrize("row_bytes", [416, 656, 1152])
def test_captured_step_beside_larger_eager_ones(mt, row_bytes):  # noqa: F811
    """A decode step in a graph, replayed after prompts of other layers and calls of other sizes: its scratch is still its own."""
    rng = np.random.default_rng(13)
    x = tokens(rng, 6, 128)
    q0 = x["q"].clone()
    new, off = lens([2, 2, 2]), u32([0, 2, 4, 6])
    M = layer(row_bytes, H=128)
    for n in (2, 4):
        want = M.step(lens([n] * 3), off, **{k: v.clone() for k, v in x.items()}).clone()
    L = layer(row_bytes, H=128)
    L.step(new, off, **{k: v.clone() for k, v in x.items()})
    new.fill_(4)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = L.step(new, off, **x)
    big = layer(row_bytes, H=128, max_len=4000, max_tokens=600, n_pages=400)
    big.step(lens([500, 60, 40]), u32([0, 500, 560, 600]), **tokens(rng, 600, 128))
    junk = [torch.full((1 << 22,), 0xff, dtype=torch.uint8, device="cuda") for _ in range(8)]
    for _ in range(3):                  # (the tables keep what they have: the step is the same each time)
        x["q"].copy_(q0)
        L.out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and L.status.item() == 0
    assert all((j == 0xff).all() for j in junk)
