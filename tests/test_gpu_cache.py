"""Block tables and slot maps, norms with rotation into the caches, 4-bit latent rows and the attention over them, against
the float64 oracle.

Tolerances.  Tables, slots, and the codes and scales of packed rows are exact.  norm_rope computes in float32: a sum of n
squares is off by less than (n / 32 + 8) 2^-24 of itself (at most n / 32 terms per lane of a full warp in turn, n / 4 of
the smallest group, then 5 exchanges; every operation 2^-24), its root and reciprocal add less than 2^-22, the products by r and the weight
2^-23, the centring of a layer norm (n / 4 + 8) 2^-24 of the largest |x|; a rotation multiplies the error by at most 2 and
adds 3 * 2^-24 of |a| + |b|.  SUM(n) = (n / 2 + 40) 2^-24 of the largest magnitude of a head bounds them together.  The output's rounding
adds half a step (bf16 2^-8 relative; FP8 codes 2^-4 relative or 2^-10 of the scale, subnormal).  Attention is held to the 2e-2 of
parity.py, per row."""
import math

import numpy as np
import pytest
import torch

from oracle import fp8 as ofp8
from oracle import latent4 as o4
from oracle import mla as omla
from oracle import paged as opaged
from oracle import rope as orope
from oracle import tables as otab
import parity

pytestmark = pytest.mark.gpu

SCALE = 1.0 / 24.0
STATUS = dict(ROW_RANGE=8, INDEX_RANGE=1, WRITE_RANGE=2, NO_PAGES=32)


@pytest.fixture(scope="module")
def mt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mtp_speculative_decode_gb300 as m
    from mtp_speculative_decode_gb300 import _native
    _native.lib()   # raises if the library is missing: no fallback
    return m


def dev(x):
    return torch.as_tensor(np.ascontiguousarray(x)).cuda()


def u32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.uint32)).cuda()


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def i32(x):
    return dev(np.asarray(x, np.int32))


# ----------------------------------------------------------------------------- block tables

def table_case(rng, B, ps, width, hi, grown):
    """(table, old_len or None, new_len, free list): requests of up to `hi` tokens, tables that hold what they have."""
    old = rng.integers(0, hi + 1, B).astype(np.int64)
    new = np.minimum(old + rng.integers(0, 3 * ps + 2, B), width * ps).astype(np.int64) if grown else old.copy()
    new[rng.integers(0, B)] = 0 if not grown else old[0]
    held = [otab.n_pages(int(n), ps) for n in old]
    ids = rng.permutation(B * width + 40).astype(np.int32)
    t = np.full((B, width), -1, np.int32)
    at = 0
    for b in range(B):
        t[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    return t, (old if grown else None), new, ids[at:].copy() if grown else ids


def check_grow(mt, t, ps, new, free, n_free, old, in_place, counts=None, T_extra=0):
    d_t, d_new, d_free, d_n = dev(t), dev(new), dev(free), i32([n_free])
    d_old = None if old is None else dev(old)
    n_out = d_n if in_place else i32([-7])
    lengths = d_old if in_place and old is not None else dev(np.full(len(t), -7, np.int64))
    st = status()
    want_t, want_len, want_n, want_st = otab.grow(t, ps, new, free, n_free, old)
    kw = {}
    if counts is not None:
        off = np.concatenate([[0], np.cumsum(counts)])
        T = int(off[-1]) + T_extra
        slots, pos = dev(np.full(max(T, 0), -9, np.int64)), dev(np.full(max(T, 0), -9, np.int64))
        kw = dict(token_offsets=u32(off), slots=slots, positions=pos)
        w_slots, w_pos, wrote, slot_st = otab.slot_map(want_t, ps, off, new, T)
        want_st |= slot_st
    got = mt.block_table_grow(d_t, ps, d_new, d_free, d_n, old_len=d_old, lengths=lengths,
                              n_free_out=None if in_place else n_out, dev_status=st, **kw)
    assert got is lengths
    assert np.array_equal(d_t.cpu().numpy(), want_t)
    assert np.array_equal(lengths.cpu().numpy(), want_len)
    assert n_out.item() == want_n and (in_place or d_n.item() == n_free)
    assert np.array_equal(d_free.cpu().numpy(), free)
    assert st.item() == want_st
    if counts is not None:
        assert np.array_equal(slots.cpu().numpy(), np.where(wrote, w_slots, -9))
        assert np.array_equal(pos.cpu().numpy(), np.where(wrote, w_pos, -9))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("grown", [True, False])
@pytest.mark.parametrize("ps,B,width", [(1, 1, 5), (1, 33, 700), (4, 7, 3), (64, 100, 40), (16, 1500, 9), (64, 3, 3000)])
def test_block_table_grow(mt, ps, B, width, grown, in_place):
    rng = np.random.default_rng(ps * 1000 + B + grown)
    t, old, new, free = table_case(rng, B, ps, width, width * ps, grown)
    need = sum(max(0, otab.n_pages(int(n), ps) - (0 if old is None else otab.n_pages(int(o), ps)))
               for n, o in zip(new, new if old is None else old))
    for n_free in (len(free), need, max(need - 1, 0), need // 2, 0):
        counts = [int(rng.integers(0, min(n, 9) + 1)) for n in new] if n_free != need else None
        check_grow(mt, t, ps, new, free, n_free, old, in_place, counts)


def test_block_table_grow_whole_prompts(mt):
    """Every token of long and short requests: steps inside a request, across requests and over empty ones."""
    rng = np.random.default_rng(5)
    new = np.array([0, 1, 127, 128, 129, 0, 40000, 31, 33, 0, 9999, 5], np.int64)
    t = np.full((12, 700), 3, np.int32)
    free = rng.permutation(900).astype(np.int32)
    for n_free in (900, 640):
        check_grow(mt, t, 64, new, free, n_free, None, False, list(new))
    many = rng.integers(0, 3, 8192).astype(np.int64)
    check_grow(mt, np.full((8192, 2), 7, np.int32), 1, many, rng.permutation(20000).astype(np.int32), 20000, None, True, list(many))


def test_block_table_grow_bad_values(mt):
    rng = np.random.default_rng(6)
    t, old, new, free = table_case(rng, 8, 4, 10, 30, True)
    old[1], new[2], new[3], old[4] = -1, -5, 41, 45
    free[len(free) - 2] = -4                        # handed out as it is
    check_grow(mt, t, 4, new, free, len(free), old, False, [0, 2, 2, 2, 2, 2, 2, 2])
    check_grow(mt, t, 4, new, free, len(free), old, True)
    check_grow(mt, t, 4, new, free, len(free) + 3, old, False)       # a count past the list, and a negative one
    check_grow(mt, t, 4, new, free, -1, old, False)
    check_grow(mt, t, 4, np.abs(new) % 40, free, 50, None, False, [3] * 8, T_extra=5)      # a padded batch
    check_grow(mt, t, 4, np.abs(new) % 40, free, 50, None, False, [3] * 8, T_extra=-5)     # arrays shorter than the offsets say


def test_block_table_empty_batch(mt):
    st, n = status(), i32([4])
    empty = torch.empty(0, dtype=torch.int64, device="cuda")
    out = mt.block_table_grow(torch.empty(0, 3, dtype=torch.int32, device="cuda"), 4, empty, i32([1, 2, 3, 4]), n, dev_status=st,
                              token_offsets=u32([0]), slots=empty, positions=empty)
    assert out.numel() == 0 and n.item() == 4 and st.item() == 0
    mt.block_table_release(torch.empty(0, 3, dtype=torch.int32, device="cuda"), 4, empty, i32([1]), n)
    mt.slot_map(torch.empty(0, 3, dtype=torch.int32, device="cuda"), 4, u32([0]), empty, dev([5, 5]))


@pytest.mark.parametrize("ps,B,width", [(1, 3, 100), (4, 40, 70), (64, 2000, 3)])
def test_block_table_release(mt, ps, B, width):
    rng = np.random.default_rng(B)
    t, _, old, ids = table_case(rng, B, ps, width, width * ps, True)
    old = np.array([int((row >= 0).sum()) * ps for row in t], np.int64)
    t[B // 2, 0] = -1                               # a hole: passed over
    held = int((t >= 0).sum())
    for keep, cap, n_free in ((None, held + 9, 9), (old // 3, held + 9, 0), (old // 3, held // 3, 2), (old + 5, 50, 7)):
        free = rng.integers(0, 99, cap).astype(np.int32)
        d_t, d_f, d_n, st = dev(t), dev(free), i32([n_free]), status()
        mt.block_table_release(d_t, ps, dev(old), d_f, d_n, keep_len=None if keep is None else dev(keep), dev_status=st)
        w_t, w_f, w_n, w_st = otab.release(t, ps, old, free, n_free, keep)
        assert np.array_equal(d_t.cpu().numpy(), w_t) and np.array_equal(d_f.cpu().numpy(), w_f)
        assert d_n.item() == w_n and st.item() == w_st
    bad = old.copy()
    bad[0], bad[-1] = -1, width * ps + 1
    for n_free in (0, 200 * B * width, -1):
        d_t, d_f, d_n, st = dev(t), dev(np.zeros(held + 9, np.int32)), i32([n_free]), status()
        mt.block_table_release(d_t, ps, dev(bad), d_f, d_n, dev_status=st)
        w_t, w_f, w_n, w_st = otab.release(t, ps, bad, np.zeros(held + 9, np.int32), n_free)
        assert np.array_equal(d_t.cpu().numpy(), w_t) and np.array_equal(d_f.cpu().numpy(), w_f)
        assert d_n.item() == w_n and st.item() == w_st


@pytest.mark.parametrize("ps,B", [(1, 9), (4, 300), (64, 20000)])
def test_slot_map(mt, ps, B):
    rng = np.random.default_rng(B)
    width = 6
    t = rng.integers(-1, 1 << 30, (B, width)).astype(np.int32)       # slots past 2^31 too
    lengths = rng.integers(0, width * ps + 3, B).astype(np.int64)    # some past the row
    counts = rng.integers(0, 5, B)
    counts[B // 3] = 100                                             # more tokens than the request has
    off = np.concatenate([[0], np.cumsum(counts)]) + 3               # the first three tokens belong to nobody
    T = int(off[-1]) + 40
    want, pos, wrote, w_st = otab.slot_map(t, ps, off, lengths, T)
    for with_pos in (True, False):
        slots, p, st = dev(np.full(T, -9, np.int64)), dev(np.full(T, -9, np.int64)), status()
        mt.slot_map(dev(t), ps, u32(off), dev(lengths), slots, positions=p if with_pos else None, dev_status=st)
        assert np.array_equal(slots.cpu().numpy(), np.where(wrote, want, -9)) and st.item() == w_st
        assert np.array_equal(p.cpu().numpy(), np.where(wrote, pos, -9) if with_pos else np.full(T, -9))


# ----------------------------------------------------------------------------- norms and rotation

def rope_table(n_pos, rot):
    ang = np.arange(n_pos)[:, None] * 1000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def reference(x, norm, weight, bias, norm_dim, eps, cs, pos, start, inter):
    y = orope.norm(x, norm, eps, weight, bias, norm_dim)
    return y if cs is None else orope.rotate(y, cs[pos], start, inter)


def tolerance(x, want, dtype, norm, eps, norm_dim, weight, bias):
    """Per head: SUM(n) of the largest magnitude (of the result, or of what a norm makes of the largest input; a bias's too), and the
    output's half step."""
    n = x.shape[-1] if norm_dim is None else norm_dim
    top = np.abs(want).max(axis=-1, keepdims=True)
    if norm is not None:
        y = x[..., :n]
        var = (y * y).mean(-1, keepdims=True) - (y.mean(-1, keepdims=True) ** 2 if norm == "layer" else 0)
        w = 1.0 if weight is None else np.abs(weight).max()
        top = np.maximum(top, np.abs(y).max(-1, keepdims=True) / np.sqrt(var + eps) * w)
    if bias is not None:
        top = top + np.abs(bias).max()
    tol = (n / 2 + 40) * 2.0 ** -24 * top
    return tol + (np.abs(want) + tol) * 2.0 ** -8 if dtype == torch.bfloat16 else tol


def rope_inputs(rng, T, H, D, dtype, spread=3.0):
    x = rng.normal(size=(T, H, D)) * np.exp(rng.uniform(-spread, spread, (1, H, 1))) + 0.3
    return torch.tensor(x).to(dtype).cuda()


ROPE = [  # D, rot, q rot_start, norm_dim
    (128, 64, 0, None), (128, 128, 0, None), (128, 64, 64, 96), (64, 64, 0, None), (576, 64, 512, 512), (256, 64, 192, None),
    (256, 256, 0, None), (512, 512, 0, 256), (1024, 64, 8, None), (1024, 1024, 0, None), (96, 96, 0, None), (80, 80, 0, None), (72, 32, 16, 40),
    (8, 0, 0, None), (192, 0, 0, 8), (1, 0, 0, None), (2, 2, 0, None), (90, 50, 3, 77), (128, 50, 0, None), (1023, 1022, 1, 1000)]


@pytest.mark.parametrize("D,rot,start,norm_dim", ROPE)
@pytest.mark.parametrize("norm", [None, "rms", "layer"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_rope(mt, D, rot, start, norm_dim, norm, dtype):
    rng = np.random.default_rng(D * 7 + rot)
    eps = 1e-6
    n = D if norm_dim is None else norm_dim
    for T, Hq, Hk, inter in ((1, 3, 1, False), (19, 5, 2, True), (130, 33, 1, False)):
        q, k = rope_inputs(rng, T, Hq, D, dtype), rope_inputs(rng, T, Hk, D, dtype)
        w, b = (1 + 0.3 * rng.normal(size=n)).astype(np.float32), rng.normal(size=n).astype(np.float32)
        w = w if norm else None
        b = b if norm and T != 19 else None
        cs = rope_table(300, rot) if rot else None
        pos = rng.integers(0, 300, T)
        st = status()
        gq, gk = mt.norm_rope(dev(pos) if rot else None, dev(cs) if rot else None, q=q, k=k, q_norm=norm, k_norm=norm,
                              q_weight=None if w is None else dev(w), k_weight=None if w is None else dev(w),
                              k_bias=None if b is None else dev(b), q_norm_dim=norm_dim, k_norm_dim=norm_dim, q_rot_start=start,
                              k_rot_start=start, interleaved=inter, eps=eps, dev_status=st)
        assert st.item() == 0
        for x, g, bias in ((q, gq, None), (k, gk, b)):
            xd = x.double().cpu().numpy()
            want = reference(xd, norm, w, bias, norm_dim, eps, cs, pos, start, inter)
            err = np.abs(g.double().cpu().numpy() - want)
            tol = tolerance(xd, want, dtype, norm, eps, norm_dim, w, bias)
            assert g.dtype == dtype and (err <= tol).all(), float((err - tol).max())


@pytest.mark.parametrize("D,rot", [(128, 64), (90, 50), (64, 64), (128, 0)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_rope_strides_types_and_in_place(mt, D, rot, dtype):
    """Views of a fused projection, odd offsets, the other output type, in place: the same values."""
    rng = np.random.default_rng(D + rot)
    T, Hq, Hk = 37, 6, 2
    cs, pos = (dev(rope_table(99, rot)), dev(rng.integers(0, 99, T))) if rot else (None, None)
    w = dev((1 + 0.2 * rng.normal(size=D)).astype(np.float32))
    kw = dict(q_norm="rms", k_norm="layer", q_weight=w, k_weight=w)
    fused = rope_inputs(rng, T, Hq + Hk, D, dtype)
    q, k = fused[:, :Hq].contiguous(), fused[:, Hq:].contiguous()
    want_q, want_k = mt.norm_rope(pos, cs, q=q, k=k, **kw)
    got = mt.norm_rope(pos, cs, q=fused[:, :Hq], k=fused[:, Hq:], **kw)
    assert torch.equal(got[0], want_q) and torch.equal(got[1], want_k)
    odd = torch.zeros(T * (Hq * D + 3) + 1, dtype=dtype, device="cuda")[1:].view(T, -1)[:, :Hq * D].view(T, Hq, D)
    odd.copy_(q)
    out = torch.zeros(T, Hq, D + 1, dtype=dtype, device="cuda")[:, :, :D]
    got_q, _ = mt.norm_rope(pos, cs, q=odd, q_norm="rms", q_weight=w, q_out=out)
    assert got_q is out
    # another kernel may sum in another order: float32 sums of D terms
    a, b = got_q.double(), want_q.double()
    step = 2.0 ** -7 if dtype == torch.bfloat16 else 0.0
    assert ((a - b).abs() <= step * b.abs() + (D + 80) * 2.0 ** -24 * b.abs().amax()).all()
    heads_first = torch.empty(Hk, T, D, dtype=dtype, device="cuda")
    heads_first.copy_(k.transpose(0, 1))
    back = torch.empty_like(heads_first)
    _, got_k = mt.norm_rope(pos, cs, k=heads_first.transpose(0, 1), k_norm="layer", k_weight=w, k_out=back.transpose(0, 1))
    assert torch.equal(back.transpose(0, 1), want_k)
    other = torch.float32 if dtype == torch.bfloat16 else torch.bfloat16
    wide, _ = mt.norm_rope(pos, cs, q=q, q_norm="rms", q_weight=w, q_out=torch.empty(T, Hq, D, dtype=other, device="cuda"))
    assert torch.equal(wide.to(torch.bfloat16), want_q.to(torch.bfloat16))
    q2, k2 = q.clone(), fused.clone()
    mt.norm_rope(pos, cs, q=q2, k=k2[:, Hq:], q_out=q2, k_out=k2[:, Hq:], **kw)
    assert torch.equal(q2, want_q) and torch.equal(k2[:, Hq:], want_k) and torch.equal(k2[:, :Hq], q)
    # in place, nothing but the turned dims
    if rot and D == 128:
        q3 = fused.clone()
        mt.norm_rope(pos, cs, q=q3, q_rot_start=D - rot, q_out=q3)
        w3, _ = mt.norm_rope(pos, cs, q=fused, q_rot_start=D - rot)
        assert torch.equal(q3, w3) and torch.equal(q3[:, :, :D - rot], fused[:, :, :D - rot])


@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_rope_fp8_into_the_indexer_cache(mt, dtype, aligned):
    """Codes and scales as the block-128 quantizer makes them of the float32 results; keys at their slots."""
    rng = np.random.default_rng(8)
    T, H, pool = 50, 64, 140
    q, k = rope_inputs(rng, T, H, 128, dtype, 2.0), rope_inputs(rng, T, 1, 128, dtype, 2.0)
    if not aligned:
        q, k = (torch.cat([x, x[:, :, :1]], 2)[:, :, :128] for x in (q, k))
    q[3, 5] = 0                                     # an empty block: scale 1, codes of zeros (0 c - 0 s is -0 where c < 0)
    cs, pos = dev(rope_table(77, 64)), rng.integers(0, 77, T)
    pos[7] = 77                                     # a token past the table: left out
    slots = rng.permutation(pool)[:T].astype(np.int64)
    slots[2], slots[4] = -1, pool
    w, b = dev((1 + 0.3 * rng.normal(size=128)).astype(np.float32)), dev(rng.normal(size=128).astype(np.float32))
    qc, qs = torch.full((T, H, 128), 99, dtype=torch.uint8, device="cuda"), torch.full((T, H), -5.0, device="cuda")
    kc, ks = torch.full((pool, 128), 99, dtype=torch.uint8, device="cuda"), torch.full((pool,), -5.0, device="cuda")
    st = status()
    args = dict(k_norm="layer", k_weight=w, k_bias=b)
    mt.norm_rope(dev(pos), cs, q=q, k=k, q_out=qc, q_scale=qs, k_out=kc, k_scale=ks, slots=dev(slots), dev_status=st, **args)
    assert st.item() == STATUS["ROW_RANGE"] | STATUS["WRITE_RANGE"]
    fq, fk = mt.norm_rope(dev(np.minimum(pos, 76)), cs, q=q, k=k, q_out=torch.empty(T, H, 128, device="cuda"),
                          k_out=torch.empty(T, 1, 128, device="cuda"), **args)
    wq, wqs = mt.quantize_fp8_block128(fq)
    wk, wks = mt.quantize_fp8_block128(fk.view(T, 128))
    ok = np.array([t for t in range(T) if t != 7])
    assert torch.equal(qc[ok], wq[ok]) and torch.equal(qs[ok], wqs.view(T, H)[ok])
    assert (qc[7] == 99).all() and (qs[7] == -5).all() and qs[3, 5] == 1 and (qc[3, 5] & 127 == 0).all()
    kept = [t for t in ok if t not in (2, 4)]
    at = dev(slots[kept])
    assert torch.equal(kc[at], wk[kept]) and torch.equal(ks[at], wks.view(-1)[kept])
    rest = torch.ones(pool, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert (kc[rest] == 99).all() and (ks[rest] == -5).all()


@pytest.mark.parametrize("fmt", [656, 416])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rot", [64, 0])
def test_norm_rope_into_latent_rows(mt, fmt, dtype, rot):
    """Cache rows equal the packing calls' rows of the float32 results."""
    rng = np.random.default_rng(fmt)
    for T in (1, 70):
        pool = 3 * T
        wide = rope_inputs(rng, T, 1, 640, dtype, 0.0).view(T, 640)
        kv = wide[:, 64:]                            # a view of a wider projection
        w = dev((1 + 0.3 * rng.normal(size=512)).astype(np.float32))
        cs, pos = (dev(rope_table(77, 64)), dev(rng.integers(0, 77, T))) if rot else (None, None)
        slots = rng.permutation(pool)[:T].astype(np.int64)
        if T > 1:
            slots[3], slots[5] = pool + 7, -2
        cache, st = torch.full((pool, fmt), 77, dtype=torch.uint8, device="cuda"), status()
        args = dict(k_norm="rms", k_weight=w, k_norm_dim=512, k_rot_start=512, interleaved=True)
        mt.norm_rope(pos, cs, k=kv, k_out=cache, slots=dev(slots), dev_status=st, **args)
        f, _ = mt.norm_rope(pos, cs, q=kv.unsqueeze(1), q_out=torch.empty(T, 1, 576, device="cuda"), q_norm="rms", q_weight=w,
                            q_norm_dim=512, q_rot_start=512, interleaved=True)
        rows = mt.pack_latent_fp8(f.view(T, 576)) if fmt == 656 else mt.pack_latent_fp4(f.view(T, 576))
        want = torch.full((pool, fmt), 77, dtype=torch.uint8, device="cuda")
        kept = [t for t in range(T) if T == 1 or t not in (3, 5)]
        want[dev(slots[kept])] = rows[kept]
        assert torch.equal(cache, want) and st.item() == (0 if T == 1 else STATUS["WRITE_RANGE"])
        # one head of three dimensions, whose head stride says nothing
        base = torch.zeros(T * 576 + 8, dtype=dtype, device="cuda")
        base[:T * 576].view(T, 576).copy_(kv)
        again = torch.empty(T, fmt, dtype=torch.uint8, device="cuda")
        mt.norm_rope(pos, cs, k=base.as_strided((T, 1, 576), (576, 577, 1)), k_out=again, **args)
        assert torch.equal(again, rows)
        # without slots: row t
        straight = torch.empty(T, fmt, dtype=torch.uint8, device="cuda")
        mt.norm_rope(pos, cs, k=kv, k_out=straight, **args)
        assert torch.equal(straight, rows)


def test_norm_rope_far_rows(mt):
    """Cache rows and queries past 2^31 elements."""
    rng = np.random.default_rng(3)
    T, D = 3, 128
    cache = torch.zeros((1 << 24) + 8, D, dtype=torch.bfloat16, device="cuda")       # 2^31 + 1024 values
    k = rope_inputs(rng, T, 1, D, torch.bfloat16)
    slots = dev(np.array([(1 << 24) + 7, 0, (1 << 24) - 1], np.int64))
    _, want = mt.norm_rope(None, None, k=k, k_norm="rms")
    mt.norm_rope(None, None, k=k, k_norm="rms", k_out=cache, slots=slots)
    assert torch.equal(cache[slots], want.view(T, D))
    big = torch.zeros((1 << 24) + 8, D, dtype=torch.bfloat16, device="cuda")
    far = big.as_strided((T, 1, D), ((1 << 30), D, 1))
    far.copy_(k)
    got, _ = mt.norm_rope(None, None, q=far, q_norm="rms")
    assert torch.equal(got, want)
    odd = big.as_strided((T, 1, 90), ((1 << 30) - 3, D, 1), 1)
    odd.copy_(k[:, :, :90])
    want, _ = mt.norm_rope(None, None, q=k[:, :, :90].contiguous(), q_norm="rms")
    got, _ = mt.norm_rope(None, None, q=odd, q_norm="rms")
    assert torch.equal(got, want)


def test_norm_rope_values_that_are_no_numbers(mt):
    """A NaN or infinity stays in its own head; zeros stay finite (eps 0: a head of zeros gives NaN as 0 / 0 does)."""
    x = torch.randn(4, 3, 128, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    clean, _ = mt.norm_rope(None, None, q=x, q_norm="rms")
    bad = x.clone()
    bad[1, 1, 5], bad[2, 0, 7], bad[3, 2] = math.nan, math.inf, 0.0
    got, _ = mt.norm_rope(None, None, q=bad, q_norm="rms")
    assert got[1, 1].isnan().all() and got[2, 0].isnan().any() and (got[3, 2] == 0).all()
    keep = torch.ones(4, 3, dtype=torch.bool, device="cuda")
    keep[1, 1] = keep[2, 0] = keep[3, 2] = False
    assert torch.equal(got[keep], clean[keep])


# ----------------------------------------------------------------------------- 4-bit rows

def latents(rng, T, wild):
    x = rng.normal(size=(T, 576))
    if wild:
        x *= np.exp(rng.uniform(-12, 14, (T, 1)))
        x[:, ::16] *= 30
        if T > 4:
            x[1] = 0
            x[2, 5], x[2, 40], x[3, 300] = np.inf, -np.inf, np.nan
            x[4, :64] = np.tile([6, -5, 3.5, 2.5, 1.75, 1.25, -0.75, 0.25], 8)      # every tie
    return x


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [1, 7, 300, 20000])
def test_pack_latent_fp4(mt, T, dtype):
    rng = np.random.default_rng(T)
    x = torch.tensor(latents(rng, T, T != 7)).to(dtype).cuda()
    want = o4.pack(x.float().cpu().numpy())
    got = mt.pack_latent_fp4(x).cpu().numpy()
    if T > 4 and T != 7:      # NaN has many bit patterns: rope values are finite here, blocks that hold one are 255 with zero codes
        assert want[3, 256 + 18] == 255 and want[2, 256] == 255
    assert np.array_equal(got, want)
    pool = T + 5
    slots = rng.permutation(pool)[:T].astype(np.int64)
    if T > 1:
        slots[0], slots[T - 1] = pool, -1
    cache, st = torch.full((pool, 416), 55, dtype=torch.uint8, device="cuda"), status()
    assert mt.pack_latent_fp4(x, cache, slots=dev(slots), dev_status=st) is cache
    full = np.full((pool, 416), 55, np.uint8)
    kept = range(1, T - 1) if T > 1 else range(T)
    full[slots[list(kept)]] = want[list(kept)]
    assert np.array_equal(cache.cpu().numpy(), full) and st.item() == (STATUS["WRITE_RANGE"] if T > 1 else 0)


def mla_case(rng, B, W, H, n_idx, lens, n_append=0):
    R = B * W
    pos = (np.asarray(lens)[:, None] + np.arange(W)).reshape(-1).astype(np.int64)        # visible: 0 .. pos
    idx = np.full((R, n_idx), -1, np.int32)
    for r in range(R):
        m = min(n_idx, int(pos[r]) + 1)
        idx[r, :m] = np.sort(rng.choice(int(pos[r]) + 1, m, replace=False))
        if m > 3 and r % 3 == 1:
            idx[r, rng.integers(0, m, 2)] = -1                                            # holes
    if R > 2:
        idx[R // 2] = -1                                                                  # nothing selected
    q = torch.tensor(rng.normal(size=(R, H, 576)) * 2).to(torch.bfloat16)
    caps = [int(n) + W + n_append for n in lens]
    rows = o4.pack(rng.normal(size=(sum(caps), 576)) * np.where(rng.random(576) < 0.02, 6, 1))
    start = np.concatenate([[0], np.cumsum(caps)[:-1]]).astype(np.int64)
    return q, rows, caps, start, pos, idx


def check_mla(out, lse, q, rows, start, W, idx, n_append=0, base=None, want_rows=None):
    R = len(idx)
    want = omla.sparse_mla(q, o4.unpack(rows), start, np.arange(R) // W, idx, SCALE, n_append, base,
                           rows=range(R) if want_rows is None else want_rows)
    o, s = out.float().cpu().numpy(), lse.cpu().numpy()
    for r, (wo, wl) in want.items():
        if not np.isfinite(wl).all():
            assert (o[r] == 0).all() and np.array_equal(s[r], wl)
            continue
        parity.check_attention_row(o[r], wo, parity.ATT_TOL_BF16)
        assert np.abs(s[r] - wl).max() <= 2e-2


@pytest.mark.parametrize("page", [0, 1, 4, 64])
@pytest.mark.parametrize("H", [16, 48, 128, 256])
def test_mla_over_4_bit_rows(mt, H, page):
    rng = np.random.default_rng(H + page)
    for B, W, n_idx, lens in ((1, 1, 1, [0]), (2, 3, 64, [70, 3]), (3, 2, 65, [0, 500, 63]), (2, 1, 700, [5000, 100]), (1, 2, 2048, [3000])):
        q, rows, caps, start, pos, idx = mla_case(rng, B, W, H, n_idx, lens)
        pool, paged, cs = rows, None, dev(start)
        if page:
            t = np.full((B, max(otab.n_pages(c, page) for c in caps) + 1), -1, np.int32)
            ids = rng.permutation(sum(otab.n_pages(c, page) for c in caps) + 2)
            at = 0
            pool = rng.integers(0, 256, (len(ids) * page, 416)).astype(np.uint8)          # unowned rows: noise
            pool[:, 256:288] |= 0                                                          # scales of any size, NaN among them
            for b in range(B):
                n = otab.n_pages(caps[b], page)
                t[b, :n] = ids[at:at + n]
                at += n
                for s in range(caps[b]):
                    pool[opaged.slot_of(t, page, b, s)] = rows[start[b] + s]
            paged, cs = (dev(t), page), None
        lse, st = torch.empty(B * W, H, device="cuda"), status()
        out = mt.sparse_mla_decode(q.cuda(), dev(pool), cs, u32(np.arange(B + 1) * W), dev(pos), dev(idx), SCALE, lse=lse,
                                   dev_status=st, paged=paged)
        assert st.item() == 0
        check_mla(out, lse, q, rows, start, W, idx)


@pytest.mark.parametrize("H", [64, 128])
def test_mla_over_4_bit_rows_appended_and_bad_entries(mt, H):
    rng = np.random.default_rng(H)
    B, W, n_idx, n_append = 4, 1, 200, 3
    q, rows, caps, start, pos, idx = mla_case(rng, B, W, H, n_idx, [900, 150, 0, 40], n_append)
    base = pos.copy()
    lse, st = torch.empty(B, H, device="cuda"), status()
    args = (q.cuda(), dev(rows), dev(start), u32(np.arange(B + 1)), dev(pos))
    out = mt.sparse_mla_decode(*args, dev(idx), SCALE, n_append=n_append, append_base=dev(base), row_pos_add=n_append, lse=lse,
                               dev_status=st)
    assert st.item() == 0
    check_mla(out, lse, q, rows, start, W, idx, n_append, base)
    bad = idx.copy()
    bad[0, 0], bad[1, 1] = 901, -3                   # past the row's position; negative, but no padding
    st = status()
    out = mt.sparse_mla_decode(*args, dev(bad), SCALE, lse=lse, dev_status=st)
    assert st.item() == STATUS["INDEX_RANGE"]
    good = np.where(bad == 901, -1, np.maximum(bad, -1))
    check_mla(out, lse, q, rows, start, W, good)
    far = dev(start + np.array([0, 0, len(rows), 0]))   # a request whose rows lie outside the pool
    st = status()
    out = mt.sparse_mla_decode(args[0], args[1], far, args[3], args[4], dev(np.abs(idx) * 0), SCALE, lse=lse, dev_status=st)
    assert st.item() == STATUS["ROW_RANGE"] and (out[2] == 0).all() and (lse[2] == -math.inf).all()


def test_mla_reads_no_row_that_is_not_selected(mt):
    """NaN scales in every other row of the cache, in bf16 rope values too."""
    rng = np.random.default_rng(77)
    q, rows, caps, start, pos, idx = mla_case(rng, 2, 2, 128, 300, [2000, 700])
    used = np.zeros(len(rows), bool)
    for r in range(4):
        used[start[r // 2] + idx[r][idx[r] >= 0]] = True
    rows[~used, 256:] = 255
    lse, st = torch.empty(4, 128, device="cuda"), status()
    out = mt.sparse_mla_decode(q.cuda(), dev(rows), dev(start), u32([0, 2, 4]), dev(pos), dev(idx), SCALE, lse=lse, dev_status=st)
    check_mla(out, lse, q, rows, start, 2, idx)


def test_mla_large_logits(mt):
    """Scores up to several hundred: the reference maximum moves, and one position takes all the weight."""
    rng = np.random.default_rng(78)
    q, rows, caps, start, pos, idx = mla_case(rng, 1, 2, 128, 512, [4000])
    q = (q.float() * 40).to(torch.bfloat16)
    order = np.argsort((q[0].float().numpy() @ o4.unpack(rows)[:4000].T).mean(0))         # rising scores: the maximum moves in every tile
    idx[0] = order[-512:]
    lse = torch.empty(2, 128, device="cuda")
    out = mt.sparse_mla_decode(q.cuda(), dev(rows), dev(start), u32([0, 2]), dev(pos), dev(idx), SCALE, lse=lse)
    want = omla.sparse_mla(q, o4.unpack(rows), start, [0, 0], idx, SCALE)
    for r in range(2):
        # a score s has an error of up to 2^-11 s (its half-precision partials) and weighs its position by it
        top = np.abs(want[r][1]).max()
        tol = 2e-2 + 2 * (math.exp(2.0 ** -11 * top * 2) - 1)
        assert np.linalg.norm(out[r].float().cpu().numpy() - want[r][0]) <= tol * np.linalg.norm(want[r][0])


def test_caches_of_4_bit_rows_move_and_write_back(mt):
    """The write-back, by position and by slot, and the accepted-KV move take 416-byte rows."""
    rng = np.random.default_rng(9)
    B, W, pool = 5, 4, 90
    src = rng.integers(0, 256, (B, W, 416)).astype(np.uint8)
    n_acc = np.array([0, 3, 1, 2, 9], np.int32)
    start, dpos = np.arange(B).astype(np.int64) * 18, np.array([0, 3, 5, 7, 9], np.int64)
    dst = rng.integers(0, 256, (pool, 416)).astype(np.uint8)
    a, nxt = dev(dst), torch.empty(B, dtype=torch.int64, device="cuda")
    mt.kv_writeback(dev(src), None, None, dev(n_acc), a, None, None, dev(start), dev(dpos), next_pos=nxt)
    slots = start[:, None] + dpos[:, None] + np.arange(W)
    c = dev(dst)
    mt.kv_writeback_slots(dev(src), None, None, dev(n_acc), c, None, None, dev(slots))
    want = dst.copy()
    for b in range(B):
        k = min(int(n_acc[b]) + 1, W)
        want[slots[b, :k]] = src[b, :k]
    assert np.array_equal(a.cpu().numpy(), want) and np.array_equal(c.cpu().numpy(), want)
    acc = np.tile(np.arange(W)[::-1].astype(np.int32), (B, 1)).copy()
    mt.kv_move_accepted(a, None, None, dev(slots), dev(acc), dev(n_acc))
    moved = want.copy()
    for b in range(B):
        k = min(int(n_acc[b]) + 1, W)
        moved[slots[b, :k]] = want[slots[b, acc[b, :k]]]
    assert np.array_equal(a.cpu().numpy(), moved)


def test_empty_calls(mt):
    """No tokens, no rows, no selected entries: nothing is written, or zeros and -inf."""
    z = lambda *sh, dtype=torch.bfloat16: torch.empty(*sh, dtype=dtype, device="cuda")  # noqa: E731
    cs, pos = dev(rope_table(9, 64)), z(0, dtype=torch.int64)
    q, k = mt.norm_rope(pos, cs, q=z(0, 4, 128), k=z(0, 128), q_norm="rms")
    assert q.shape == (0, 4, 128) and k.shape == (0, 128)
    cache = torch.full((5, 416), 7, dtype=torch.uint8, device="cuda")
    mt.norm_rope(pos, cs, k=z(0, 576), k_rot_start=512, k_out=cache, slots=pos)
    mt.pack_latent_fp4(z(0, 576), cache, slots=pos)
    assert mt.pack_latent_fp4(z(0, 576)).shape == (0, 416) and (cache == 7).all()
    for H in (16, 128):
        lse = torch.zeros(2, H, device="cuda")
        out = mt.sparse_mla_decode(torch.ones(2, H, 576, dtype=torch.bfloat16, device="cuda"), cache, dev([0]), u32([0, 2]), dev([3, 4]),
                                   z(2, 0, dtype=torch.int32), SCALE, lse=lse)
        assert (out == 0).all() and (lse == -math.inf).all()
        none = mt.sparse_mla_decode(z(0, H, 576), cache, dev([0]), u32([0, 0]), pos, z(0, 8, dtype=torch.int32), SCALE)
        assert none.shape == (0, H, 512)
