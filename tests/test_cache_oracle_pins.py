"""The oracle of the calls that fill the caches against worked examples and closed forms, the C structures' layout, and the host-side
refusals of those calls.  CPU only (no launch)."""
import ctypes as C

import numpy as np
import pytest

from oracle import latent4, paged, rope, tables
from test_abi import _c_offsets, native  # noqa: F401


# ----------------------------------------------------------------------------- block tables

def test_grow_worked_example():
    free = np.array([10, 11, 12, 13, 14, 15, 99], np.int32)
    t = np.full((3, 4), -1, np.int32)
    t[0, :2], t[2, :1] = [1, 2], [3]
    # request 0: 5 -> 9 tokens of pages of 4 (2 -> 3 pages), 1: 0 -> 8 (2 pages), 2: 4 -> 4 (none)
    out, lengths, left, st = tables.grow(t, 4, [9, 8, 4], free, 6, [5, 0, 4])
    assert out.tolist() == [[1, 2, 15, -1], [14, 13, -1, -1], [3, -1, -1, -1]]
    assert lengths.tolist() == [9, 8, 4] and left == 3 and st == 0
    # two pages free: the first request takes one, the second is not served, the third needs none
    out, lengths, left, st = tables.grow(t, 4, [9, 8, 3], free, 2, [5, 0, 4])
    assert out.tolist() == [[1, 2, 11, -1], [-1] * 4, [3, -1, -1, -1]]
    assert lengths.tolist() == [9, 0, 4] and left == 1 and st == tables.NO_PAGES
    # built anew; a length past the row
    out, lengths, left, st = tables.grow(t, 4, [1, 17, 16], free, 6)
    assert out.tolist() == [[15, -1, -1, -1], [-1] * 4, [14, 13, 12, 11]]
    assert lengths.tolist() == [1, 0, 16] and left == 1 and st == tables.ROW_RANGE


def test_release_returns_what_grow_took():
    rng = np.random.default_rng(0)
    for ps in (1, 4, 64):
        B, width = 9, 12
        free = rng.permutation(200).astype(np.int32)
        t = np.full((B, width), -1, np.int32)
        new = rng.integers(0, width * ps + 1, B)
        out, _, left, st = tables.grow(t, ps, new, free, 200)
        assert st == 0
        back, again, n, st = tables.release(out, ps, new, free, left)
        assert st == 0 and n == 200 and (back == -1).all() and sorted(again.tolist()) == list(range(200))
        keep = new // 2
        back, again, n, st = tables.release(out, ps, new, free, left, keep)
        assert n - left == sum(tables.n_pages(int(a), ps) - tables.n_pages(int(k), ps) for a, k in zip(new, keep))


def test_slot_map_agrees_with_the_window_plan():
    rng = np.random.default_rng(1)
    t = rng.permutation(60).astype(np.int32).reshape(6, 10)
    t[2, 3] = -1
    start = np.array([0, 5, 11, 17, 38, 30], np.int64)
    W = 4
    want = paged.assign_cache_locs(t, 4, start, W)
    slots, pos, written, st = tables.slot_map(t, 4, np.arange(7) * W, start + W, 24)
    assert np.array_equal(slots.reshape(6, W), want) and written.all() and st == tables.ROW_RANGE
    assert np.array_equal(pos.reshape(6, W), start[:, None] + np.arange(W))


# ----------------------------------------------------------------------------- norms and rotation

def test_norms_closed_forms():
    x = np.array([[3.0, -4.0, 7.0]])
    assert np.allclose(rope.norm(x, "rms", 0.0, norm_dim=2), [[3 / np.sqrt(12.5), -4 / np.sqrt(12.5), 7.0]])
    assert np.allclose(rope.norm(x, "layer", 0.0, norm_dim=2), [[1.0, -1.0, 7.0]])
    assert np.allclose(rope.norm(x, "rms", 12.5, [2.0, 1.0], [1.0, 0.0], 2), [[6 / 5 + 1, -4 / 5, 7.0]])
    assert np.array_equal(rope.norm(x, None, 1.0), x)


def test_rotation_closed_forms():
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    quarter = np.array([[0.0, 0.0, 1.0, 1.0]])           # two pairs by 90 degrees
    assert rope.rotate(x, quarter, 2, False).tolist() == [[[1, 2, -5, -6, 3, 4, 7, 8]]]
    assert rope.rotate(x, quarter, 2, True).tolist() == [[[1, 2, -4, 3, -6, 5, 7, 8]]]
    rng = np.random.default_rng(2)
    ang = rng.uniform(0, 7, (5, 3))
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    y = rng.normal(size=(5, 2, 6))
    for inter in (False, True):
        z = rope.rotate(y, cs, 0, inter)
        assert np.allclose(np.linalg.norm(z, axis=2), np.linalg.norm(y, axis=2))
        assert np.allclose(rope.rotate(z, cs * [1, 1, 1, -1, -1, -1], 0, inter), y)


# ----------------------------------------------------------------------------- 4-bit rows

def test_scale_codes():
    assert latent4.SCALES[0] == 0 and latent4.SCALES[128] == 1.0 and latent4.SCALES[129] == 1.125 and np.isnan(latent4.SCALES[255])
    assert latent4.SCALES[1] == 2.0 ** -16 * 1.125 and latent4.SCALES[254] == 2.0 ** 15 * 1.75
    assert (np.diff(latent4.SCALES[:255]) > 0).all()


def test_row_worked_example():
    x = np.zeros((1, 576), np.float32)
    x[0, :8] = [6, -3, 0.25, 0.75, -0.0, 2.5, 5.0, -100 / 3]     # amax 33.3 / 6 = 5.56 -> scale 5.5 (code 147)
    x[0, 16:24] = [0.5, -0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 6.0]   # scale 1: every tie
    x[0, 32] = 2.0 ** -30                                         # below half the least scale
    x[0, 48] = np.inf
    x[0, 64] = 1e9                                                # past the greatest scale
    x[0, 512], x[0, 575] = 1.00390625, -2.0                       # a bf16 tie
    r = latent4.pack(x)[0]
    assert r[256:261].tolist() == [147, 128, 0, 255, 254] and (r[261:288] == 0).all()
    # values 0..7 in units of 5.5: 1.09 -> 1, -0.55 -> -0.5, 0, 0.14 -> 0, -0, 0.45 -> 0.5, 0.91 -> 1, -6.06 -> -6
    nib = [2, 9, 0, 0, 8, 1, 2, 15]
    word = sum(n << (4 * (i // 2) + 16 * (i % 2)) for i, n in enumerate(nib))
    assert int.from_bytes(bytes(r[:4]), "little") == word
    # ties go to the even code: -0.25 -> -0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4
    nib = [1, 8, 2, 2, 4, 4, 6, 7]
    word = sum(n << (4 * (i // 2) + 16 * (i % 2)) for i, n in enumerate(nib))
    assert int.from_bytes(bytes(r[8:12]), "little") == word
    y = latent4.unpack(r[None])[0]
    assert y[:8].tolist() == [5.5, -2.75, 0, 0, 0, 2.75, 5.5, -33.0] and y[16:24].tolist() == [0.5, 0, 1, 1, 2, 2, 4, 6]
    assert y[32] == 0 and np.isnan(y[48:64]).all() and y[64] == 6 * 57344 and y[512] == 1.0 and y[575] == -2.0


def test_rows_error_bound():
    """A scale is off by at most 1/16 of itself, so |x| <= 6.4 scales; a code by half its step, at most 1 (between 4 and 6), or
    what is cut above 6."""
    rng = np.random.default_rng(3)
    x = (rng.normal(size=(50, 576)) * np.exp(rng.uniform(-6, 6, (50, 1)))).astype(np.float32)
    y = latent4.unpack(latent4.pack(x))
    amax = np.abs(x[:, :512].reshape(50, 32, 16)).max(axis=2, keepdims=True)
    err = np.abs(y - x)[:, :512].reshape(50, 32, 16)
    assert (err <= amax / 6 * (17 / 16) * (1 + 1e-6)).all()
    for c in range(1, 255):       # every scale times every code is a bf16 value
        v = latent4.SCALES[c] * latent4.MAGNITUDES
        bits = v.astype(np.float32).view(np.uint32)
        assert (v == v.astype(np.float32)).all() and (bits & 0xffff == 0).all()


# ----------------------------------------------------------------------------- C structures and refusals

@pytest.mark.parametrize("cname,pyname", [("mtpsd_block_table_args", "BlockTableArgs"), ("mtpsd_head_side", "HeadSide")])
def test_struct_layout(native, cname, pyname):  # noqa: F811
    st = getattr(native, pyname)
    fields = [f for f, _ in st._fields_]
    got = _c_offsets(cname, fields)
    assert got[0] == C.sizeof(st) and got[1:] == [getattr(st, f).offset for f in fields]


def test_table_refusals(native):  # noqa: F811
    lib, N = native.lib(), native
    good = dict(block_table=8, bt_stride=4, page_size=16, B=2, free_cap=8, new_len=8, free_pages=8, n_free=8, n_free_out=8)
    grow = lambda **k: lib.mtpsd_block_table_grow(C.byref(N.BlockTableArgs(**{**good, **k})), None)  # noqa: E731
    assert lib.mtpsd_block_table_grow(None, None) == N.MTPSD_EINVAL
    for bad in (dict(page_size=0), dict(page_size=48), dict(page_size=1 << 17), dict(bt_stride=0), dict(B=-1), dict(free_cap=-1),
                dict(block_table=None), dict(new_len=None), dict(free_pages=None), dict(n_free=None), dict(n_free_out=None),
                dict(new_len=4), dict(block_table=2), dict(old_len=12), dict(lengths=20), dict(lengths=8),
                dict(token_offsets=8, T=5), dict(token_offsets=8, T=-1, slots=8), dict(token_offsets=8, T=1 << 32, slots=8),
                dict(token_offsets=2, T=5, slots=8), dict(token_offsets=8, T=5, slots=12), dict(dev_status=2)):
        assert grow(**bad) == N.MTPSD_EINVAL, bad
        assert b"block_table_grow" in lib.mtpsd_last_error()
    assert grow(B=8193) == N.MTPSD_EUNSUPPORTED
    release = lambda *a: lib.mtpsd_block_table_release(*a, None, None)  # noqa: E731
    assert release(8, 4, 16, 0, 8, None, 8, 8, 8) == N.MTPSD_OK
    for bad in ((8, 4, 3, 2, 8, None, 8, 8, 8), (8, 0, 16, 2, 8, None, 8, 8, 8), (8, 4, 16, -1, 8, None, 8, 8, 8),
                (None, 4, 16, 2, 8, None, 8, 8, 8), (8, 4, 16, 2, None, None, 8, 8, 8), (8, 4, 16, 2, 8, None, None, 8, 8),
                (8, 4, 16, 2, 8, None, 8, 8, None), (8, 4, 16, 2, 12, None, 8, 8, 8), (8, 4, 16, 2, 8, 4, 8, 8, 8),
                (8, 4, 16, 2, 8, None, 8, -1, 8)):
        assert release(*bad) == N.MTPSD_EINVAL, bad
    assert release(8, 4, 16, 8193, 8, None, 8, 8, 8) == N.MTPSD_EUNSUPPORTED
    pk = N.PagedKV(block_table=8, bt_stride=4, page_size=16)
    smap = lambda p, *a: lib.mtpsd_slot_map(C.byref(p) if p else None, *a, None, None, None)  # noqa: E731
    assert smap(pk, 0, 8, 8, 4, 8) == N.MTPSD_OK and smap(pk, 2, 8, 8, 0, None) == N.MTPSD_OK
    for bad in ((None, 2, 8, 8, 4, 8), (N.PagedKV(block_table=8, bt_stride=4, page_size=5), 2, 8, 8, 4, 8),
                (N.PagedKV(block_table=None, bt_stride=4, page_size=4), 2, 8, 8, 4, 8), (pk, -1, 8, 8, 4, 8),
                (pk, 2, None, 8, 4, 8), (pk, 2, 8, None, 4, 8), (pk, 2, 8, 8, 4, None), (pk, 2, 8, 8, -1, 8),
                (pk, 2, 8, 8, 1 << 32, 8), (pk, 2, 8, 4, 4, 8)):
        assert smap(*bad) == N.MTPSD_EINVAL, bad


def test_norm_rope_refusals(native):  # noqa: F811
    lib, N = native.lib(), native
    good = dict(x=16, x_token_stride=128, x_head_stride=128, heads=1, D=128, dtype=N.MTPSD_BF16, norm=0, norm_dim=0, rot_start=0,
                out=32, out_token_stride=128, out_head_stride=128, out_dtype=N.MTPSD_BF16)

    def call(q=None, k=None, T=2, pos=8, cs=16, n_pos=10, rot=64, eps=0.0, slots=None, pool=0):
        q, k = (None if s is None else C.byref(N.HeadSide(**{**good, **s})) for s in (q, k))
        return lib.mtpsd_norm_rope(q, k, T, pos, cs, n_pos, rot, 0, eps, slots, pool, None, None)

    assert call() == N.MTPSD_EINVAL                                       # neither side
    assert call(q={}, T=0) == N.MTPSD_OK
    for bad in (dict(T=-1), dict(T=1 << 31), dict(rot=3), dict(rot=-2), dict(rot=2000), dict(eps=-1.0), dict(eps=float("nan")),
                dict(pos=None), dict(cs=None), dict(n_pos=-1), dict(pos=4), dict(cs=2), dict(slots=8)):
        assert call(q={}, **bad) == N.MTPSD_EINVAL, bad
    for bad in (dict(heads=0), dict(heads=65536), dict(D=0), dict(D=1025), dict(norm=3), dict(norm=1, norm_dim=0),
                dict(norm=1, norm_dim=129), dict(weight=16), dict(rot_start=-1), dict(rot_start=65), dict(x=None), dict(out=None),
                dict(x=17), dict(out=33), dict(x_token_stride=-1), dict(out=16, out_token_stride=256),
                dict(out=16, out_dtype=N.MTPSD_F32), dict(out_dtype=N.MTPSD_FP8_E4M3), dict(weight=6, norm=1, norm_dim=8)):
        assert call(q=bad) == N.MTPSD_EINVAL, bad
        assert b"norm_rope" in lib.mtpsd_last_error()
    for bad in (dict(dtype=2), dict(out_dtype=9), dict(out_dtype=N.MTPSD_FP8_E4M3, D=64), dict(out_dtype=N.MTPSD_FP4_MLA, D=576),
                dict(out_dtype=N.MTPSD_FP8_DS_MLA)):
        assert call(q=bad) == N.MTPSD_EUNSUPPORTED, bad
    assert call(q=dict(heads=2), T=1 << 30) == N.MTPSD_EUNSUPPORTED
    assert call(k=dict(out=16), slots=8, pool=4) == N.MTPSD_EINVAL         # in place into a cache
    assert call(k={}, slots=8, pool=-1) == N.MTPSD_EINVAL
    row = dict(D=576, rot_start=512, out_dtype=N.MTPSD_FP4_MLA, out_token_stride=416, x_token_stride=576)
    for bad in (dict(heads=2), dict(rot_start=256), dict(norm=1, norm_dim=576), dict(norm=1, norm_dim=500), dict(x=18),
                dict(x_token_stride=577), dict(norm=1, norm_dim=512, weight=20)):
        assert call(k={**row, **bad}) == N.MTPSD_EUNSUPPORTED, bad
    assert call(k=row, rot=32) == N.MTPSD_EUNSUPPORTED and call(k=row, cs=20) == N.MTPSD_EUNSUPPORTED
    for bad in (dict(out_token_stride=400), dict(out_token_stride=424), dict(out=40)):
        assert call(k={**row, **bad}) == N.MTPSD_EINVAL, bad


def test_latent4_refusals(native):  # noqa: F811
    lib, N = native.lib(), native
    pack = lambda *a: lib.mtpsd_pack_latent_fp4(*a, None, None)  # noqa: E731
    assert pack(None, N.MTPSD_BF16, 0, None, None, 0) == N.MTPSD_OK
    for bad in ((16, 1, -1, 16, None, 4), (16, 1, 5, 16, None, 4), (16, 1, 2, 16, 8, -1), (None, 1, 2, 16, None, 4),
                (16, 1, 2, None, None, 4), (24, 1, 2, 16, None, 4), (16, 1, 2, 24, None, 4), (16, 1, 2, 16, 4, 4)):
        assert pack(*bad) == N.MTPSD_EINVAL, bad
    assert pack(16, N.MTPSD_FP8_E4M3, 2, 16, None, 4) == N.MTPSD_EUNSUPPORTED
    m = dict(B=1, R=1, d_latent=576, d_v=512, n_idx=16, dtype=N.MTPSD_FP4_MLA)
    assert lib.mtpsd_sparse_mla_decode(C.byref(N.MlaArgs(n_heads=20, **m)), None) == N.MTPSD_EUNSUPPORTED
    assert lib.mtpsd_sparse_mla_decode(C.byref(N.MlaArgs(n_heads=16, **m)), None) == N.MTPSD_EINVAL
    m = N.MlaArgs(n_heads=16, q=16, latent=24, cache_start=8, row_offsets=8, row_pos=8, idx=8, out=16, **m)
    assert lib.mtpsd_sparse_mla_decode(C.byref(m), None) == N.MTPSD_EINVAL
